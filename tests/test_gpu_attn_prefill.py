"""Causal attention over packed prompts and its gradients on the GPU against
plain 64-bit attention (attn_ref), elementwise within the bound that the
number formats allow."""

import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu

HEADS = [(16, 16), (32, 32), (64, 64), (128, 128), (192, 128)]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _inputs(seed, lens, H, Hkv, dk, dv, dtype, gate, spare=0, size=1.0):
    """Packed inputs; `spare` rows behind the last sequence hold NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, n = sum(lens) + spare, sum(lens)
    new = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    x = {"q": new(T, H, dk) * size, "k": new(T, Hkv, dk), "v": new(T, Hkv, dv), "dy": new(T, H, dv),
         "z": new(T, H, dv) if gate else None}
    for name, t in x.items():
        if t is not None:
            t[n:] = float("nan")
            x[name] = t.to(dtype)
    return x


def _64(x):
    return None if x is None else x.double()


def _forward(K, x, lens, scale=None):
    T, H, dv = x["q"].shape[0], x["q"].shape[1], x["v"].shape[2]
    out = torch.full((T, H, dv), 7.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    K.kda_attn_prefill(x["q"], x["k"], x["v"], out_gate=x["z"], cu_seqlens=_cu(lens), out=out, lse=lse, scale=scale)
    torch.cuda.synchronize()
    return out, lse


def _check_forward(K, x, lens, dtype, scale=None):
    n, sc = sum(lens), scale or x["q"].shape[2] ** -0.5
    out, lse = _forward(K, x, lens, scale)
    want, bo, wl, bl = R.prefill(_64(x["q"]), _64(x["k"]), _64(x["v"]), _64(x["z"]), lens, sc, dtype)
    R.check("out", out[:n], want[:n], bo[:n])
    R.check("lse", lse[:n], wl[:n], bl[:n])
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all()), "rows behind the last sequence were written"
    return out, lse


def _check_backward(K, x, lens, dtype, out, lse):
    n = sum(lens)
    g = K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], out, lse, x["dy"], out_gate=x["z"], cu_seqlens=_cu(lens))
    torch.cuda.synchronize()
    want = R.backward(*(_64(x[t]) for t in ("q", "k", "v", "z", "dy")), lens, x["q"].shape[2] ** -0.5, dtype)
    for name, w in want.items():
        assert (w is None) == (g[name] is None)
        if w is not None:
            assert g[name].dtype == dtype
            R.check(name, g[name][:n], w[0][:n], w[1][:n])
    return g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_ragged_batch(K, dk, dv, dtype):
    """Empty, one-token and ragged sequences, shared heads, a gate, spare rows."""
    lens = [129, 1, 0, 63, 200, 64, 0]
    print(f"ragged {dk}/{dv} {dtype}", flush=True)
    x = _inputs(dk + dv, lens, 4, 2, dk, dv, TYPES[dtype], True, spare=5)
    out, lse = _check_forward(K, x, lens, TYPES[dtype])
    _check_backward(K, x, lens, TYPES[dtype], out, lse)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [127], [128], [255, 257], [700]])
def test_lengths(K, lens, dtype):
    print(f"lengths {lens} {dtype}", flush=True)
    x = _inputs(sum(lens), lens, 2, 1, 64, 64, TYPES[dtype], False)
    out, lse = _check_forward(K, x, lens, TYPES[dtype])
    _check_backward(K, x, lens, TYPES[dtype], out, lse)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 3), (8, 1), (5, 5), (32, 8)])
def test_head_layouts(K, H, Hkv):
    lens = [150, 40]
    print(f"heads {H}/{Hkv}", flush=True)
    x = _inputs(H, lens, H, Hkv, 128, 128, torch.bfloat16, H == 6)
    out, lse = _check_forward(K, x, lens, torch.bfloat16)
    _check_backward(K, x, lens, torch.bfloat16, out, lse)


def test_longer_sequences(K):
    """Several query tiles per sequence, tiles of every level."""
    lens = [1500, 300, 900]
    x = _inputs(5, lens, 4, 2, 128, 128, torch.bfloat16, True)
    out, lse = _check_forward(K, x, lens, torch.bfloat16)
    _check_backward(K, x, lens, torch.bfloat16, out, lse)


def test_many_sequences(K):
    """More sequences than lanes: the tile search takes several passes."""
    lens = [(i * 37) % 19 for i in range(150)] + [300] + [(i * 11) % 7 for i in range(70)]
    x = _inputs(6, lens, 2, 2, 32, 32, torch.float32, False)
    out, lse = _check_forward(K, x, lens, torch.float32)
    _check_backward(K, x, lens, torch.float32, out, lse)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steep_softmax(K, dtype):
    """Scores of several hundred: nothing overflows, the running maximum carries."""
    lens = [300, 77]
    x = _inputs(7, lens, 2, 2, 64, 64, TYPES[dtype], False, size=60.0)
    x["k"][150:160] *= 4
    _check_forward(K, x, lens, TYPES[dtype])


def test_rising_scores(K):
    """Every key above all before it: the maximum moves at each tile."""
    n = 400
    x = _inputs(8, [n], 1, 1, 32, 32, torch.float32, False)
    x["q"][:] = 1.0
    x["k"][:] = torch.linspace(0, 40, n, device="cuda")[:, None, None]
    _check_forward(K, x, [n], torch.float32, scale=0.25)


def test_scale(K):
    x = _inputs(9, [90], 2, 1, 64, 64, torch.float32, False)
    _check_forward(K, x, [90], torch.float32, scale=1.0)


def test_no_sequence_reads_another(K):
    """NaN and infinity in one sequence leave the others' bits alone."""
    lens = [70, 50, 33]
    for dtype in (torch.float32, torch.bfloat16):
        x = _inputs(10, lens, 2, 1, 64, 64, dtype, True)
        out, lse = _forward(K, x, lens)
        g = K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], out, lse, x["dy"], out_gate=x["z"], cu_seqlens=_cu(lens))
        y = {n: t.clone() for n, t in x.items()}
        for n, t in y.items():
            t[70:120] = float("nan") if n != "k" else float("inf")
        out2, lse2 = _forward(K, y, lens)
        g2 = K.kda_attn_prefill_backward(y["q"], y["k"], y["v"], out2, lse2, y["dy"], out_gate=y["z"], cu_seqlens=_cu(lens))
        torch.cuda.synchronize()
        for r in (slice(0, 70), slice(120, 153)):
            assert torch.equal(out[r], out2[r]) and torch.equal(lse[r], lse2[r])
            for n in g:
                assert torch.equal(g[n][r], g2[n][r]), n


def test_gradients_against_differences(K):
    """fp32 gradients against central differences of the 64-bit forward."""
    lens = [9, 5]
    x = _inputs(11, lens, 2, 1, 16, 16, torch.float32, True)
    out, lse = _forward(K, x, lens)
    g = K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], out, lse, x["dy"], out_gate=x["z"], cu_seqlens=_cu(lens))
    d = {n: t.double() for n, t in x.items()}

    def loss(y):
        o = R.prefill(y["q"], y["k"], y["v"], y["z"], lens, 0.25, torch.float32)[0]
        return float((o * y["dy"]).sum())

    r = torch.Generator().manual_seed(1)
    for name, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("z", "dz")):
        for _ in range(6):
            way = torch.randn(d[name].shape, generator=r).double().cuda()
            h = 1e-5
            up, down = dict(d), dict(d)
            up[name], down[name] = d[name] + h * way, d[name] - h * way
            want = (loss(up) - loss(down)) / (2 * h)
            got = float((g[gn].double() * way).sum())
            # each of the gradient's values is within 2^-17 of its magnitude here; the difference is exact to h^2
            bound = float((g[gn].double().abs() * way.abs()).sum()) * 2.0 ** -17 + 1e-6
            assert abs(got - want) <= bound, (name, got, want, bound)


def test_same_bits_twice(K):
    """No result depends on timing."""
    lens = [500, 130, 7]
    x = _inputs(12, lens, 8, 2, 128, 128, torch.bfloat16, True)
    one = _forward(K, x, lens)
    two = _forward(K, x, lens)
    a = K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], *one, x["dy"], out_gate=x["z"], cu_seqlens=_cu(lens))
    b = K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], *two, x["dy"], out_gate=x["z"], cu_seqlens=_cu(lens))
    assert all(torch.equal(u, w) for u, w in zip(one, two))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_captured_and_replayed(K):
    """Forward and backward in one graph, replayed on changing inputs with
    eager work between the replays."""
    lens = [200, 60]
    cu = _cu(lens)
    x = _inputs(13, lens, 4, 2, 64, 64, torch.bfloat16, True)
    ws = torch.empty(K.kda_attn_backward_workspace_bytes(260, 2, 4, 2, 64, 64, torch.bfloat16, True), dtype=torch.uint8,
                     device="cuda")

    def step():
        o, l = K.kda_attn_prefill(x["q"], x["k"], x["v"], out_gate=x["z"], cu_seqlens=cu)
        return o, l, K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], o, l, x["dy"], out_gate=x["z"], cu_seqlens=cu,
                                                 workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l, g = step()
    for i in range(4):
        y = _inputs(20 + i, lens, 4, 2, 64, 64, torch.bfloat16, True)
        for n in x:
            x[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, l, *g.values())]
        eo, el, eg = step()
        torch.cuda.synchronize()
        assert all(torch.equal(u, w) for u, w in zip(got, (eo, el, *eg.values()))), i


def test_on_another_stream(K):
    lens = [300]
    x = _inputs(14, lens, 4, 4, 128, 128, torch.bfloat16, False)
    want = _forward(K, x, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = K.kda_attn_prefill(x["q"], x["k"], x["v"], cu_seqlens=_cu(lens))
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refuses(K):
    x = _inputs(15, [20], 4, 2, 64, 64, torch.float32, False)
    with pytest.raises(ValueError):
        K.kda_attn_prefill(x["q"].transpose(0, 1), x["k"], x["v"])  # another shape
    with pytest.raises(ValueError):
        K.kda_attn_prefill(x["q"][:, ::2], x["k"], x["v"])  # not contiguous
    with pytest.raises(TypeError):
        K.kda_attn_prefill(x["q"], x["k"].bfloat16(), x["v"])
    with pytest.raises(ValueError):
        K.kda_attn_prefill(x["q"], x["k"].cpu(), x["v"])
    with pytest.raises(Exception, match="does not divide"):
        K.kda_attn_prefill(x["q"][:, :3].contiguous(), x["k"], x["v"])
    with pytest.raises(Exception, match="scale"):
        K.kda_attn_prefill(x["q"], x["k"], x["v"], scale=0.0)


def test_empty_batch(K):
    e = lambda h, d: torch.empty((0, h, d), device="cuda")  # noqa: E731
    out, lse = K.kda_attn_prefill(e(2, 64), e(1, 64), e(1, 64))
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    g = K.kda_attn_prefill_backward(e(2, 64), e(1, 64), e(1, 64), out, lse, e(2, 64), out_gate=e(2, 64))
    assert g["dz"].shape == (0, 2, 64)
