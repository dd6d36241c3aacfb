"""Attention with a sliding window and first tokens that stay visible over
packed prompts, and its gradients, on the GPU against plain 64-bit attention
(attn_ref), elementwise within the bound that the number formats allow."""

import pytest
import torch

import attn_ref as R
from test_gpu_attn_prefill import HEADS, TYPES, _64, _cu, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


def _forward(K, x, lens, window, sinks, scale=None):
    T, H, dv = x["q"].shape[0], x["q"].shape[1], x["v"].shape[2]
    out = torch.full((T, H, dv), 7.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    K.kda_attn_window_prefill(x["q"], x["k"], x["v"], window, sinks=sinks, out_gate=x["z"], cu_seqlens=_cu(lens), out=out, lse=lse,
                              scale=scale)
    torch.cuda.synchronize()
    return out, lse


def _backward(K, x, lens, window, sinks, out, lse, **kw):
    return K.kda_attn_window_prefill_backward(x["q"], x["k"], x["v"], out, lse, x["dy"], window, sinks=sinks, out_gate=x["z"],
                                              cu_seqlens=_cu(lens), **kw)


def _check(K, x, lens, window, sinks, dtype):
    n, sc = sum(lens), x["q"].shape[2] ** -0.5
    out, lse = _forward(K, x, lens, window, sinks)
    view = R.windowed(window, sinks)
    want, bo, wl, bl = R.prefill(_64(x["q"]), _64(x["k"]), _64(x["v"]), _64(x["z"]), lens, sc, dtype, view)
    R.check("out", out[:n], want[:n], bo[:n])
    R.check("lse", lse[:n], wl[:n], bl[:n])
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all()), "rows behind the last sequence were written"
    g = _backward(K, x, lens, window, sinks, out, lse)
    torch.cuda.synchronize()
    ref = R.backward(*(_64(x[t]) for t in ("q", "k", "v", "z", "dy")), lens, sc, dtype, view)
    for name, w in ref.items():
        assert (w is None) == (g[name] is None)
        if w is not None:
            assert g[name].dtype == dtype
            R.check(name, g[name][:n], w[0][:n], w[1][:n])
    return out, lse, g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_ragged_batch(K, dk, dv, dtype):
    """Empty, one-token and ragged sequences, shared heads, a gate, spare rows."""
    lens = [129, 1, 0, 63, 300, 64, 0]
    print(f"window ragged {dk}/{dv} {dtype}", flush=True)
    x = _inputs(dk + dv, lens, 4, 2, dk, dv, TYPES[dtype], True, spare=5)
    _check(K, x, lens, 50, 3, TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (31, 0), (32, 32), (33, 5), (64, 0), (64, 65), (100, 3), (127, 64), (128, 1),
                                          (129, 130), (193, 0), (300, 4), (10000, 7), (5, 10000), (1, 299), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows(K, window, sinks, dtype):
    lens = [400, 1, 65, 200]
    print(f"window {window} sinks {sinks} {dtype}", flush=True)
    x = _inputs(window % 1000 + sinks % 1000, lens, 2, 1, 64, 64, TYPES[dtype], False)
    _check(K, x, lens, window, sinks, TYPES[dtype])


@pytest.mark.parametrize("dk,dv", [(16, 16), (128, 128), (192, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 33), (70, 4), (256, 129)])
def test_windows_of_other_heads(K, window, sinks, dk, dv):
    lens = [500, 130]
    for dtype in ("bf16", "f32"):
        print(f"window {window} sinks {sinks} {dk}/{dv} {dtype}", flush=True)
        x = _inputs(window + sinks, lens, 2, 1, dk, dv, TYPES[dtype], True)
        _check(K, x, lens, window, sinks, TYPES[dtype])


@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 3), (8, 1), (5, 5), (32, 8)])
def test_head_layouts(K, H, Hkv):
    lens = [260, 40]
    print(f"window heads {H}/{Hkv}", flush=True)
    x = _inputs(H, lens, H, Hkv, 128, 128, torch.bfloat16, H == 6)
    _check(K, x, lens, 70, 4, torch.bfloat16)


@pytest.mark.parametrize("window,sinks", [(500, 4), (96, 200), (700, 0)])
def test_longer_sequences(K, window, sinks):
    """Most tiles behind the window, a few whole ones inside it, first tokens far away."""
    lens = [3000, 300, 1700]
    print(f"window long {window} {sinks}", flush=True)
    x = _inputs(5, lens, 4, 2, 128, 128, torch.bfloat16, True)
    _check(K, x, lens, window, sinks, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(40, 3), (90, 140), (3, 131), (200, 1)])
def test_first_tokens_of_many_long_sequences(K, window, sinks, dtype):
    """Their far queries are worked on apart: sequences that begin anywhere, of
    just the lengths at which there are some, between short and empty ones."""
    reach = window + 128
    lens = [reach - 1, 0, reach, 5, reach + 1, 700, 130, reach + 33, 1, 1100, reach - 1, 257]
    print(f"first tokens {window} {sinks} {dtype}", flush=True)
    x = _inputs(window, lens, 2, 1, 32, 32, TYPES[dtype], True, spare=9)
    _check(K, x, lens, window, sinks, TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 1)])
@pytest.mark.parametrize("lens,window,sinks", [([161], 33, 162), ([129], 1, 1000), ([0, 161, 0], 33, 2 ** 31 - 1), ([161], 33, 161), ([192], 64, 193),
                                               ([225], 97, 226), ([162], 33, 162), ([160], 33, 162), ([70, 91], 33, 162)])
def test_more_first_tokens_than_tokens(K, lens, window, sinks, H, Hkv, dtype):
    """At the lengths at which first tokens begin to have far queries.  What is
    around a workspace of just the size asked for stays as it was."""
    print(f"first tokens {lens} {window} {sinks} {H}/{Hkv} {dtype}", flush=True)
    x = _inputs(window + sum(lens), lens, H, Hkv, 64, 64, TYPES[dtype], False)
    out, lse, g = _check(K, x, lens, window, sinks, TYPES[dtype])
    need = K.kda_attn_window_backward_workspace_bytes(sum(lens), len(lens), H, Hkv, 64, 64, TYPES[dtype], False, window, sinks)
    around = 1 << 20
    room = torch.full((need + 2 * around,), 0xa5, dtype=torch.uint8, device="cuda")
    got = _backward(K, x, lens, window, sinks, out, lse, workspace=room[around:around + need])
    torch.cuda.synchronize()
    assert bool((room[:around] == 0xa5).all()) and bool((room[around + need:] == 0xa5).all())
    assert all(torch.equal(got[n], g[n]) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_first_tokens_of_long_sequences_among_many_short_ones(K, dtype):
    """More sequences than could have far queries."""
    reach = 40 + 128
    short = [i % 4 for i in range(12)]
    lens = [*short, reach, *short, reach + 33, reach - 1, *short, 700, 2]
    assert len(lens) > sum(lens) // reach
    print(f"first tokens, many short {dtype}", flush=True)
    x = _inputs(23, lens, 4, 2, 32, 32, TYPES[dtype], False, spare=3)
    _check(K, x, lens, 40, 35, TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_first_tokens_where_tiles_are_not_cut(K, dtype):
    """So many key tiles that none is cut into parts; the far queries are."""
    lens = [2500, 129, 2100]
    x = _inputs(17, lens, 32, 32, 16, 16, TYPES[dtype], False)
    _check(K, x, lens, 100, 5, TYPES[dtype])


def test_many_sequences(K):
    lens = [(i * 37) % 19 for i in range(150)] + [300] + [(i * 11) % 7 for i in range(70)]
    x = _inputs(6, lens, 2, 2, 32, 32, torch.float32, False)
    _check(K, x, lens, 9, 2, torch.float32)


def test_a_window_of_everything_is_causal(K):
    lens = [333, 129]
    for dtype in (torch.float32, torch.bfloat16):
        x = _inputs(21, lens, 4, 2, 64, 64, dtype, True)
        want = K.kda_attn_prefill(x["q"], x["k"], x["v"], out_gate=x["z"], cu_seqlens=_cu(lens))
        got = _forward(K, x, lens, 333, 0)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        a = K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], *want, x["dy"], out_gate=x["z"], cu_seqlens=_cu(lens))
        b = _backward(K, x, lens, 333, 0, *got)
        # the same products; the sums over queries may be cut into other parts
        ref = R.backward(*(_64(x[t]) for t in ("q", "k", "v", "z", "dy")), lens, 0.125, dtype)
        for n in a:
            assert bool(((a[n].double() - b[n].double()).abs() <= 2 * ref[n][1]).all()), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steep_softmax(K, dtype):
    """Scores of several hundred, the largest of them outside of many windows."""
    lens = [300, 77]
    x = _inputs(7, lens, 2, 2, 64, 64, TYPES[dtype], False, size=60.0)
    x["k"][100:110] *= 4
    n = sum(lens)
    out, lse = _forward(K, x, lens, 40, 2)
    want, bo, wl, bl = R.prefill(_64(x["q"]), _64(x["k"]), _64(x["v"]), None, lens, 0.125, TYPES[dtype], R.windowed(40, 2))
    R.check("out", out[:n], want, bo)
    R.check("lse", lse[:n], wl, bl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_broken_rows_far_away(K, dtype):
    """NaN and infinity in a sequence reach what attends them and at most 190
    tokens more, other sequences not at all; nothing is read for rows that have
    left a token behind but for the first ones."""
    lens = [1500, 60]
    window, sinks = 100, 4
    x = _inputs(10, lens, 2, 1, 64, 64, TYPES[dtype], True)
    out, lse, g = _check(K, x, lens, window, sinks, TYPES[dtype])
    for bad in (20, 640):
        y = {n: t.clone() for n, t in x.items()}
        for n, t in y.items():
            t[bad] = float("inf") if n == "k" else float("nan")
        o2, l2 = _forward(K, y, lens, window, sinks)
        g2 = _backward(K, y, lens, window, sinks, o2, l2)
        torch.cuda.synchronize()
        assert bool(torch.isnan(l2[bad]).all())
        reach = range(max(0, bad - 127), bad + window + 190)
        clean = torch.tensor([r for r in range(1560) if r not in reach], device="cuda")
        assert torch.equal(out[clean], o2[clean]) and torch.equal(lse[clean], l2[clean]), bad
        # a gradient of a token: rows that are broken reach what they attend
        lost = set(range(max(0, bad - window - 2 * 127), bad + 2 * window + 2 * 127)) | set(range(128))
        clean = torch.tensor([r for r in range(1560) if r not in lost], device="cuda")
        for n in ("dk", "dv"):
            assert torch.equal(g[n][clean], g2[n][clean]), (n, bad)


def test_gradients_against_differences(K):
    """fp32 gradients against central differences of the 64-bit forward."""
    lens = [19, 5]
    x = _inputs(11, lens, 2, 1, 16, 16, torch.float32, True)
    out, lse = _forward(K, x, lens, 4, 2)
    g = _backward(K, x, lens, 4, 2, out, lse)
    d = {n: t.double() for n, t in x.items()}

    def loss(y):
        o = R.prefill(y["q"], y["k"], y["v"], y["z"], lens, 0.25, torch.float32, R.windowed(4, 2))[0]
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
    lens = [900, 130, 7]
    x = _inputs(12, lens, 8, 2, 128, 128, torch.bfloat16, True)
    one, two = _forward(K, x, lens, 200, 4), _forward(K, x, lens, 200, 4)
    a, b = _backward(K, x, lens, 200, 4, *one), _backward(K, x, lens, 200, 4, *two)
    assert all(torch.equal(u, w) for u, w in zip(one, two))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_captured_and_replayed(K):
    """Forward and backward in one graph, replayed on changing inputs with
    eager work between the replays."""
    lens = [400, 60]
    cu = _cu(lens)
    x = _inputs(13, lens, 4, 2, 64, 64, torch.bfloat16, True)
    ws = torch.empty(K.kda_attn_window_backward_workspace_bytes(460, 2, 4, 2, 64, 64, torch.bfloat16, True, 70, 4), dtype=torch.uint8,
                     device="cuda")

    def step():
        o, l = K.kda_attn_window_prefill(x["q"], x["k"], x["v"], 70, sinks=4, out_gate=x["z"], cu_seqlens=cu)
        return o, l, K.kda_attn_window_prefill_backward(x["q"], x["k"], x["v"], o, l, x["dy"], 70, sinks=4, out_gate=x["z"],
                                                        cu_seqlens=cu, workspace=ws)
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


def test_on_several_streams(K):
    lens = [300]
    xs = [_inputs(14 + i, lens, 4, 4, 128, 128, torch.bfloat16, False) for i in range(3)]
    cu = _cu(lens)
    want = [_forward(K, x, lens, 90, 1) for x in xs]
    grads = [_backward(K, x, lens, 90, 1, *w) for x, w in zip(xs, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            o = K.kda_attn_window_prefill(x["q"], x["k"], x["v"], 90, sinks=1, cu_seqlens=cu)
            got.append((o, K.kda_attn_window_prefill_backward(x["q"], x["k"], x["v"], *o, x["dy"], 90, sinks=1, cu_seqlens=cu)))
    torch.cuda.synchronize()
    for w, g, (o, b) in zip(want, grads, got):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
        assert all(torch.equal(b[n], g[n]) for n in ("dq", "dk", "dv"))


def test_binding_refuses(K):
    x = _inputs(15, [20], 4, 2, 64, 64, torch.float32, False)
    with pytest.raises(ValueError):
        K.kda_attn_window_prefill(x["q"][:, ::2], x["k"], x["v"], 8)  # not contiguous
    with pytest.raises(TypeError):
        K.kda_attn_window_prefill(x["q"], x["k"].bfloat16(), x["v"], 8)
    with pytest.raises(ValueError):
        K.kda_attn_window_prefill(x["q"], x["k"].cpu(), x["v"], 8)
    with pytest.raises(Exception, match="window=0"):
        K.kda_attn_window_prefill(x["q"], x["k"], x["v"], 0)
    with pytest.raises(Exception, match="sinks=-1"):
        K.kda_attn_window_prefill(x["q"], x["k"], x["v"], 8, sinks=-1)
    out, lse = K.kda_attn_window_prefill(x["q"], x["k"], x["v"], 8)
    with pytest.raises(Exception, match="window=-3"):
        K.kda_attn_window_prefill_backward(x["q"], x["k"], x["v"], out, lse, x["dy"], -3)


def test_empty_batch(K):
    e = lambda h, d: torch.empty((0, h, d), device="cuda")  # noqa: E731
    out, lse = K.kda_attn_window_prefill(e(2, 64), e(1, 64), e(1, 64), 5)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    g = K.kda_attn_window_prefill_backward(e(2, 64), e(1, 64), e(1, 64), out, lse, e(2, 64), 5, out_gate=e(2, 64))
    assert g["dz"].shape == (0, 2, 64)
