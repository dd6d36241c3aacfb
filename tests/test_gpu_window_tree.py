"""Drafted tokens over a paged cache with a sliding window and first tokens
that stay visible, on the GPU against plain 64-bit attention (attn_ref)."""

import math

import pytest
import torch

import attn_ref as R
from test_gpu_attn_tree import HEADS, TYPES, _make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


def _call(K, x, window, sinks, **kw):
    got = K.kda_attn_window_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"], x["lens"], window, sinks=sinks,
                                 tree_mask=x["mask"], out_gate=x["z"], slot_indices=x["rows"], **kw)
    torch.cuda.synchronize()
    return got


def _seen(x, b, window, sinks):
    """[T, cached + drafts]: what each token attends."""
    n, T = x["ctx_k"][b].shape[0], x["q"].shape[1]
    seen = torch.zeros(T, n + T, dtype=torch.bool)
    for t in range(T):
        word = (2 << t) - 1 if x["mask"] is None else int(x["mask"][b, t])
        line = list(range(n)) + [n + j for j in range(T) if word >> j & 1]
        for place, key in enumerate(line):
            seen[t, key] = place < sinks or place >= len(line) - window
    return seen.cuda()


def _check(K, x, window, sinks, dtype, scale=None, dropped=None):
    out, lse = _call(K, x, window, sinks, scale=scale)
    B, T, H, dk = x["q"].shape
    Hkv = x["k_new"].shape[2]
    G, sc = H // Hkv, scale or dk ** -0.5
    for b in range(B):
        n = x["ctx_k"][b].shape[0]
        seen = _seen(x, b, window, sinks)
        if dropped and b in dropped:
            seen[:, :n] &= ~dropped[b]
        for h in range(H):
            k = torch.cat([x["ctx_k"][b][:, h // G], x["k_new"][b, :, h // G]]).double()
            v = torch.cat([x["ctx_v"][b][:, h // G], x["v_new"][b, :, h // G]]).double()
            o, bo, l, bl, _, _ = R.softmax_rows(x["q"][b, :, h].double(), k, v, sc, seen, R.UNIT[dtype])
            if x["z"] is not None:
                g = torch.sigmoid(x["z"][b, :, h].double())
                o, bo = o * g, bo * g + o.abs() * g * 2.0 ** -20
            R.check(f"out {b},{h}", out[b, :, h], o, bo + R.UNIT[dtype] * (o.abs() + bo) + 1e-30)
            R.check(f"lse {b},{h}", lse[b, :, h], l, bl)
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_head_sizes(K, dk, dv, dtype):
    print(f"window tree {dk}/{dv} {dtype}", flush=True)
    x = _make(dk, [0, 1, 15, 16, 17, 33, 230], 7, 4, 2, dk, dv, 16, TYPES[dtype], gate=True)
    _check(K, x, 40, 3, TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (3, 0), (3, 40), (5, 203), (31, 0), (32, 32), (64, 1), (65, 33), (100, 4), (199, 16),
                                          (200, 0), (210, 5), (1 << 20, 3), (2 ** 31 - 1, 2 ** 31 - 1), (2, 1 << 20)])
def test_windows(K, window, sinks, dtype):
    """Windows of fewer tokens than a row's drafts, first tokens that are drafts."""
    print(f"window tree {window} {sinks} {dtype}", flush=True)
    x = _make(window % 97 + sinks % 97, [200, 31, 0, 3], 9, 4, 2, 64, 64, 32, TYPES[dtype], gate=True)
    _check(K, x, window, sinks, TYPES[dtype])


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("T,H,Hkv", [(1, 4, 4), (1, 8, 1), (4, 4, 2), (33, 2, 1), (64, 2, 2)])
def test_tokens_heads_pages(K, T, H, Hkv, page):
    print(f"window tree T={T} H={H}/{Hkv} page={page}", flush=True)
    for mask in ("tree", "chain"):
        x = _make(T + page, [300, 31, 0], T, H, Hkv, 64, 64, page, torch.bfloat16, mask=mask)
        _check(K, x, 50, 5, torch.bfloat16)


@pytest.mark.parametrize("T,G", [(16, 4), (64, 16)])
def test_many_rows(K, T, G):
    print(f"window tree rows T={T} G={G}", flush=True)
    for dk, dv in ((128, 128), (192, 128)):
        x = _make(T, [300, 5], T, G, 1, dk, dv, 64, torch.bfloat16)
        _check(K, x, 37, 40, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 9])
def test_split_over_a_long_window(K, T, dtype):
    print(f"window tree long T={T} {dtype}", flush=True)
    x = _make(T, [5000, 700, 1], T, 4, 2, 128, 128, 64, TYPES[dtype], gate=True, mask="chain" if T == 1 else "tree")
    for window, sinks in ((2500, 100), (600, 4), (4000, 0)):
        _check(K, x, window, sinks, TYPES[dtype])


def test_a_window_of_everything_is_the_plain_call(K):
    x = _make(4, [77, 200], 9, 4, 2, 128, 128, 32, torch.bfloat16, gate=True)
    want = K.kda_attn_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"], x["lens"], tree_mask=x["mask"],
                           out_gate=x["z"], slot_indices=x["rows"])
    for got in (_call(K, x, 10000, 0), _call(K, x, 1, 10000)):
        for a, b in zip(want, got):  # the same sums, in parts of other sizes where the context is cut
            assert float((a.double() - b.double()).abs().max()) <= 2.0 ** -7 * float(a.double().abs().max())


@pytest.mark.parametrize("width", [None, 300])
def test_rows_that_attend_nothing(K, width):
    x = _make(5, [0, 50], 6, 2, 1, 64, 64, 16, torch.bfloat16, gate=True, width=width)
    x["mask"][0, 2] = 0
    x["mask"][0, 4] = -64  # bits 6 and up only
    x["mask"][1, 3] = 0
    out, lse = _check(K, x, 10, 2, torch.bfloat16)
    assert bool((out[0, [2, 4]] == 0).all()) and bool(torch.isneginf(lse[0, [2, 4]]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_window_whose_pages_are_gone(K, dtype):
    """Every token of a row's view was in a page that is gone: 0 and -infinity;
    the row beside it, that attends a draft, is not that."""
    x = _make(6, [64, 64], 2, 2, 1, 32, 32, 16, TYPES[dtype])
    r = int(x["rows"][0])
    x["table"][r, 3] = -1
    gone = torch.zeros(64, dtype=torch.bool, device="cuda")
    gone[48:] = True
    x["mask"][0, 0], x["mask"][0, 1] = 0, 2
    out, lse = _check(K, x, 10, 0, TYPES[dtype], dropped={0: gone})
    assert bool((out[0, 0] == 0).all()) and bool(torch.isneginf(lse[0, 0]).all()) and bool(torch.isfinite(lse[0, 1]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_behind_the_window_can_go(K, dtype):
    x = _make(7, [400, 64], 4, 2, 1, 32, 32, 16, TYPES[dtype])
    want = _call(K, x, 90, 3)
    r = int(x["rows"][0])
    x["table"][r, 1:19] = -1  # the places 16 .. 303; the window begins at 310 at the least
    got = _call(K, x, 90, 3)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [20, 600])
def test_values_that_are_not_finite(K, dtype, value, width):
    """In the cache: they reach the rows whose window holds them, and no others,
    also where they share a tile with what is attended."""
    x = _make(8, [300], 40, 4, 2, 64, 64, 16, TYPES[dtype], mask="chain", width=width)
    window, sinks = 50, 5
    want, wl = _call(K, x, window, sinks)
    for place in (2, 5, 30, 249, 251, 260, 289, 299):
        y = dict(x, kc=x["kc"].clone(), vc=x["vc"].clone())
        page = int(x["table"][int(x["rows"][0]), place // 16])
        y["vc"][page, 1, place % 16, 7] = value
        if place < 200 and place >= sinks:
            y["kc"][page, 1, place % 16] = value
        out, lse = _call(K, y, window, sinks)
        assert torch.equal(lse, wl), place
        w = want.clone()
        for t in range(40):  # row t stands at place 300 + t
            if place < sinks or 300 + t - place < window:
                w[0, t, 2:, 7] = value
        same = (out == w) | (torch.isnan(out) & torch.isnan(w))
        assert bool(same.all()), place


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_broken_key_at_the_edge(K, dtype):
    """A cached key of NaN: the rows whose window holds it are NaN, the others as before."""
    x = _make(18, [300], 40, 4, 2, 64, 64, 16, TYPES[dtype], mask="chain")
    want, wl = _call(K, x, 50, 5)
    place = 270
    x["kc"][int(x["table"][int(x["rows"][0]), place // 16]), 0, place % 16, 3] = math.nan
    out, lse = _call(K, x, 50, 5)
    for t in range(40):
        hit = 300 + t - place < 50
        assert bool(torch.isnan(lse[0, t, :2]).all()) == hit and bool(torch.isnan(out[0, t, :2]).all()) == hit
        assert torch.equal(lse[0, t, 2:], wl[0, t, 2:]) and torch.equal(out[0, t, 2:], want[0, t, 2:])
        if not hit:
            assert torch.equal(out[0, t], want[0, t])


def test_padding_rows_and_slots_used_twice(K):
    x = _make(9, [60, 20, 90, 10], 3, 4, 2, 64, 64, 16, torch.float32, gate=True)
    want = _call(K, x, 15, 2)
    rows = x["rows"].clone()
    x["rows"][1], x["rows"][2] = -1, x["table"].shape[0]
    out, lse = _call(K, x, 15, 2)
    for b in (1, 2):
        assert bool((out[b] == 0).all()) and bool(torch.isneginf(lse[b]).all())
    for b in (0, 3):
        assert torch.equal(out[b], want[0][b]) and torch.equal(lse[b], want[1][b])
    x["rows"] = rows[[0, 0, 3, 3]].contiguous()
    for n in ("q", "k_new", "v_new", "z", "mask"):
        x[n] = x[n][[0, 0, 3, 3]].contiguous()
    out, lse = _call(K, x, 15, 2)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], want[0][0]) and torch.equal(out[3], want[0][3])


def test_captured_and_replayed(K):
    """One graph over a decode step whose lengths and tables change."""
    x = _make(11, [900, 300, 20], 4, 8, 2, 128, 128, 64, torch.bfloat16, width=40)
    lens = x["lens"].clone()
    ws = torch.empty(max(256, K.kda_attn_window_tree_workspace_bytes(3, 4, 8, 2, 128, 128, torch.bfloat16, 40 * 64, 400, 4)),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _call(K, x, 400, 4, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = K.kda_attn_window_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"], x["lens"], 400, sinks=4,
                                          tree_mask=x["mask"], slot_indices=x["rows"], workspace=ws)
    for i in range(4):
        x["lens"].copy_((lens - 5 * i).clamp(min=0))
        x["q"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        want = _call(K, x, 400, 4)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


def test_binding_refuses(K):
    x = _make(12, [20], 2, 2, 1, 64, 64, 16, torch.float32)
    args = (x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"], x["lens"])
    with pytest.raises(Exception, match="window=0"):
        K.kda_attn_window_tree(*args, 0, slot_indices=x["rows"])
    with pytest.raises(Exception, match="sinks=-2"):
        K.kda_attn_window_tree(*args, 3, sinks=-2, slot_indices=x["rows"])
    with pytest.raises(TypeError):
        K.kda_attn_window_tree(*args[:5], x["table"].long(), x["lens"], 3)


def test_empty_batches(K):
    x = _make(13, [20], 2, 2, 1, 64, 64, 16, torch.float32)
    out, lse = K.kda_attn_window_tree(x["q"][:0], x["k_new"][:0], x["v_new"][:0], x["kc"], x["vc"], x["table"], x["lens"], 4,
                                      slot_indices=x["rows"][:0])
    assert out.shape == (0, 2, 2, 64)
    out, lse = K.kda_attn_window_tree(x["q"][:, :0], x["k_new"][:, :0], x["v_new"][:, :0], x["kc"], x["vc"], x["table"], x["lens"], 4,
                                      slot_indices=x["rows"])
    assert out.shape == (1, 0, 2, 64)
