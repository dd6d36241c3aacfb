"""The attention weights that cached tokens gather, on the GPU against their sum
in 64 bits.

A weight e^(s - lse) of fp32 operations is off by (4 sqrt(dk) + 8) 2^-24 sum |q k|
scale (the score), |lse| 2^-23 (its product with log2 e and the difference) and
2^-20 (the exponential), relative to itself; a sum of n weights by n 2^-24 more, and
the addition to what was there by 2^-24 of the result."""

import math
import random

import pytest
import torch

import attn_ref as R
from test_gpu_attn_tree import TYPES, _make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


def _setup(seed, lens, counts, H, Hkv, dk, page, dtype, pick=False, spare=0, window=0, sinks=0, width=None):
    """A cache, each sequence's last queries with the lse of what they attend,
    weights gathered before; `pick`: the queries stand in rows of a larger
    tensor; `spare`: query rows behind the last sequence's."""
    dv = 128 if dk == 192 else dk
    x = _make(seed, lens, 1, H, Hkv, dk, dv, page, dtype, width=width)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    total, G = sum(counts), H // Hkv
    src = 2 * total + 3 if pick else total + spare
    rows = random.Random(seed).sample(range(src), total) if pick else list(range(total))
    q = torch.randn((src, H, dk), generator=g, device="cuda").to(dtype)
    lse = torch.full((src, H), math.nan, device="cuda")
    at = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        for i in range(c):
            p, row = n - c + i, rows[at]
            at += 1
            if p < 0:
                lse[row] = 1.0
                continue
            j = torch.arange(n, device="cuda")
            seen = (j <= p) & ((p - j < (window or n + 1)) | (j < sinks))
            for h in range(H):
                s = (x["ctx_k"][b][:, h // G].double() @ q[row, h].double()) * dk ** -0.5
                lse[row, h] = torch.logsumexp(torch.where(seen, s, -math.inf), 0).float()
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    slots, width = x["table"].shape
    x.update(q=q, lse=lse, counts=counts, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), lens_of=lens, scale=None,
             pick=torch.tensor(rows, dtype=torch.int32, device="cuda") if pick or spare else None, pick_list=rows,
             weights=torch.rand((slots, width * page), generator=g, device="cuda"))
    return x


def _call(K, x, window=0, sinks=0, **kw):
    w = x["weights"].clone()
    K.kda_cache_weigh(x["q"], x["lse"], x["kc"], x["table"], x["lens"], w, cu_seqlens=x["cu"], rows=x["pick"], slot_indices=x["rows"],
                      window=window, sinks=sinks, scale=x["scale"], **kw)
    torch.cuda.synchronize()
    return w


def _want(x, window, sinks, dropped=None):
    """(weights, bound) in 64 bits."""
    want, bound = x["weights"].double(), torch.zeros_like(x["weights"], dtype=torch.float64)
    H, dk = x["q"].shape[1:]
    G, sc, at = H // x["kc"].shape[1], x["scale"] or dk ** -0.5, 0
    for b, c in enumerate(x["counts"]):
        n, slot = x["lens_of"][b], int(x["rows"][b])
        rows = x["pick_list"][at:at + c]
        at += c
        if not 0 <= slot < x["table"].shape[0] or c == 0 or n == 0:
            continue
        p = torch.arange(n - c, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        seen = (j <= p) & ((p - j < (window or n + c + 1)) | (j < sinks)) & (p >= 0)
        if dropped and b in dropped:
            seen &= ~dropped[b]
        sum_w, sum_b = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
        terms = 0
        for h in range(H):
            q, k = x["q"][rows, h].double(), x["ctx_k"][b][:, h // G].double()
            lse = x["lse"][rows, h].double()[:, None]
            on = seen & torch.isfinite(lse)
            s = (q @ k.T) * sc
            w = torch.where(on, torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0)), 0.0)
            size = (q.abs() @ k.abs().T) * sc
            eps = (4 * math.sqrt(dk) + 8) * R.F * size + torch.where(torch.isfinite(lse), lse.abs(), 0.0) * 2.0 ** -23 + 2.0 ** -20
            sum_w += w.sum(0)
            sum_b += torch.where(on, w * eps, 0.0).sum(0)
            terms = terms + on.sum(0)
        want[slot, :n] += sum_w
        bound[slot, :n] += torch.where(terms > 0, 1.1 * (sum_b + (terms + 8) * R.F * sum_w) + 2 * R.F * want[slot, :n].abs(), 0.0)
    return want, bound


def _check(K, x, window=0, sinks=0, dropped=None):
    got = _call(K, x, window, sinks)
    want, bound = _want(x, window, sinks, dropped)
    kept = bound == 0
    assert torch.equal(got[kept], x["weights"][kept]), "a token that no query attends was changed"
    R.check("weights", got[~kept], want[~kept], bound[~kept])
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk", [16, 32, 64, 128, 192])
def test_head_sizes(K, dk, dtype):
    print(f"weigh {dk} {dtype}", flush=True)
    x = _setup(dk, [1, 15, 16, 17, 33, 230], [1, 15, 2, 5, 33, 40], 4, 2, dk, 16, TYPES[dtype], pick=True)
    _check(K, x)


@pytest.mark.parametrize("page", [16, 32, 64, 1024])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 1), (6, 3), (32, 8), (1, 1), (48, 1)])
def test_heads_and_pages(K, H, Hkv, page):
    print(f"weigh {H}/{Hkv} page {page}", flush=True)
    for counts in ([1, 1, 1], [3, 0, 31], [70, 1, 7]):
        x = _setup(H + page, [200, 5, 63], counts, H, Hkv, 64, page, torch.bfloat16)
        _check(K, x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,counts", [([700], [700]), ([1000], [129]), ([600, 90, 400], [600, 90, 1]), ([2500], [1]), ([2500, 3], [8, 3])])
def test_prompts_and_steps(K, lens, counts, dtype):
    """All of a prompt, its last tokens, a step: every way in which the work is cut."""
    print(f"weigh {lens} {counts} {dtype}", flush=True)
    _check(K, _setup(sum(counts), lens, counts, 8, 2, 128, 64, TYPES[dtype]))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (31, 1), (64, 33), (100, 4), (130, 200), (500, 0), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
def test_windows(K, window, sinks):
    print(f"weigh window {window} sinks {sinks}", flush=True)
    for counts in ([1, 1, 1], [40, 3, 64]):
        x = _setup(window % 91, [300, 20, 150], counts, 4, 2, 64, 32, torch.bfloat16, window=window, sinks=sinks)
        _check(K, x, window, sinks)
    x = _setup(window % 91, [700], [700], 4, 2, 64, 32, torch.float32, window=window, sinks=sinks)
    _check(K, x, window, sinks)


def test_wide_table(K):
    """Room for far more than is there."""
    _check(K, _setup(3, [40, 0, 300], [2, 0, 4], 4, 1, 64, 64, torch.bfloat16, width=500))


def test_weights_of_a_row_add_up_to_one(K):
    x = _setup(31, [900, 41], [1, 1], 8, 2, 64, 64, torch.float32)
    x["weights"].zero_()
    w = _call(K, x)
    # 8 heads of weights whose sum is 1: each within what is derived above, (900 + 8) 2^-24 and 2^-18 for the scores
    for b in range(2):
        assert abs(float(w[int(x["rows"][b])].double().sum()) - 8) <= 8 * (2.0 ** -18 + 908 * R.F)


def test_what_is_skipped(K):
    """Slots and rows that are not there, more queries than tokens, rows that
    attended nothing or are broken, tokens behind the last sequence."""
    x = _setup(5, [60, 20, 90, 10, 8], [3, 2, 4, 12, 1], 4, 2, 64, 16, torch.float32, pick=True)
    x["rows"][1], x["rows"][4] = -1, x["table"].shape[0]
    x["lse"][x["pick_list"][0], 1] = -math.inf
    x["lse"][x["pick_list"][1], 2] = math.nan
    x["lse"][x["pick_list"][6], 0] = math.inf
    _check(K, x)
    # rows outside the source: as if their lse were not finite
    y = dict(x, lse=x["lse"].clone())
    y["lse"][x["pick_list"][2]] = math.nan
    want = _call(K, y)
    for bad in (-1, x["q"].shape[0]):
        y = dict(x, pick=x["pick"].clone())
        y["pick"][2] = bad
        assert torch.equal(_call(K, y), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[3, 2], [90, 33]])
def test_broken_rows_and_keys(K, counts, dtype):
    """A query that is not finite has an lse that is not: it weighs nothing and
    the rows beside it are as before.  A key that is not finite gathers nothing."""
    x = _setup(41, [200, 64], counts, 4, 2, 64, 16, TYPES[dtype])
    want, g = _call(K, x), x["pick_list"]
    y = dict(x, q=x["q"].clone(), lse=x["lse"].clone())
    y["lse"][g[1], 2] = math.nan
    clean = _call(K, y)
    for value in (math.nan, math.inf, -math.inf):
        y["q"][g[1], 2, 5] = value
        assert torch.equal(_call(K, y), clean), value
    assert not torch.equal(clean, want)
    # every row of the heads over a broken key attends it: none of them weighs anything
    z = dict(x, kc=x["kc"].clone(), lse=x["lse"].clone())
    page, n = int(x["table"][int(x["rows"][0]), 2]), counts[0]
    z["kc"][page, 1, 3, 7] = math.nan
    z["lse"][g[:n], 2:] = math.nan
    got = _call(K, z)
    y = dict(x, lse=z["lse"])
    want, bound = _want(y, 0, 0)
    slot, place = int(x["rows"][0]), 35
    assert float((got[slot, place].double() - want[slot, place]).abs()) <= float(bound[slot, place])
    R.check("weights", got, want, bound + 1e-30)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[3, 2], [33, 70]])
def test_rows_that_no_query_names(K, counts, dtype):
    """What a source holds beside the queries (rows that no attention call wrote)
    is nothing to them, nor to a row of the list that is not there."""
    x = _setup(57, [200, 90], counts, 4, 2, 64, 16, TYPES[dtype], pick=True)
    x["lse"][x["pick_list"][1]] = math.nan
    rest = [r for r in range(x["q"].shape[0]) if r not in x["pick_list"]]
    assert rest[0] < 3
    order = [rest[0]] + [r for r in range(x["q"].shape[0]) if r != rest[0]]  # such a row is the first one
    x["pick_list"] = [order.index(r) for r in x["pick_list"]]
    x.update(q=x["q"][order].contiguous(), lse=x["lse"][order].contiguous(),
             pick=torch.tensor(x["pick_list"], dtype=torch.int32, device="cuda"))
    want = _check(K, x)
    rest = [r for r in range(x["q"].shape[0]) if r not in x["pick_list"]]
    assert rest[0] == 0
    for value in (math.nan, math.inf, 1e30):
        y = dict(x, q=x["q"].clone(), lse=x["lse"].clone())
        y["q"][rest], y["lse"][rest] = value, 0.0
        assert torch.equal(_call(K, y), want), value
        for bad in (-1, x["q"].shape[0]):
            y["pick"] = x["pick"].clone()
            y["pick"][1] = bad
            assert torch.equal(_call(K, y), want), (value, bad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_broken_head_of_a_key(K, dtype):
    """A key that is not finite in one head still gathers what the other heads'
    queries give, also where one workgroup takes all heads of a tile."""
    x = _setup(43, [600] + [0] * 299, [160] + [0] * 299, 128, 2, 16, 16, TYPES[dtype])
    slot, place, page = int(x["rows"][0]), 35, 16
    x["kc"][int(x["table"][slot, place // page]), 1, place % page, 7] = math.nan
    x["lse"][x["pick_list"], 64:] = math.nan
    want, bound = _want(x, 0, 0)
    got = _call(K, x)
    assert float(want[slot, place] - x["weights"][slot, place]) > 8 * float(bound[slot, place])
    R.check("weights", got, want, bound + 1e-30)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[1, 2], [90, 33]])
def test_broken_key_that_no_lse_knows_of(K, counts, dtype):
    """Weighed without the window that their lse is of, queries meet a key that is
    not finite: it gathers nothing of that head, and all that the others give."""
    x = _setup(47, [300, 64], counts, 8, 2, 64, 16, TYPES[dtype], window=40)
    slot, place, page = int(x["rows"][0]), 35, 16
    at = int(x["table"][slot, place // page]), 1, place % page, 7
    want, bound = _want(x, 0, 0)
    y = dict(x, lse=x["lse"].clone())
    y["lse"][:, 4:] = math.nan
    others, near = _want(y, 0, 0)
    want[slot, place], bound[slot, place] = others[slot, place], near[slot, place]
    assert float(others[slot, place] - x["weights"][slot, place]) > 8 * float(near[slot, place])
    for value in (math.nan, math.inf, -math.inf):
        y = dict(x, kc=x["kc"].clone())
        y["kc"][at] = value
        R.check(f"weights {value}", _call(K, y), want, bound + 1e-30)


def test_lengths_past_the_table(K):
    x = _setup(6, [64, 32], [2, 3], 2, 2, 64, 16, torch.float32, width=4)
    want = _call(K, x)
    x["lens"][int(x["rows"][0])] = 2 ** 31 - 1
    assert torch.equal(_call(K, x), want)
    x["lens"][int(x["rows"][1])] = -5
    got = _call(K, x)
    r = int(x["rows"][1])
    assert torch.equal(got[r], x["weights"][r])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_entries_that_name_no_page_and_stale_rows(K, dtype):
    """(Unused memory of the pools holds NaN.)"""
    for counts in ([4, 2], [130, 64]):
        x = _setup(7, [200, 64], counts, 2, 1, 32, 16, TYPES[dtype])
        r = int(x["rows"][0])
        x["table"][r, 3], x["table"][r, 6] = -1, x["kc"].shape[0]
        gone = torch.zeros(200, dtype=torch.bool, device="cuda")
        gone[48:64] = True
        gone[96:112] = True
        _check(K, x, dropped={0: gone})


def test_far_scores(K):
    """Scores of thousands: a weight is as right as its lse."""
    x = _setup(8, [300, 40], [5, 40], 4, 2, 64, 16, torch.float32)
    y = dict(x, q=x["q"] * 300)
    at = 0
    for b, (n, c) in enumerate(zip(x["lens_of"], x["counts"])):
        for i in range(c):
            for h in range(4):
                s = (x["ctx_k"][b][:n - c + i + 1, h // 2].double() @ y["q"][at, h].double()) / 8
                y["lse"][at, h] = torch.logsumexp(s, 0).float()
            at += 1
    _check(K, y)


def test_slots_without_indices_and_one_sequence(K):
    x = _setup(9, [50], [6], 4, 2, 64, 16, torch.float32)
    want = _call(K, x)
    table = x["table"][x["rows"].long()].contiguous()
    w = x["weights"][x["rows"].long()].clone()
    K.kda_cache_weigh(x["q"], x["lse"], x["kc"], table, x["lens"][x["rows"].long()].contiguous(), w)
    assert torch.equal(w, want[x["rows"].long()])


def test_same_bits_twice_and_streams(K):
    xs = [_setup(10 + i, [900, 77], [c, 5], 8, 2, 128, 64, torch.bfloat16) for i, c in enumerate((1, 40, 900))]
    want = [_call(K, x) for x in xs]
    assert all(torch.equal(_call(K, x), w) for x, w in zip(xs, want))
    streams, got = [torch.cuda.Stream() for _ in xs], [x["weights"].clone() for x in xs]
    torch.cuda.synchronize()
    for s, x, w in zip(streams, xs, got):
        with torch.cuda.stream(s):
            K.kda_cache_weigh(x["q"], x["lse"], x["kc"], x["table"], x["lens"], w, cu_seqlens=x["cu"], slot_indices=x["rows"])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("count", [2, 150])
def test_captured_and_replayed(K, count):
    x = _setup(13, [700, 300], [count, 1], 8, 2, 64, 64, torch.bfloat16)
    lens = x["lens"].clone()
    ws = torch.empty(max(256, K.kda_cache_weigh_workspace_bytes(count + 1, 2, 8, 2)), dtype=torch.uint8, device="cuda")
    w = x["weights"].clone()

    def step(to):
        K.kda_cache_weigh(x["q"], x["lse"], x["kc"], x["table"], x["lens"], to, cu_seqlens=x["cu"], slot_indices=x["rows"], workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(w)
    for i in range(4):
        x["lens"].copy_((lens - 7 * i).clamp(min=0))
        x["q"].normal_()
        before = w.clone()
        graph.replay()
        torch.cuda.synchronize()
        step(before)
        torch.cuda.synchronize()
        assert torch.equal(before, w), i


def test_binding_refuses(K):
    x = _setup(14, [20], [2], 4, 2, 64, 16, torch.float32)
    good = [x["q"], x["lse"], x["kc"], x["table"], x["lens"], x["weights"]]
    for i, bad in ((1, x["lse"][:, :2]), (1, x["lse"].double()), (2, x["kc"].bfloat16()), (3, x["table"].long()), (4, x["lens"][:-1]),
                   (5, x["weights"][:, :-1]), (5, x["weights"].cpu())):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError)):
            K.kda_cache_weigh(*args, slot_indices=x["rows"])
    with pytest.raises(Exception, match="window=-1"):
        K.kda_cache_weigh(*good, slot_indices=x["rows"], window=-1)
    K.kda_cache_weigh(x["q"][:0], x["lse"][:0], *good[2:], slot_indices=x["rows"])
