"""Slots cut down to their heaviest tokens, on the GPU against a plain model
that takes the entries one after another, and the bounded operators together as
a server uses them."""

import math
import random

import numpy as np
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


def _cache(seed, lens, page, Hkv=2, dk=16, dv=16, dtype=torch.float32, spare=2, width=None, kind="random"):
    """A cache of slots of these lengths; weights of some kind."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    need = [-(-n // page) for n in lens]
    width, pages = width or max(max(need), 1) + 1, sum(need) + 3
    slots = len(lens) + spare
    order = r.sample(range(pages), pages)
    table, length = np.full((slots, width), -1, np.int32), np.zeros(slots, np.int32)
    refs, at, slot = np.zeros(pages, np.int32), 0, r.sample(range(slots), len(lens))
    for s, n, k in zip(slot, lens, need):
        for j in range(k):
            table[s, j] = order[at]
            refs[order[at]] += 1
            at += 1
        length[s] = n
    w = torch.rand((slots, width * page), generator=g, device="cuda")
    if kind == "few values":
        w = (w * 4).floor()
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "odd":
        w = w - 0.5
        pick = torch.rand(w.shape, generator=g, device="cuda")
        for i, v in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42, -1e-42, -math.nan)):
            w[(pick > 0.06 * i) & (pick < 0.06 * (i + 1))] = v
    elif kind == "wide":
        w = torch.exp(60 * (w - 0.5))
    new = lambda d: torch.randn((pages, Hkv, page, d), generator=g, device="cuda").to(dtype)  # noqa: E731
    to = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return dict(page=page, slot=slot, kc=new(dk), vc=new(dv), table=to(table), lens=to(length), refs=to(refs), weights=w)


def _model(x, entries, keep, first, recent):
    """What a call leaves: the cache's arrays on the host, kept, status."""
    page = x["page"]
    kc, vc, w = x["kc"].float().cpu().numpy(), x["vc"].float().cpu().numpy(), x["weights"].cpu().numpy().copy()
    table, lens, refs = (x[n].cpu().numpy().copy() for n in ("table", "lens", "refs"))
    kc, vc = kc.copy(), vc.copy()
    refs0 = refs.copy()  # counts as the call found them
    kept, status = np.full((len(entries), keep), -1, np.int32), np.zeros(len(entries), np.int32)
    for i, s in enumerate(entries):
        if not 0 <= s < len(lens) or s in entries[:i]:
            status[i] = 2
            continue
        n = min(max(int(lens[s]), 0), table.shape[1] * page)
        if n <= keep:
            kept[i, :n] = np.arange(n)
            continue
        if any(not 0 <= table[s, j] < len(refs) for j in range(-(-n // page))):
            status[i] = 2
            continue
        middle = list(range(first, n - recent))
        key = {p: -math.inf if math.isnan(w[s, p]) else float(w[s, p]) + 0.0 for p in middle}
        middle.sort(key=lambda p: (bool(np.isnan(w[s, p])), -key[p], p))
        stay = sorted(list(range(first)) + list(range(n - recent, n)) + middle[:keep - first - recent])
        moved = [d for d, p in enumerate(stay) if d != p]
        start = moved[0] if moved else keep
        if any(refs0[table[s, j]] > 1 for j in range(start // page, -(-keep // page))):
            status[i] = 2
            continue
        kept[i] = stay
        for pool in (kc, vc):
            rows = [pool[table[s, p // page], :, p % page].copy() for p in stay]
            for d, row in enumerate(rows):
                pool[table[s, d // page], :, d % page] = row
        w[s, :n] = np.concatenate([w[s, stay], np.zeros(n - keep, np.float32)])
        for j in range(-(-keep // page), table.shape[1]):
            if 0 <= table[s, j] < len(refs):
                refs[table[s, j]] -= 1
            table[s, j] = -1
        lens[s] = keep
    return dict(kc=kc, vc=vc, weights=w, table=table, lens=lens, refs=refs, kept=kept, status=status)


def _check(K, x, entries, keep, first=0, recent=0, **kw):
    want = _model(x, entries, keep, first, recent)
    kept, status = K.kda_cache_evict(torch.tensor(entries, dtype=torch.int32, device="cuda"), keep, x["kc"], x["vc"], x["table"],
                                     x["lens"], x["refs"], x["weights"], first=first, recent=recent, **kw)
    torch.cuda.synchronize()
    got = dict(x, kept=kept, status=status)
    for name in ("status", "kept", "lens", "table", "refs", "weights", "kc", "vc"):
        a = got[name].float().cpu().numpy() if name in ("kc", "vc") else got[name].cpu().numpy()
        assert np.array_equal(a, want[name], equal_nan=a.dtype.kind == "f"), name
    return status.tolist()


@pytest.mark.parametrize("kind", ["random", "few values", "equal", "odd", "wide"])
@pytest.mark.parametrize("keep,first,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (16, 4, 4), (17, 0, 5), (31, 31, 0), (32, 0, 32), (50, 4, 9),
                                               (63, 20, 43), (64, 1, 0), (100, 3, 30), (199, 4, 10)])
def test_budgets(K, keep, first, recent, kind):
    print(f"evict {keep} {first} {recent} {kind}", flush=True)
    x = _cache(keep, [200, 64, 1, 0, 65, 33], 16, kind=kind)
    assert set(_check(K, x, list(x["slot"]), keep, first, recent)) == {0}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 32), (64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_heads(K, Hkv, dk, dv, dtype):
    print(f"evict heads {Hkv} {dk}/{dv} {dtype}", flush=True)
    x = _cache(dk, [300, 130], 32, Hkv, dk, dv, TYPES[dtype])
    _check(K, x, list(x["slot"]), 90, 4, 20)


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("n,keep", [(5000, 1200), (5000, 4999), (3000, 7), (2049, 1025)])
def test_longer_slots(K, n, keep, page):
    """More tokens than a workgroup takes at once, moved over many steps."""
    print(f"evict {n} to {keep} page {page}", flush=True)
    x = _cache(n + keep, [n, 100, n - 1], page, kind="random")
    _check(K, x, list(x["slot"]), keep, min(4, keep), min(keep - min(4, keep), 100))


@pytest.mark.parametrize("kind", ["random", "few values", "odd"])
@pytest.mark.parametrize("lens,keep,first,recent", [([8192, 8193, 100], 100, 4, 7), ([20000, 16385], 16384, 0, 0), ([25000], 9000, 8200, 500),
                                                    ([16390, 8200], 8192, 3, 8189), ([40000], 1, 0, 0)])
def test_slots_of_several_steps(K, lens, keep, first, recent, kind):
    """More tokens than a planning workgroup holds at once."""
    print(f"evict steps {lens} {keep} {kind}", flush=True)
    x = _cache(len(lens) + keep, lens, 64, Hkv=1, kind=kind)
    assert _check(K, x, x["slot"], keep, first, recent) == [0] * len(lens)


@pytest.mark.parametrize("n", [50, 20000])
def test_weights_that_begin_anywhere(K, n):
    x = _cache(n, [n, 33], 16, kind="few values")
    flat = torch.empty(x["weights"].numel() + 1, device="cuda")[1:]
    flat.copy_(x["weights"].flatten())
    x["weights"] = flat.view(x["weights"].shape)
    assert x["weights"].data_ptr() % 16 == 4
    assert _check(K, x, x["slot"], 29, 2, 3) == [0, 0]


def test_as_many_heads_as_there_can_be(K):
    x = _cache(77, [40], 16, Hkv=(1 << 15) - 1, dtype=torch.bfloat16, spare=0)
    print("evict 32767 heads", flush=True)
    assert _check(K, x, x["slot"], 17, 1, 2) == [0]


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_ordered_weights(K, order):
    """Only the last stay (every row moves as far as it can), or only the first
    (none moves, the last page stays partly filled)."""
    for keep in (33, 64):
        x = _cache(3, [400, 90], 16)
        t = torch.arange(x["weights"].shape[1], device="cuda").float()
        x["weights"][:] = t if order == "rising" else -t
        _check(K, x, list(x["slot"]), keep)


def test_again_and_again(K):
    """Cut, filled up and cut: as a server does."""
    x = _cache(4, [150, 90, 120], 16, width=12)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    slots = torch.tensor(x["slot"], dtype=torch.int32, device="cuda")
    for step in range(4):
        _check(K, x, list(x["slot"]), 60, 4, 16)
        new = x["lens"][slots.long()] + 40
        status = K.kda_cache_reserve(slots, new, 16, x["table"], x["lens"], x["refs"])
        assert status.tolist() == [0, 0, 0]
        rows = torch.randn((120, 2, 16), generator=g, device="cuda")
        K.kda_cache_append(rows, rows.clone(), x["kc"], x["vc"], x["table"], x["lens"],
                           torch.tensor([0, 40, 80, 120], dtype=torch.int32, device="cuda"), slot_indices=slots)
        x["lens"][slots.long()] = new
        x["weights"][slots.long()] += torch.rand(x["weights"][slots.long()].shape, generator=g, device="cuda") * (
            torch.arange(x["weights"].shape[1], device="cuda") < new[:, None])


def test_refused_entries(K):
    x = _cache(6, [100, 100, 100, 20], 16)
    a, b, c, d = x["slot"]
    x["table"][b, 2] = -1
    x["table"][c, 4] = x["refs"].numel()
    free = [s for s in range(x["table"].shape[0]) if s not in x["slot"]][0]
    assert _check(K, x, [a, b, -1, c, a, x["table"].shape[0], d, free, d], 40, 2, 5) == [0, 2, 2, 2, 2, 2, 0, 0, 2]


def test_shared_pages(K):
    """A slot whose rows to write are another's too is refused; what the first
    tokens fill stays shared, and so do pages that only leave."""
    x = _cache(7, [100, 1], 16, spare=3)
    a = x["slot"][0]
    b, c = [s for s in range(x["table"].shape[0]) if s not in x["slot"]][:2]
    K.kda_cache_fork(torch.tensor([a, a], dtype=torch.int32, device="cuda"), torch.tensor([b, c], dtype=torch.int32, device="cuda"),
                     x["kc"], x["vc"], x["table"], x["lens"], x["refs"])
    x["weights"][[b, c]] = torch.rand((2, x["weights"].shape[1]), device="cuda")
    assert _check(K, x, [a, b], 40, 0, 5) == [2, 2]
    # the pages that are written belong to one slot: give slot b its own ones
    for j in range(2, 6):
        page = int((x["refs"] == 0).nonzero()[0, 0]) if bool((x["refs"] == 0).any()) else None
        if page is None:
            break
        x["refs"][int(x["table"][b, j])] -= 1
        x["table"][b, j] = page
        x["refs"][page] = 1
    assert _check(K, x, [b, c, a], 40, 32, 4)[0] == 0
    # whole pages that only leave may be shared; a last one that stays partly filled may not
    t = torch.arange(x["weights"].shape[1], device="cuda").float()
    x["weights"][:] = -t
    assert _check(K, x, [a, c], 32) == [0, 0]
    assert _check(K, x, [a], 20) == [2]
    assert _check(K, x, [a, c], 16) == [0, 0]


def test_lengths_past_the_table(K):
    x = _cache(8, [64, 32], 16, width=4)
    x["lens"][x["slot"][0]] = 2 ** 31 - 1
    x["lens"][x["slot"][1]] = -7
    _check(K, x, list(x["slot"]), 20, 2, 3)


def test_offsets_past_32_bits(K):
    """Pools of more than 2^32 bytes, the pages in use at their end."""
    Hkv, page, d = 8, 64, 128
    pages = (1 << 32) // (Hkv * page * d * 2) + 9
    small = _cache(9, [300], page, Hkv, d, d, torch.bfloat16, spare=0)
    kc = torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    table, refs = small["table"].clone(), torch.zeros(pages, dtype=torch.int32, device="cuda")
    for j in range(5):
        p, q = int(table[0, j]), pages - 1 - j
        kc[q], vc[q] = small["kc"][p], small["vc"][p]
        table[0, j] = q
        refs[q] = 1
    w = small["weights"].clone()
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = small["lens"].clone()
    kept, status = K.kda_cache_evict(one, 130, kc, vc, table, lens, refs, w, first=4, recent=20)
    want, ws = K.kda_cache_evict(one, 130, small["kc"], small["vc"], small["table"], small["lens"], small["refs"], small["weights"],
                                 first=4, recent=20)
    assert torch.equal(kept, want) and status.tolist() == ws.tolist() == [0] and torch.equal(w, small["weights"])
    for j in range(3):
        p = int(small["table"][0, j])
        rows = min(page, 130 - j * page)
        assert torch.equal(kc[pages - 1 - j][:, :rows], small["kc"][p][:, :rows])
        assert torch.equal(vc[pages - 1 - j][:, :rows], small["vc"][p][:, :rows])


def test_captured_and_replayed(K):
    x = _cache(10, [300, 200, 40], 16, width=24)
    names = ("kc", "vc", "table", "lens", "refs", "weights")
    start = {n: x[n].clone() for n in names}
    slots = torch.tensor(x["slot"], dtype=torch.int32, device="cuda")
    ws = torch.empty(K.kda_cache_evict_workspace_bytes(3, 90), dtype=torch.uint8, device="cuda")

    def step(y):
        return K.kda_cache_evict(slots, 90, y["kc"], y["vc"], y["table"], y["lens"], y["refs"], y["weights"], first=3, recent=10,
                                 workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, status = step(x)
    for i in range(4):
        start["weights"].uniform_()
        for n in names:
            x[n].copy_(start[n])
        graph.replay()
        torch.cuda.synchronize()
        y = {n: start[n].clone() for n in names}
        a, b = step(y)
        torch.cuda.synchronize()
        assert torch.equal(kept, a) and torch.equal(status, b)
        assert all(torch.equal(x[n], y[n]) for n in names), i


def test_outputs_that_are_not_wanted(K):
    """kept and status may be NULL."""
    import ctypes
    from gated_delta_rule_64_amd import _lib
    x, P = _cache(11, [100, 50], 16), lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    want = _model(x, list(x["slot"]), 30, 2, 3)
    slots = torch.tensor(x["slot"], dtype=torch.int32, device="cuda")
    ws = torch.empty(K.kda_cache_evict_workspace_bytes(2, 30), dtype=torch.uint8, device="cuda")
    S, W = x["table"].shape
    st = _lib.lib().kda_cache_evict(2, P(slots), 30, 2, 3, 2, 16, 16, 0, P(x["kc"]), P(x["vc"]), x["kc"].shape[0], 16, P(x["table"]), S, W,
                                    P(x["lens"]), P(x["refs"]), P(x["weights"]), None, None, P(ws), ws.numel(),
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and np.array_equal(x["kc"].cpu().numpy(), want["kc"]) and np.array_equal(x["lens"].cpu().numpy(), want["lens"])


def test_nothing_to_do(K):
    x = _cache(12, [40], 16)
    before = {n: x[n].clone() for n in ("kc", "vc", "table", "lens", "refs", "weights")}
    kept, status = K.kda_cache_evict(torch.zeros(0, dtype=torch.int32, device="cuda"), 8, x["kc"], x["vc"], x["table"], x["lens"],
                                     x["refs"], x["weights"])
    assert kept.shape == (0, 8) and status.shape == (0,)
    assert _check(K, x, list(x["slot"]), 40) == [0]
    assert all(torch.equal(before[n], x[n]) for n in before)


def test_binding_refuses(K):
    x = _cache(13, [40], 16)
    s = torch.tensor(x["slot"], dtype=torch.int32, device="cuda")
    args = (x["kc"], x["vc"], x["table"], x["lens"], x["refs"])
    with pytest.raises(Exception, match="keep=0"):
        K.kda_cache_evict(s, 0, *args, x["weights"])
    with pytest.raises(Exception, match="more than keep"):
        K.kda_cache_evict(s, 8, *args, x["weights"], first=5, recent=4)
    with pytest.raises(ValueError):
        K.kda_cache_evict(s, 8, *args, x["weights"][:, :-1])
    with pytest.raises(TypeError):
        K.kda_cache_evict(s.long(), 8, *args, x["weights"])
    with pytest.raises(ValueError):
        K.kda_cache_evict(s, 8, *args, x["weights"], kept=torch.empty((1, 9), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_server_with_a_bounded_cache(K, dtype):
    """Prompts through the windowed prefill and its cache, a draft tree, its
    accepted path committed, weighed, the slots cut, and on: every result
    against 64-bit attention over what the model says the cache holds."""
    dt, H, Hkv, d, page, window, sinks = TYPES[dtype], 4, 2, 64, 16, 60, 4
    G, keep, first, recent, u = H // Hkv, 48, 4, 16, R.UNIT[TYPES[dtype]]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, slots = [150, 33, 90], ints([2, 0, 3])
    pages, width = 40, 12
    kc, vc = new(pages, Hkv, page, d), new(pages, Hkv, page, d)
    table = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
    length, refs = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    weights = torch.zeros((4, width * page), device="cuda")
    cu = ints([0, 150, 183, 273])
    q, k, v = new(273, H, d), new(273, Hkv, d), new(273, Hkv, d)
    out, lse = K.kda_attn_window_prefill(q, k, v, window, sinks=sinks, cu_seqlens=cu)
    assert K.kda_cache_reserve(slots, ints(lens), page, table, length, refs).tolist() == [0, 0, 0]
    K.kda_cache_append(k, v, kc, vc, table, length, cu, slot_indices=slots)
    length[slots.long()] = ints(lens)
    K.kda_cache_weigh(q, lse, kc, table, length, weights, cu_seqlens=cu, slot_indices=slots, window=window, sinks=sinks)
    # each row's weights add up to 1: (150 + 8) 2^-24 and 2^-17 for scores and lse of at most 2^5
    for s, n in zip(slots.tolist(), lens):
        assert abs(float(weights[s].double().sum()) - n * H) <= n * H * (2.0 ** -17 + 158 * R.F)
    at = [0, 150, 183]
    hold = [(k[a:a + n].double(), v[a:a + n].double()) for a, n in zip(at, lens)]
    T = 3
    for step in range(3):
        kept, status = K.kda_cache_evict(slots, keep, kc, vc, table, length, refs, weights, first=first, recent=recent)
        assert status.tolist() == [0, 0, 0]
        for b in range(3):
            stay = kept[b][kept[b] >= 0].long()
            assert stay.numel() == min(keep, hold[b][0].shape[0]) == int(length[slots[b].long()])
            hold[b] = tuple(t[stay] for t in hold[b])
        now = length[slots.long()]
        assert K.kda_cache_reserve(slots, now + T, page, table, length, refs).tolist() == [0, 0, 0]
        tq, tk, tv = new(3, T, H, d), new(3, T, Hkv, d), new(3, T, Hkv, d)
        mask = torch.tensor([1, 3, 5], dtype=torch.int64, device="cuda").repeat(3, 1)  # 0, 0-1, 0-2
        out, lse = K.kda_attn_window_tree(tq, tk, tv, kc, vc, table, length, 40, sinks=2, tree_mask=mask, slot_indices=slots)
        for b in range(3):
            n = hold[b][0].shape[0]
            line = torch.arange(n + T, device="cuda")
            seen = torch.zeros(T, n + T, dtype=torch.bool, device="cuda")
            for t, path in enumerate(([0], [0, 1], [0, 2])):
                ends = n + len(path)
                places = torch.cat([line[:n], torch.tensor(path, device="cuda") + n])
                view = (torch.arange(ends, device="cuda") < 2) | (torch.arange(ends, device="cuda") >= ends - 40)
                seen[t, places[view]] = True
            for h in range(H):
                o, bo, l, bl, _, _ = R.softmax_rows(tq[b, :, h].double(), torch.cat([hold[b][0][:, h // G], tk[b, :, h // G].double()]),
                                                    torch.cat([hold[b][1][:, h // G], tv[b, :, h // G].double()]), d ** -0.5, seen, u)
                R.check(f"step {step} {b},{h}", out[b, :, h], o, bo + u * (o.abs() + bo) + 1e-30)
                R.check(f"lse {step} {b},{h}", lse[b, :, h], l, bl)
        # the path 0-2 is accepted
        rows, cu2 = ints([0, 2, 3, 5, 6, 8]), ints([0, 2, 4, 6])
        K.kda_cache_append(tk.view(-1, Hkv, d), tv.view(-1, Hkv, d), kc, vc, table, length, cu2, rows=rows, slot_indices=slots)
        length[slots.long()] = now + 2
        before = weights.double().sum(1)
        K.kda_cache_weigh(tq.view(-1, H, d), lse.view(-1, H), kc, table, length, weights, cu_seqlens=cu2, rows=rows, slot_indices=slots,
                          window=40, sinks=2)
        more = weights.double().sum(1) - before
        for b, s in enumerate(slots.tolist()):
            assert abs(float(more[s]) - 2 * H) <= 2 * H * (2.0 ** -17 + 158 * R.F) + float(weights[s].double().sum()) * 2 * R.F
            hold[b] = tuple(torch.cat([t, x[b, [0, 2]].double()]) for t, x in zip(hold[b], (tk, tv)))
    assert int(refs.sum()) == int((table >= 0).sum())
