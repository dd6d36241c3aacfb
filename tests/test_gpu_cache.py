"""The pages of an attention cache on the GPU against a plain model that takes
the entries of a call one after another, and the attention operators together
as a server uses them."""

import math
import random

import numpy as np
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


class Model:
    """A cache on the host; every page's rows are numbered integers."""

    def __init__(self, pages, page, slots, width):
        self.page = page
        self.table = np.full((slots, width), -1, dtype=np.int32)
        self.lens = np.zeros(slots, dtype=np.int32)
        self.refs = np.zeros(pages, dtype=np.int32)

    def free_pages(self):
        return [p for p in range(len(self.refs)) if self.refs[p] <= 0]

    def there(self, s):
        return 0 <= s < len(self.lens)

    def names(self, e):
        return 0 <= e < len(self.refs)

    def free(self, slots):
        for s in slots:
            if not self.there(s):
                continue
            for e in self.table[s]:
                if self.names(e):
                    self.refs[e] -= 1
            self.table[s] = -1
            self.lens[s] = 0

    def reserve(self, slots, new_lens):
        width = self.table.shape[1]
        status, seen, wants = [], set(), []
        for s, n in zip(slots, new_lens):
            cols = -(-max(n, 0) // self.page)
            if not self.there(s) or cols > width or s in seen:
                status.append(2)
                wants.append([])
                continue
            seen.add(s)
            first = -(-max(int(self.lens[s]), 0) // self.page)
            status.append(0)
            wants.append([(s, j) for j in range(first, cols) if not self.names(self.table[s, j])])
        free, at, full = self.free_pages(), 0, False
        for i, w in enumerate(wants):
            if not w:
                continue
            if full or at + len(w) > len(free):
                status[i], full = 1, True
                continue
            for s, j in w:
                self.table[s, j] = free[at]
                self.refs[free[at]] = 1
                at += 1
        return status

    def fork(self, src, dst):
        """(status, copies as (from page, to page, rows))"""
        table, lens = self.table.copy(), self.lens.copy()  # sources as they were at the start
        status, copies, seen = [], [], set()
        free, at = self.free_pages(), 0
        for s, d in zip(src, dst):
            good = self.there(s) and self.there(d) and s != d and lens[d] == 0 and not self.names(table[d, 0]) and d not in seen
            if not good:
                status.append(2)
                continue
            seen.add(d)
            n = min(max(int(lens[s]), 0), self.page * table.shape[1])
            full, part = n // self.page, n % self.page
            last = table[s, full] if part else -1
            if part and self.names(last):
                if at >= len(free):
                    status.append(1)
                    continue
                copies.append((int(last), free[at], part))
                last = free[at]
                self.refs[last] = 1
                at += 1
            elif part:
                last = -1
            status.append(0)
            self.table[d, :full] = table[s, :full]
            for e in table[s, :full]:
                if self.names(e):
                    self.refs[e] += 1
            if part:
                self.table[d, full] = last
            self.lens[d] = n
        return status, copies

    def compact(self):
        """(pages in use, moves as (from, to))"""
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        live = len(used)
        moves = list(zip([p for p in used if p >= live], [p for p in range(live) if self.refs[p] <= 0]))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        for i, e in np.ndenumerate(self.table):
            if int(e) in to:
                self.table[i] = to[int(e)]
        return live, moves


class Device:
    """The same cache on the device, its pools filled with numbers that name
    their place."""

    def __init__(self, m, Hkv, dk, dv, dtype=torch.float32):
        self.table, self.lens, self.refs = (torch.from_numpy(x.copy()).cuda() for x in (m.table, m.lens, m.refs))
        pages = len(m.refs)
        fill = lambda d: torch.arange(pages * Hkv * m.page * d, device="cuda").remainder(251).to(dtype).view(pages, Hkv, m.page, d)  # noqa: E731
        self.kc, self.vc = fill(dk).contiguous(), fill(dv).contiguous() + 1

    def same(self, m):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), m.table)
        assert np.array_equal(self.lens.cpu().numpy(), m.lens)
        assert np.array_equal(self.refs.cpu().numpy(), m.refs)


def _ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _filled(seed, pages=60, page=16, slots=12, width=9, used=7):
    m, r = Model(pages, page, slots, width), random.Random(seed)
    order = list(range(pages))
    r.shuffle(order)
    for s in r.sample(range(slots), used):
        n = r.choice([1, page - 1, page, page + 1, 3 * page, r.randint(1, 5 * page)])
        for j in range(-(-n // page)):
            m.table[s, j] = order.pop()
            m.refs[m.table[s, j]] += 1
        m.lens[s] = n
    return m, r


@pytest.mark.parametrize("seed", range(4))
def test_free(K, seed):
    m, r = _filled(seed)
    d = Device(m, 1, 16, 16)
    slots = [r.randint(-2, 13) for _ in range(5)]
    slots += slots[:2]  # the same slot twice
    print("free", slots, flush=True)
    K.kda_cache_free(_ints(slots), d.table, d.lens, d.refs)
    m.free(slots)
    d.same(m)


@pytest.mark.parametrize("seed", range(6))
def test_reserve(K, seed):
    m, r = _filled(seed, pages=[60, 40, 45][seed % 3])
    d = Device(m, 1, 16, 16)
    slots = [r.randint(-1, 12) for _ in range(9)]
    lens = [r.choice([0, -3, 5, 16, 17, 60, 144, 145, r.randint(0, 200)]) for _ in slots]
    print("reserve", slots, lens, flush=True)
    got = K.kda_cache_reserve(_ints(slots), _ints(lens), m.page, d.table, d.lens, d.refs)
    want = m.reserve(slots, lens)
    assert got.tolist() == want
    d.same(m)


def test_reserve_in_a_large_pool(K):
    """A pool of several scan steps, full but for its end; a row filled whole."""
    m = Model(30000, 16, 40, 700)
    m.refs[:] = 1
    m.refs[25000:] = 0
    m.refs[::97] = 0
    d = Device(m, 1, 16, 16)
    slots, lens = list(range(40)), [700 * 16 if s == 3 else 37 * s for s in range(40)]
    got = K.kda_cache_reserve(_ints(slots), _ints(lens), 16, d.table, d.lens, d.refs)
    assert got.tolist() == m.reserve(slots, lens)
    d.same(m)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(16, 16), (192, 128)])
@pytest.mark.parametrize("seed", range(4))
def test_fork(K, seed, dk, dv, dtype):
    m, r = _filled(seed, pages=[60, 38][seed % 2])
    d = Device(m, 3, dk, dv, dtype)
    k0, v0 = d.kc.clone(), d.vc.clone()
    src = [r.randint(-1, 12) for _ in range(14)]
    dst = [r.randint(-1, 12) for _ in range(14)]
    print("fork", src, dst, flush=True)
    got = K.kda_cache_fork(_ints(src), _ints(dst), d.kc, d.vc, d.table, d.lens, d.refs)
    want, copies = m.fork(src, dst)
    assert got.tolist() == want
    d.same(m)
    for a, b, n in copies:
        k0[b, :, :n], v0[b, :, :n] = k0[a, :, :n], v0[a, :, :n]
    assert torch.equal(d.kc, k0) and torch.equal(d.vc, v0)


def test_fork_many_from_one(K):
    """One parent, more beams than a planning step has lanes."""
    n = 1500
    m = Model(1600, 16, n + 1, 4)
    m.table[0, :3], m.lens[0] = [5, 1599, 7], 40
    m.refs[[5, 1599, 7]] = 1
    d = Device(m, 1, 16, 16)
    src, dst = [0] * n, list(range(n, 0, -1))
    got = K.kda_cache_fork(_ints(src), _ints(dst), d.kc, d.vc, d.table, d.lens, d.refs)
    assert got.tolist() == m.fork(src, dst)[0]
    d.same(m)


@pytest.mark.parametrize("seed", range(4))
def test_compact(K, seed):
    m, r = _filled(seed, pages=[60, 200, 36, 45][seed])
    m.free([s for s in range(12) if r.random() < 0.4])
    src = [s for s in range(12) if m.lens[s]][:1]
    m.fork(src * 3, [s for s in range(12) if not m.lens[s]][:3])  # shared pages move once
    d = Device(m, 2, 32, 32)
    k0, v0 = d.kc.clone(), d.vc.clone()
    live = K.kda_cache_compact(d.kc, d.vc, d.table, d.refs)
    want, moves = m.compact()
    assert live.tolist() == [want]
    d.same(m)
    for a, b in moves:
        k0[b], v0[b] = k0[a], v0[a]
    assert torch.equal(d.kc, k0) and torch.equal(d.vc, v0)


@pytest.mark.parametrize("fill", [0, 1])
def test_compact_empty_and_full(K, fill):
    m = Model(20000, 16, 3, 4)
    m.refs[:] = fill
    d = Device(m, 1, 16, 16)
    k0 = d.kc.clone()
    live = K.kda_cache_compact(d.kc, d.vc, d.table, d.refs)
    assert live.tolist() == [20000 * fill]
    d.same(m)
    assert torch.equal(d.kc, k0)


@pytest.mark.parametrize("shape,dtype", [((9, 4), torch.float32), ((12, 2, 128, 128), torch.float32), ((7, 8), torch.bfloat16),
                                         ((5, 3, 16, 40), torch.bfloat16)])
def test_copy(K, shape, dtype):
    """Rows of any pool: KDA states, conv histories, pages."""
    pool = torch.randn(shape, device="cuda").to(dtype)
    src, dst = [0, 2, -1, 1, 3, 0, shape[0]], [4, shape[0] - 1, 1, 1, -5, shape[0], 2]
    want = pool.clone()
    want[4], want[shape[0] - 1] = pool[0], pool[2]
    print("copy", shape, flush=True)
    if shape[0] - 1 == 4:  # one row written twice: keep the first
        src, dst = src[:1], dst[:1]
        want = pool.clone()
        want[4] = pool[0]
    K.kda_cache_copy(pool, _ints(src), _ints(dst))
    assert torch.equal(pool, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Hkv,dk,dv,page", [(1, 16, 16, 16), (3, 64, 64, 32), (2, 192, 128, 64), (8, 128, 128, 16)])
def test_append(K, Hkv, dk, dv, page, dtype):
    """Packed prompts, then an accepted path per sequence; what has no page,
    no slot or no source is dropped; nothing else is written."""
    counts, ctx = [70, 0, 5, 1, 33], [0, 9, page - 2, 3 * page, 2]
    N, slots = len(counts), 8
    rows_of = [6, 0, 2, 9, 4]  # the fourth has no slot
    m = Model(60, page, slots, 9)
    free = list(range(59, -1, -1))
    for n, s in enumerate(rows_of):
        if s < slots:
            for j in range(-(-(ctx[n] + counts[n]) // page)):
                m.table[s, j] = free.pop()
            m.lens[s] = ctx[n]
    m.table[6, 1] = -1  # the first sequence lacks its second page
    d = Device(m, Hkv, dk, dv, dtype)
    total = sum(counts)
    cu = _ints(np.concatenate([[0], np.cumsum(counts)]))
    spare = 3
    k, v = torch.randn(total + spare, Hkv, dk, device="cuda").to(dtype), torch.randn(total + spare, Hkv, dv, device="cuda").to(dtype)
    for rows in (None, torch.randperm(total + spare, device="cuda").to(torch.int32)):
        if rows is not None:
            rows[3], rows[71] = -1, total + spare
        k0, v0 = d.kc.clone(), d.vc.clone()
        K.kda_cache_append(k, v, d.kc, d.vc, d.table, d.lens, cu, rows=rows, slot_indices=_ints(rows_of))
        t = 0
        for n, s in enumerate(rows_of):
            for i in range(counts[n]):
                src = t if rows is None else int(rows[t])
                t += 1
                pos = ctx[n] + i
                if s >= slots or not 0 <= src < total + spare or m.table[s, pos // page] < 0:
                    continue
                p = m.table[s, pos // page]
                k0[p, :, pos % page], v0[p, :, pos % page] = k[src], v[src]
        assert torch.equal(d.kc, k0) and torch.equal(d.vc, v0)
        d.same(m)


def test_append_behind_the_table(K):
    m = Model(4, 16, 1, 2)
    m.table[0], m.lens[0] = [1, 3], 30
    d = Device(m, 1, 16, 16)
    k0 = d.kc.clone()
    k = torch.randn(5, 1, 16, device="cuda")
    K.kda_cache_append(k, k, d.kc, d.vc, d.table, d.lens)
    k0[3, 0, 14:16] = k[:2, 0]
    assert torch.equal(d.kc, k0)
    d.lens[0] = 2 ** 31 - 1  # far behind: nothing is written
    K.kda_cache_append(k, k, d.kc, d.vc, d.table, d.lens)
    assert torch.equal(d.kc, k0)


def test_append_past_32_bits(K):
    Hkv, page, dim = 8, 64, 128
    pages = (1 << 32) // (Hkv * page * dim * 2) + 5
    kc = torch.zeros((pages, Hkv, page, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table = _ints([pages - 1]).view(1, 1)
    k = torch.randn(7, Hkv, dim, device="cuda").bfloat16()
    K.kda_cache_append(k, k, kc, vc, table, _ints([2]))
    assert torch.equal(kc[-1, :, 2:9], k.transpose(0, 1)) and torch.equal(vc[-1, :, 2:9], k.transpose(0, 1))
    assert float(kc[:-1].abs().max()) == 0
    rows = _ints([pages - 1]), _ints([pages - 2])
    K.kda_cache_copy(kc, *rows)
    assert torch.equal(kc[-2], kc[-1])


def test_captured_and_replayed(K):
    """A beam step (free, fork, reserve) in one graph, replayed."""
    m, _ = _filled(1, pages=80)
    parents = [s for s in range(12) if m.lens[s]][:3]
    empty = [s for s in range(12) if not m.lens[s]][:4]
    src, dst = [parents[i % 3] for i in range(4)], empty
    new = [int(m.lens[s]) + 20 for s in src]
    d = Device(m, 2, 16, 16)
    args = _ints(src), _ints(dst), _ints(new)
    ws = torch.empty(K.kda_cache_workspace_bytes(80, 12, 4), dtype=torch.uint8, device="cuda")
    st = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")

    def step():
        K.kda_cache_free(args[1], d.table, d.lens, d.refs)
        K.kda_cache_fork(args[0], args[1], d.kc, d.vc, d.table, d.lens, d.refs, status=st[0], workspace=ws)
        K.kda_cache_reserve(args[1], args[2], 16, d.table, d.lens, d.refs, status=st[1], workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    m.fork(src, dst)
    m.reserve(dst, new)
    d.same(m)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        order = src[i:] + src[:i]
        args[0].copy_(_ints(order))
        args[2].copy_(_ints([int(m.lens[p]) + 20 for p in order]))
        graph.replay()
        torch.cuda.synchronize()
        m.free(dst)
        m.fork(order, dst)
        m.reserve(dst, [int(m.lens[p]) + 20 for p in order])
        d.same(m)


def test_debug_check_of_copies(K, monkeypatch):
    monkeypatch.setenv("KDA_DEBUG_CHECK", "1")
    pool = torch.zeros(6, 4, device="cuda")
    with pytest.raises(Exception, match="written twice"):
        K.kda_cache_copy(pool, _ints([0, 1]), _ints([3, 3]))
    with pytest.raises(Exception, match="written by the same copy"):
        K.kda_cache_copy(pool, _ints([0, 3]), _ints([3, 4]))
    K.kda_cache_copy(pool, _ints([0, 0]), _ints([3, 4]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_server_run(K, dtype):
    """Prompts in, draft trees verified, their accepted paths committed, a
    beam forked (its KDA state with it), an old sequence freed, the pool
    compacted; every attention output against plain attention over the
    sequence as it then is."""
    H, Hkv, dk, dv, page, scale = 4, 2, 64, 64, 16, 64 ** -0.5
    g, r = torch.Generator(device="cuda"), random.Random(3)
    g.manual_seed(3)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    pages, slots, width = 40, 4, 12
    kc, vc = (torch.full((pages, Hkv, page, d), math.nan, dtype=dtype, device="cuda") for d in (dk, dv))
    table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(slots, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    state = torch.randn(slots, H, 64, 64, generator=g, device="cuda")
    prompts = [37, 16, 50]
    use = _ints([2, 0, 3])
    T = sum(prompts)
    cu = _ints(np.concatenate([[0], np.cumsum(prompts)]))
    q, k, v = new(T, H, dk), new(T, Hkv, dk), new(T, Hkv, dv)
    assert K.kda_cache_reserve(use, _ints(prompts), page, table, lens, refs).tolist() == [0, 0, 0]
    K.kda_cache_append(k, v, kc, vc, table, lens, cu, slot_indices=use)
    lens.index_add_(0, use.long(), _ints(prompts))
    out, lse = K.kda_attn_prefill(q, k, v, cu_seqlens=cu, scale=scale)
    want, bo, wl, bl = R.prefill(q.double(), k.double(), v.double(), None, prompts, scale, dtype)
    R.check("prompt", out, want, bo)
    # the last prompt token again, as a decode step over the tokens before it: the same row
    tail = torch.tensor(prompts, device="cuda").cumsum(0) - 1
    lens.index_add_(0, use.long(), _ints([-1] * 3))
    o1, l1 = K.kda_attn_tree(q[tail][:, None].contiguous(), k[tail][:, None].contiguous(), v[tail][:, None].contiguous(), kc, vc,
                             table, lens, slot_indices=use, scale=scale)
    R.check("decode of the last token", o1[:, 0], want[tail], bo[tail] * 2)
    R.check("its lse", l1[:, 0], wl[tail], bl[tail] * 2)
    lens.index_add_(0, use.long(), _ints([1] * 3))
    held = {2: [k[:37], v[:37]], 0: [k[37:53], v[37:53]], 3: [k[53:], v[53:]]}

    def verify(order, D):
        B = len(order)
        qd, kd, vd = new(B, D, H, dk), new(B, D, Hkv, dk), new(B, D, Hkv, dv)
        parents = [[-1] + [r.randint(-1, t - 1) for t in range(1, D)] for _ in order]
        words = torch.zeros(B, D, dtype=torch.int64)
        paths = []
        for b in range(B):
            ps = []
            for t in range(D):
                p = [t]
                while parents[b][p[0]] >= 0:
                    p.insert(0, parents[b][p[0]])
                ps.append(p)
                words[b, t] = sum(1 << a for a in p)
            paths.append(ps)
        o, l = K.kda_attn_tree(qd, kd, vd, kc, vc, table, lens, tree_mask=words.cuda(), slot_indices=_ints(order), scale=scale)
        for b, s in enumerate(order):
            n = held[s][0].shape[0]
            assert int(lens[s]) == n
            new_seen = torch.tensor([[bool(int(words[b, t]) >> j & 1) for j in range(D)] for t in range(D)], device="cuda")
            seen = torch.cat([torch.ones(D, n, dtype=torch.bool, device="cuda"), new_seen], 1)
            for h in range(H):
                kk, vv = (torch.cat([held[s][i][:, h // 2], (kd, vd)[i][b, :, h // 2]]).double() for i in (0, 1))
                w, bw, wl_, bl_, _, _ = R.softmax_rows(qd[b, :, h].double(), kk, vv, scale, seen, R.UNIT[dtype])
                R.check(f"verify slot {s} head {h}", o[b, :, h], w, bw + R.UNIT[dtype] * (w.abs() + bw) + 1e-30)
        # accept a path of each tree
        taken = [r.choice(p) for p in paths]
        counts = [len(p) for p in taken]
        rows = _ints([b * D + t for b, p in enumerate(taken) for t in p])
        st = K.kda_cache_reserve(_ints(order), _ints([held[s][0].shape[0] + c for s, c in zip(order, counts)]), page, table, lens, refs)
        assert st.tolist() == [0] * B
        K.kda_cache_append(kd.view(B * D, Hkv, dk), vd.view(B * D, Hkv, dv), kc, vc, table, lens,
                           _ints(np.concatenate([[0], np.cumsum(counts)])), rows=rows, slot_indices=_ints(order))
        lens.index_add_(0, _ints(order).long(), _ints(counts))
        for b, s in enumerate(order):
            held[s] = [torch.cat([held[s][0], kd[b, taken[b]]]), torch.cat([held[s][1], vd[b, taken[b]]])]

    verify([2, 0, 3], 7)
    verify([0, 3, 2], 12)
    # slot 2 goes on in two ways
    assert K.kda_cache_fork(_ints([2]), _ints([1]), kc, vc, table, lens, refs).tolist() == [0]
    K.kda_cache_copy(state, _ints([2]), _ints([1]))
    assert torch.equal(state[1], state[2])
    held[1] = list(held[2])
    verify([1, 2, 0, 3], 5)
    K.kda_cache_free(_ints([0]), table, lens, refs)
    live = int(K.kda_cache_compact(kc, vc, table, refs))
    assert live == int((refs > 0).sum()) and int(table.max()) < live and bool((refs[live:] == 0).all())
    kc[live:], vc[live:] = math.nan, math.nan  # nothing there is read any more
    verify([3, 1, 2], 9)
    K.kda_cache_free(_ints([0, 1, 2, 3]), table, lens, refs)
    assert int(refs.abs().sum()) == 0 and bool((table == -1).all()) and int(lens.sum()) == 0
