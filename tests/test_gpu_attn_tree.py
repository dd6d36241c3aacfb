"""Attention of drafted tokens over a paged cache on the GPU against plain
64-bit attention (attn_ref)."""

import math
import random

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


def _make(seed, lens, T, H, Hkv, dk, dv, page, dtype, gate=False, mask="tree", spare_slots=2, width=None):
    """A cache whose unused memory holds NaN, drafts and masks for one
    sequence per entry of lens."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    width = width or max(max(need, default=0), 1) + 1
    pages, slots = sum(need) + 3, B + spare_slots
    order = list(range(pages))
    r.shuffle(order)
    row = r.sample(range(slots), B)
    table = torch.full((slots, width), -1, dtype=torch.int32)
    length = torch.zeros(slots, dtype=torch.int32)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    kc = torch.full((pages, Hkv, page, dk), math.nan, dtype=dtype, device="cuda")
    vc = torch.full((pages, Hkv, page, dv), math.nan, dtype=dtype, device="cuda")
    ctx_k, ctx_v, at = [], [], 0
    for b, n in enumerate(lens):
        k, v = new(n, Hkv, dk), new(n, Hkv, dv)
        ctx_k.append(k)
        ctx_v.append(v)
        for j in range(need[b]):
            p = order[at]
            at += 1
            table[row[b], j] = p
            m = min(page, n - j * page)
            kc[p, :, :m] = k[j * page:j * page + m].transpose(0, 1)
            vc[p, :, :m] = v[j * page:j * page + m].transpose(0, 1)
        length[row[b]] = n
    words = None
    if mask == "tree":
        words = torch.zeros((B, T), dtype=torch.int64)
        for b in range(B):
            parents = [-1] + [r.randint(-1, t - 1) for t in range(1, T)]
            for t in range(T):
                w, a = 0, t
                while a >= 0:
                    w |= 1 << a
                    a = parents[a]
                words[b, t] = w - (1 << 64) if w >= 1 << 63 else w
        words = words.cuda()
    return dict(q=new(B, T, H, dk), k_new=new(B, T, Hkv, dk), v_new=new(B, T, Hkv, dv), kc=kc, vc=vc,
                table=table.cuda(), lens=length.cuda(), rows=torch.tensor(row, dtype=torch.int32, device="cuda"),
                mask=words, z=new(B, T, H, dv) if gate else None, ctx_k=ctx_k, ctx_v=ctx_v)


def _call(K, x, **kw):
    got = K.kda_attn_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"], x["lens"], tree_mask=x["mask"],
                          out_gate=x["z"], slot_indices=x["rows"], **kw)
    torch.cuda.synchronize()
    return got


def _check(K, x, dtype, scale=None, dropped=None):
    """dropped: {b: truth values over the context's tokens that are not there}."""
    out, lse = _call(K, x, scale=scale)
    B, T, H, dk = x["q"].shape
    Hkv, dv = x["k_new"].shape[2], x["v_new"].shape[3]
    G, sc = H // Hkv, scale or dk ** -0.5
    for b in range(B):
        n = x["ctx_k"][b].shape[0]
        new = torch.zeros(T, T, dtype=torch.bool, device="cuda")
        for t in range(T):
            for j in range(T):
                new[t, j] = j <= t if x["mask"] is None else bool(int(x["mask"][b, t]) >> j & 1)
        old = torch.ones(T, n, dtype=torch.bool, device="cuda")
        if dropped and b in dropped:
            old &= ~dropped[b]
        seen = torch.cat([old, new], 1)
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
    """Contexts of every length around a tile and a page, a gate."""
    print(f"tree {dk}/{dv} {dtype}", flush=True)
    x = _make(dk, [0, 1, 15, 16, 17, 33, 130], 7, 4, 2, dk, dv, 16, TYPES[dtype], gate=True)
    _check(K, x, TYPES[dtype])


@pytest.mark.parametrize("page", [16, 32, 64, 256, 1024])
@pytest.mark.parametrize("T,H,Hkv", [(1, 4, 4), (1, 8, 1), (4, 4, 2), (33, 2, 1), (64, 2, 2)])
def test_tokens_heads_pages(K, T, H, Hkv, page):
    print(f"tree T={T} H={H}/{Hkv} page={page}", flush=True)
    x = _make(T + page, [200, 31, 0], T, H, Hkv, 64, 64, page, torch.bfloat16)
    _check(K, x, torch.bfloat16)


@pytest.mark.parametrize("T,G", [(16, 4), (40, 8), (64, 16)])
def test_many_rows(K, T, G):
    """More rows per key head than one workgroup takes."""
    print(f"tree rows T={T} G={G}", flush=True)
    for dk, dv in ((128, 128), (192, 128)):
        x = _make(T, [300, 5], T, G, 1, dk, dv, 64, torch.bfloat16)
        _check(K, x, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 9])
def test_split_over_a_long_context(K, T, dtype):
    """Few rows, many keys: several workgroups per head, joined after."""
    print(f"tree long T={T} {dtype}", flush=True)
    x = _make(T, [5000, 700, 1], T, 4, 2, 128, 128, 64, TYPES[dtype], gate=True, mask="chain" if T == 1 else "tree")
    _check(K, x, TYPES[dtype])


def test_long_table_short_contexts(K):
    """A table with room for far more than is there: most parts are empty."""
    x = _make(3, [40, 0, 3], 3, 4, 1, 64, 64, 64, torch.bfloat16, gate=True, width=500)
    _check(K, x, torch.bfloat16)


def test_chain_equals_its_mask(K):
    x = _make(4, [77, 200], 9, 4, 2, 128, 128, 32, torch.bfloat16, mask="chain")
    a = _call(K, x)
    x["mask"] = torch.tensor([(1 << (t + 1)) - 1 for t in range(9)], dtype=torch.int64, device="cuda").repeat(2, 1)
    b = _call(K, x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("width", [None, 300])
def test_rows_that_attend_nothing(K, width):
    """Empty masks over an empty context: 0 and -infinity; bits behind the
    last draft are not looked at."""
    x = _make(5, [0, 50], 6, 2, 1, 64, 64, 16, torch.bfloat16, gate=True, width=width)
    x["mask"][0, 2] = 0
    x["mask"][0, 4] = -64  # bits 6 and up only
    x["mask"][1, 3] = 0
    out, lse = _check(K, x, torch.bfloat16)
    assert bool((out[0, [2, 4]] == 0).all()) and bool(torch.isneginf(lse[0, [2, 4]]).all())


@pytest.mark.parametrize("width", [None, 300])
def test_padding_rows_and_slots_used_twice(K, width):
    x = _make(6, [60, 20, 90, 10], 3, 4, 2, 64, 64, 16, torch.float32, gate=True, width=width)
    want = _call(K, x)
    rows = x["rows"].clone()
    x["rows"][1], x["rows"][2] = -1, x["table"].shape[0]
    x["q"][1], x["z"][2] = math.nan, math.nan
    out, lse = _call(K, x)
    for b in (1, 2):
        assert bool((out[b] == 0).all()) and bool(torch.isneginf(lse[b]).all())
    for b in (0, 3):
        assert torch.equal(out[b], want[0][b]) and torch.equal(lse[b], want[1][b])
    x["rows"] = rows[[0, 0, 3, 3]].contiguous()
    for n in ("q", "k_new", "v_new", "z", "mask"):
        x[n] = x[n][[0, 0, 3, 3]].contiguous()
    out, lse = _call(K, x)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], want[0][0]) and torch.equal(out[3], want[0][3])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_entries_that_name_no_page(K, dtype):
    """A page dropped from the middle, one outside the pool: their tokens are
    not attended."""
    x = _make(7, [200, 64], 4, 2, 1, 32, 32, 16, TYPES[dtype])
    r = int(x["rows"][0])
    x["table"][r, 3], x["table"][r, 6] = -1, x["kc"].shape[0]
    gone = torch.zeros(200, dtype=torch.bool, device="cuda")
    gone[48:64] = True
    gone[96:112] = True
    _check(K, x, TYPES[dtype], dropped={0: gone})


def test_lengths_past_the_table(K):
    """A length above what the row holds is clamped, a negative one is none."""
    x = _make(8, [64, 32], 2, 2, 2, 64, 64, 16, torch.float32, width=4)
    want = _call(K, x)
    x["lens"][int(x["rows"][0])] = 2 ** 31 - 1
    got = _call(K, x)
    assert torch.equal(got[0], want[0])
    x["lens"][int(x["rows"][1])] = -5
    x["ctx_k"][1], x["ctx_v"][1] = x["ctx_k"][1][:0], x["ctx_v"][1][:0]
    _check(K, x, torch.float32)


def test_steep_softmax_across_parts(K):
    x = _make(9, [3000], 2, 2, 1, 64, 64, 64, torch.float32)
    x["q"] *= 50
    _check(K, x, torch.float32)


def test_offsets_past_32_bits(K):
    """Pools of more than 2^32 bytes, the pages in use at their end."""
    Hkv, page, d = 8, 64, 128
    pages = (1 << 32) // (Hkv * page * d * 2) + 9
    kc = torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    x = _make(10, [100], 1, 16, Hkv, d, d, page, torch.bfloat16, mask="chain", spare_slots=0)
    small = x["table"].clone()
    for j in range(2):
        p = pages - 1 - 3 * j
        kc[p], vc[p] = x["kc"][int(small[0, j])], x["vc"][int(small[0, j])]
        x["table"][0, j] = p
    x["kc"], x["vc"] = kc, vc
    _check(K, x, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_drafts_that_are_not_finite(K, dtype):
    """Unused drafts may hold anything (a padded tree); a value that is not
    finite reaches the rows that attend its draft and no others."""
    x = _make(14, [70, 0, 33], 40, 4, 2, 64, 64, 16, TYPES[dtype])
    want, wl = _call(K, x)
    words = x["mask"].cpu()
    y = dict(x, k_new=x["k_new"].clone(), v_new=x["v_new"].clone(), mask=x["mask"].clone())
    for b, j in ((0, 7), (1, 39), (2, 33)):  # drafts that nobody attends any more
        y["mask"][b] &= ~(1 << j)
        y["k_new"][b, j], y["v_new"][b, j] = math.nan, math.inf
    out, lse = _call(K, y)
    clean = dict(y, k_new=x["k_new"], v_new=x["v_new"])
    a, al = _call(K, clean)
    assert torch.equal(out, a) and torch.equal(lse, al)
    y = dict(x, v_new=x["v_new"].clone())
    y["v_new"][0, 5, 1, 3], y["v_new"][0, 38, 0, 63] = math.nan, -math.inf
    out, lse = _call(K, y)
    assert torch.equal(lse, wl)
    for t in range(40):
        w = want[0, t].clone()
        if int(words[0, t]) >> 5 & 1:
            w[2:, 3] = math.nan
        if int(words[0, t]) >> 38 & 1:
            w[:2, 63] = -math.inf
        assert torch.equal(torch.isnan(out[0, t]), torch.isnan(w)), t
        fine = ~torch.isnan(w)
        assert torch.equal(out[0, t][fine], w[fine]), t
    assert torch.equal(out[1:], want[1:])


def test_captured_and_replayed(K):
    """One graph over a decode step whose lengths and tables change."""
    x = _make(11, [900, 300, 20], 4, 8, 2, 128, 128, 64, torch.bfloat16, width=40)
    lens = x["lens"].clone()
    ws = torch.empty(max(256, K.kda_attn_tree_workspace_bytes(3, 4, 8, 2, 128, 128, torch.bfloat16, 40 * 64)),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _call(K, x, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = K.kda_attn_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"], x["lens"],
                                   tree_mask=x["mask"], slot_indices=x["rows"], workspace=ws)
    for i in range(4):
        x["lens"].copy_((lens - 5 * i).clamp(min=0))
        x["q"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        want = _call(K, x)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i


def test_binding_refuses(K):
    x = _make(12, [20], 2, 2, 1, 64, 64, 16, torch.float32)
    with pytest.raises(ValueError):
        K.kda_attn_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"][:-1], x["table"], x["lens"])
    with pytest.raises(TypeError):
        K.kda_attn_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"].long(), x["lens"])
    with pytest.raises(Exception, match="slot_indices is NULL"):
        K.kda_attn_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"], x["lens"])


def test_empty_batches(K):
    x = _make(13, [20], 2, 2, 1, 64, 64, 16, torch.float32)
    out, lse = K.kda_attn_tree(x["q"][:0], x["k_new"][:0], x["v_new"][:0], x["kc"], x["vc"], x["table"], x["lens"],
                               slot_indices=x["rows"][:0])
    assert out.shape == (0, 2, 2, 64)
    out, lse = K.kda_attn_tree(x["q"][:, :0], x["k_new"][:, :0], x["v_new"][:, :0], x["kc"], x["vc"], x["table"], x["lens"],
                               slot_indices=x["rows"])
    assert out.shape == (1, 0, 2, 64)
