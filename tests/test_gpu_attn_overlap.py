"""Attention and cache calls that run at the same time, that share a workspace
in turn, and that name slots of a large cache."""

import random

import pytest
import torch

from test_gpu_attn_prefill import _check_backward, _check_forward, _cu, _inputs
from test_gpu_attn_tree import _check, _make
from test_gpu_cache import Device, Model, _ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


def _calls(K):
    """Calls with their workspaces' sizes: two gradients whose parts are joined
    and two split trees."""
    made = []
    for seed, lens in ((1, [700, 300]), (2, [64, 1, 900])):
        x = _inputs(seed, lens, 8, 2, 128, 128, torch.bfloat16, True)
        cu = _cu(lens)
        out, lse = K.kda_attn_prefill(x["q"], x["k"], x["v"], out_gate=x["z"], cu_seqlens=cu)
        need = K.kda_attn_backward_workspace_bytes(sum(lens), len(lens), 8, 2, 128, 128, torch.bfloat16, True)

        def gradients(ws, x=x, cu=cu, out=out, lse=lse):
            return [*K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], out, lse, x["dy"], out_gate=x["z"], cu_seqlens=cu,
                                                 workspace=ws).values()]
        made.append((need, gradients))
    for seed, lens in ((3, [5000, 70]), (4, [3001])):
        x = _make(seed, lens, 6, 8, 2, 128, 128, 64, torch.bfloat16, gate=True)
        need = K.kda_attn_tree_workspace_bytes(len(lens), 6, 8, 2, 128, 128, torch.bfloat16, x["table"].shape[1] * 64)
        assert need > 0, "these contexts are split"

        def draft(ws, x=x):
            return [*K.kda_attn_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["table"], x["lens"], tree_mask=x["mask"],
                                     out_gate=x["z"], slot_indices=x["rows"], workspace=ws)]
        made.append((need, draft))
    return made


def _space(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def test_at_the_same_time(K):
    """Every call on a stream of its own, with a workspace of its own."""
    made = _calls(K)
    want = [fn(_space(n)) for n, fn in made]
    spaces = [_space(n) for n, _ in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = []
    for _ in range(3):
        for s, (_, fn), ws in zip(streams, made, spaces):
            with torch.cuda.stream(s):
                got.append(fn(ws))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % len(made)])), i


def test_graphs_that_share_a_workspace(K):
    """A graph per call over one workspace, replayed in turn with eager calls on
    the same workspace between them."""
    made = _calls(K)
    want = [fn(_space(n)) for n, fn in made]
    ws = _space(max(n for n, _ in made))
    torch.cuda.synchronize()
    graphs = []
    for _, fn in made:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fn(ws)
        graphs.append((graph, out))
    for turn in range(3):
        for i, (graph, out) in enumerate(graphs):
            for t in out:
                t.zero_()
            made[(i + turn + 1) % len(made)][1](ws)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i])), (turn, i)


@pytest.mark.parametrize("slots", [8192, 8193, 20000])
def test_slots_of_a_large_cache(K, slots):
    """Entries that name a slot twice, in caches whose slots are claimed in LDS
    and in the workspace."""
    r = random.Random(slots)
    m = Model(4000, 16, slots, 3)
    d = Device(m, 1, 16, 16)
    some = r.sample(range(slots), 1100) + [0, slots - 1]
    lists = some + some[:300] + [-1, slots]
    r.shuffle(lists)
    new = [r.randint(0, 48) for _ in lists]
    ws = _space(K.kda_cache_workspace_bytes(4000, slots, 2 * len(lists)))
    got = K.kda_cache_reserve(_ints(lists), _ints(new), 16, d.table, d.lens, d.refs, workspace=ws)
    assert got.tolist() == m.reserve(lists, new)
    d.same(m)
    for s in set(some):  # lengths within what was reserved
        m.lens[s] = max(16 * int((m.table[s] >= 0).sum()) - 5, 0)
    d.lens.copy_(torch.from_numpy(m.lens))
    src = [r.choice(some) for _ in range(1500)]
    dst = [r.randrange(-1, slots + 1) for _ in range(1500)]
    got = K.kda_cache_fork(_ints(src), _ints(dst), d.kc, d.vc, d.table, d.lens, d.refs, workspace=ws)
    assert got.tolist() == m.fork(src, dst)[0]
    d.same(m)
    gone = lists + dst
    K.kda_cache_free(_ints(gone), d.table, d.lens, d.refs)
    m.free(gone)
    d.same(m)
    assert not m.refs.any()


@pytest.mark.parametrize("T", [32, 33, 63, 64])
def test_chains_of_many_tokens(K, T):
    """The last bits of a mask word, as a chain and as words of all ones up to
    the token (bit 63 makes a word negative)."""
    x = _make(21, [50, 0], T, 4, 2, 64, 64, 32, torch.float32, mask="chain")
    a = _check(K, x, torch.float32)
    words = [(1 << (t + 1)) - 1 for t in range(T)]
    x["mask"] = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda").repeat(2, 1)
    b = _check(K, x, torch.float32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[0, 129, 0, 1], [0, 0, 0], [500, 3, 0]])
def test_empty_sequences_and_a_gate(K, lens, dk, dv, dtype):
    """Sequences of no tokens between others, and a batch of nothing but rows
    behind the last sequence."""
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x = _inputs(31, lens, 4, 1, dk, dv, t, True, spare=130)
    out, lse = _check_forward(K, x, lens, t)
    if sum(lens):
        _check_backward(K, x, lens, t, out, lse)
    else:
        K.kda_attn_prefill_backward(x["q"], x["k"], x["v"], out, lse, x["dy"], out_gate=x["z"], cu_seqlens=_cu(lens))
        torch.cuda.synchronize()
