"""The windowed attention calls, the weights that cached tokens gather and the
cutting of slots refuse bad arguments on the host, before any device work, and
their workspaces hold every smaller call (CPU only)."""

import random

import pytest

import test_attn_abi as A
from gated_delta_rule_64_amd import _lib, kda
from test_attn_abi import BAD, CACHE_REFUSALS, FAKE, HEAD_REFUSALS, M, P, PAGE_REFUSALS, SMALL, UNSUP, _at, detail


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def prefill(lib, **kw):
    a = dict(T=64, H=4, Hkv=2, dk=64, dv=64, cu=None, N=1, x=1, scale=0.125, z=None, window=8, sinks=2, **_at(["q", "k", "v", "out", "lse"]))
    a.update(kw)
    return lib.kda_attn_window_prefill(a["T"], a["H"], a["Hkv"], a["dk"], a["dv"], P(a["cu"]), a["N"], a["x"], a["scale"], a["window"],
                                       a["sinks"], P(a["q"]), P(a["k"]), P(a["v"]), P(a["z"]), P(a["out"]), P(a["lse"]), None)


def backward(lib, **kw):
    a = dict(T=64, H=4, Hkv=2, dk=64, dv=64, cu=None, N=1, x=1, scale=0.125, z=None, gz=None, ws=FAKE + (1 << 36), ws_bytes=None,
             window=8, sinks=2, **_at(["q", "k", "v", "out", "lse", "dy", "gq", "gk", "gv"]))
    a.update(kw)
    if a["ws_bytes"] is None:
        a["ws_bytes"] = lib.kda_attn_window_backward_workspace_bytes(a["T"], a["N"], a["H"], a["Hkv"], a["dk"], a["dv"], a["x"],
                                                                     a["z"] is not None, a["window"], a["sinks"])
    return lib.kda_attn_window_prefill_backward(a["T"], a["H"], a["Hkv"], a["dk"], a["dv"], P(a["cu"]), a["N"], a["x"], a["scale"],
                                                a["window"], a["sinks"], P(a["q"]), P(a["k"]), P(a["v"]), P(a["z"]), P(a["out"]),
                                                P(a["lse"]), P(a["dy"]), P(a["gq"]), P(a["gk"]), P(a["gv"]), P(a["gz"]), P(a["ws"]),
                                                a["ws_bytes"], None)


def tree(lib, **kw):
    a = dict(B=2, T=4, H=4, Hkv=2, dk=64, dv=64, x=1, scale=0.125, mask=None, z=None, pages=10, page=16, slots=2, width=4, idx=None,
             ws=FAKE + (1 << 36), ws_bytes=1 << 30, window=8, sinks=2, **_at(["q", "k", "v", "kc", "vc", "table", "lens", "out", "lse"]))
    a.update(kw)
    return lib.kda_attn_window_tree(a["B"], a["T"], a["H"], a["Hkv"], a["dk"], a["dv"], a["x"], a["scale"], a["window"], a["sinks"],
                                    P(a["q"]), P(a["k"]), P(a["v"]), P(a["mask"]), P(a["z"]), P(a["kc"]), P(a["vc"]), a["pages"],
                                    a["page"], P(a["table"]), a["slots"], a["width"], P(a["lens"]), P(a["idx"]), P(a["out"]),
                                    P(a["lse"]), P(a["ws"]), a["ws_bytes"], None)


def weigh(lib, **kw):
    a = dict(T=8, N=1, cu=None, R=8, rows=None, H=4, Hkv=2, dk=64, x=1, scale=0.125, window=0, sinks=0, pages=10, page=16, slots=2,
             width=4, idx=None, ws=FAKE + (1 << 36), ws_bytes=1 << 30, **_at(["q", "lse", "kc", "table", "lens", "w"]))
    a.update(kw)
    return lib.kda_cache_weigh(a["T"], a["N"], P(a["cu"]), a["R"], P(a["rows"]), a["H"], a["Hkv"], a["dk"], a["x"], a["scale"],
                               a["window"], a["sinks"], P(a["q"]), P(a["lse"]), P(a["kc"]), a["pages"], a["page"], P(a["table"]),
                               a["slots"], a["width"], P(a["lens"]), P(a["idx"]), P(a["w"]), P(a["ws"]), a["ws_bytes"], None)


def evict(lib, **kw):
    a = dict(n=2, keep=20, first=2, recent=4, Hkv=2, dk=64, dv=64, x=1, pages=10, page=16, slots=2, width=4, ws=FAKE + (1 << 36),
             ws_bytes=1 << 30, kept=None, status=None, **_at(["list", "kc", "vc", "table", "lens", "refs", "w"]))
    a.update(kw)
    return lib.kda_cache_evict(a["n"], P(a["list"]), a["keep"], a["first"], a["recent"], a["Hkv"], a["dk"], a["dv"], a["x"], P(a["kc"]),
                               P(a["vc"]), a["pages"], a["page"], P(a["table"]), a["slots"], a["width"], P(a["lens"]), P(a["refs"]),
                               P(a["w"]), P(a["kept"]), P(a["status"]), P(a["ws"]), a["ws_bytes"], None)


WINDOWS = [(dict(window=0), BAD, "window=0"), (dict(window=-5), BAD, "window=-5"), (dict(sinks=-1), BAD, "sinks=-1")]


@pytest.mark.parametrize("kw,status,word", HEAD_REFUSALS + WINDOWS + [
    (dict(T=-1), BAD, "T_tot"), (dict(T=2**31), BAD, "T_tot"), (dict(T=2**29, H=1, Hkv=1, dk=16, dv=16), UNSUP, "2^29"), (dict(N=0), BAD, "N=0"),
    (dict(N=2), BAD, "cu_seqlens"), (dict(q=None), BAD, "q is NULL"), (dict(v=FAKE + 2 * M + 8), BAD, "aligned"),
    (dict(T=1 << 28, H=8, Hkv=1, dk=16, dv=16), UNSUP, "workgroups")])
def test_prefill_refuses(lib, kw, status, word):
    assert prefill(lib, **kw) == status
    assert word in detail(lib)


@pytest.mark.parametrize("kw,status,word", HEAD_REFUSALS + WINDOWS + [
    (dict(z=FAKE + 20 * M), BAD, "grad_out_gate"), (dict(lse=None), BAD, "lse is NULL"), (dict(ws_bytes=8), SMALL, "kda_attn_window_prefill_backward"),
    (dict(ws=FAKE + (1 << 36) + 16), BAD, "256-byte"), (dict(T=1 << 26, H=16, Hkv=1, dk=16, dv=16), UNSUP, "workgroups")])
def test_backward_refuses(lib, kw, status, word):
    assert backward(lib, **kw) == status
    assert word in detail(lib)


@pytest.mark.parametrize("kw,status,word", HEAD_REFUSALS + WINDOWS + CACHE_REFUSALS + PAGE_REFUSALS[:-1] + [
    (dict(T=65), BAD, "T=65"), (dict(B=-1), BAD, "B=-1"), (dict(slots=5), BAD, "slot_indices"), (dict(kc=None), BAD, "k_cache is NULL"),
    (dict(width=1 << 19, page=1024), UNSUP, "2^29"), (dict(width=600, window=9000, ws_bytes=64), SMALL, "kda_attn_window_tree")])
def test_tree_refuses(lib, kw, status, word):
    assert tree(lib, **kw) == status
    assert word in detail(lib)


@pytest.mark.parametrize("kw,status,word", [r for r in HEAD_REFUSALS if "dv" not in r[0]] + WINDOWS[1:] + CACHE_REFUSALS + PAGE_REFUSALS[:-1] + [
    (dict(dk=96), UNSUP, "dk=96"), (dict(T=-1), BAD, "T_tot"), (dict(T=1 << 29, R=1 << 29), UNSUP, "2^29"), (dict(N=0), BAD, "N=0"),
    (dict(N=2), BAD, "cu_seqlens"), (dict(R=7), BAD, "src_rows"), (dict(R=-1), BAD, "src_rows"), (dict(N=3, cu=FAKE + 9 * M), BAD, "slots=2"),
    (dict(N=1 << 23, cu=FAKE + (1 << 38), idx=FAKE + (1 << 39)), UNSUP, "workgroups"), (dict(q=None), BAD, "q is NULL"),
    (dict(lse=None), BAD, "lse is NULL"), (dict(w=None), BAD, "weights is NULL"), (dict(w=FAKE + 5 * M + 2), BAD, "aligned"),
    (dict(rows=FAKE + 30 * M + 2), BAD, "aligned"), (dict(width=1 << 19, page=1024), UNSUP, "2^29"),
    (dict(N=1, T=4096, R=4096, H=32, Hkv=8, width=64, page=64, pages=64, ws_bytes=0), SMALL, "kda_cache_weigh"),
    (dict(N=1, T=4096, R=4096, H=32, Hkv=8, width=64, page=64, pages=64, ws=None), BAD, "256-byte")])
def test_weigh_refuses(lib, kw, status, word):
    assert weigh(lib, **kw) == status
    assert word in detail(lib)


@pytest.mark.parametrize("kw,status,word", CACHE_REFUSALS + PAGE_REFUSALS[:-1] + [
    (dict(n=-1), BAD, "n=-1"), (dict(n=1 << 16), UNSUP, "entries"), (dict(keep=0), BAD, "keep=0"), (dict(keep=-3), BAD, "keep=-3"),
    (dict(first=-1), BAD, "first=-1"), (dict(recent=-1), BAD, "recent=-1"), (dict(first=17), BAD, "more than keep"),
    (dict(first=2**31 - 1, recent=2**31 - 1), BAD, "more than keep"), (dict(keep=1 << 29), UNSUP, "keep="), (dict(Hkv=0), BAD, "Hkv"),
    (dict(Hkv=1 << 15, dk=16, dv=16), UNSUP, "Hkv="), (dict(dk=48, dv=48), UNSUP, "dk=48"), (dict(x=3), BAD, "x_dtype"),
    (dict(width=1 << 19, page=1024), UNSUP, "2^29"), (dict(list=None), BAD, "slot_list is NULL"), (dict(refs=None), BAD, "refs is NULL"),
    (dict(w=None), BAD, "weights is NULL"), (dict(kept=FAKE + 20 * M + 2), BAD, "aligned"), (dict(ws_bytes=64), SMALL, "kda_cache_evict"),
    (dict(ws=None), BAD, "256-byte")])
def test_evict_refuses(lib, kw, status, word):
    assert evict(lib, **kw) == status
    assert word in detail(lib)


def test_calls_of_nothing(lib):
    assert prefill(lib, T=0, q=None, k=None, v=None, out=None, lse=None) == _lib.KDA_OK
    none = {n: None for n in ["q", "k", "v", "kc", "vc", "table", "lens", "out", "lse"]}
    assert tree(lib, B=0, slots=0, **none) == tree(lib, T=0, **none) == _lib.KDA_OK
    assert weigh(lib, T=0, R=0, q=None, lse=None, kc=None, table=None, lens=None, w=None, ws=None, ws_bytes=0) == _lib.KDA_OK
    assert evict(lib, n=0, list=None, kc=None, vc=None, table=None, lens=None, refs=None, w=None, ws=None, ws_bytes=0) == _lib.KDA_OK


WS = FAKE + (1 << 36)
BIG = dict(T=4096, R=4096, N=2, H=32, Hkv=8, width=64, page=64, pages=64, ws=WS)
# call, its sizes, its buffers that are read, its buffers that are written
CALLS = {
    "prefill": (prefill, dict(N=2), "q k v z cu", "out lse"),
    "backward": (backward, dict(N=2, ws=WS), "q k v z out lse dy cu", "gq gk gv gz ws"),
    "tree": (tree, dict(width=600, window=9000, ws=WS), "q k v mask z kc vc table lens idx", "out lse ws"),
    "weigh": (weigh, BIG, "q lse kc table lens cu rows idx", "w ws"),
    "evict": (evict, dict(ws=WS), "list", "kc vc table lens refs w kept status ws"),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_that_overlap(lib, name):
    call, sizes, read, written = CALLS[name]
    read, written = read.split(), written.split()
    at = {n: FAKE + (1 << 38) + i * (1 << 30) for i, n in enumerate(read + written)}
    at.update(sizes)
    pairs = [(w, o) for i, w in enumerate(written) for o in read + written[i + 1:]]
    for w, o in pairs:
        kw = dict(at)
        kw[w] = kw[o] = FAKE + (1 << 37)
        assert call(lib, **kw) == BAD, (w, o)
        assert "overlaps" in detail(lib), (w, o, detail(lib))


BF16, F32 = 1, 0


@pytest.mark.parametrize("H,Hkv,dk,dv,x", [(32, 8, 128, 128, BF16), (8, 1, 192, 128, F32), (64, 1, 64, 64, F32)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (500, 4), (1000, 10000), (1 << 20, 0)])
@pytest.mark.parametrize("B,T,context", [(256, 1, 4096), (20, 9, 8192), (1, 1, 64)])
def test_workspaces_of_trees(B, T, context, window, sinks, H, Hkv, dk, dv, x):
    most = kda.kda_attn_window_tree_max_workspace_bytes(B, T, H, Hkv, dk, dv, x, context, window, sinks)
    # (a context that the window holds just so, with a tile at its start and one at the sinks' end, is cut into the most parts)
    contexts = (0, context // 2, context - 1, context, min(context, window + sinks + 64))
    every = [kda.kda_attn_window_tree_workspace_bytes(b, t, H, Hkv, dk, dv, x, c, window, sinks)
             for b in range(B + 1) for t in range(T + 1) for c in contexts]
    assert max(every) == most
    if window >= context:
        assert most == kda.kda_attn_tree_max_workspace_bytes(B, T, H, Hkv, dk, dv, x, context)


@pytest.mark.parametrize("H,Hkv,dk,dv,x,gate", [(32, 8, 128, 128, BF16, 0), (8, 1, 192, 128, F32, 1), (2, 2, 16, 16, F32, 0), (64, 64, 64, 64, BF16, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (500, 4), (100, 1000), (1 << 20, 3)])
@pytest.mark.parametrize("T", [0, 1, 128, 1000, 5000, 40000])
def test_workspaces_of_gradients(T, window, sinks, H, Hkv, dk, dv, x, gate):
    most = kda.kda_attn_window_backward_max_workspace_bytes(T, H, Hkv, dk, dv, x, gate, window, sinks)
    need = lambda t, n: kda.kda_attn_window_backward_workspace_bytes(t, n, H, Hkv, dk, dv, x, gate, window, sinks)  # noqa: E731
    r = random.Random(T)
    some = range(T + 1) if T <= 1000 else sorted({T, T - 1, *(r.randint(0, T) for _ in range(1000)),
                                                  *(t for i in range(T // 128 + 1) for t in (128 * i, 128 * i + 127) if t <= T)})
    assert max(need(t, n) for t in some for n in (1, 2, 3, 17, 300)) <= most
    assert T == 0 or most > 0


@pytest.mark.parametrize("H,Hkv,dk,dv,x,gate", [(8, 2, 128, 128, F32, 0), (4, 1, 128, 128, BF16, 1), (32, 8, 16, 16, BF16, 0), (2, 2, 192, 128, F32, 1)])
@pytest.mark.parametrize("window", [1, 2, 33, 64, 65, 512, 513])
def test_first_tokens_past_the_sequences_end(window, H, Hkv, dk, dv, x, gate):
    """More first tokens than there are, and a window of more, are the call of
    just as many: it needs as much, also at the lengths at which first tokens begin
    to have queries that are worked on apart."""
    reach = window + 128
    need = lambda t, n, w, s: kda.kda_attn_window_backward_workspace_bytes(t, n, H, Hkv, dk, dv, x, gate, w, s)  # noqa: E731
    for T in (window - 1, window, window + 1, reach - 1, reach, reach + 1, 2 * reach):
        if T == 0:
            continue
        for sinks in (T - 1, T, T + 1, reach - 1, reach, reach + 1, T + 200, 2 ** 31 - 1):
            for N in (1, 2, 5):
                assert need(T, N, window, sinks) == need(T, N, min(window, T), min(sinks, T)), (T, N, sinks)
    for sinks in range(reach - 2, reach + 203, 3):
        for T in (reach - 1, reach, reach + 1, 2 * reach):
            most = kda.kda_attn_window_backward_max_workspace_bytes(T, H, Hkv, dk, dv, x, gate, window, sinks)
            assert max(need(t, n, window, sinks) for t in range(1, T + 1) for n in (1, 3)) <= most, (T, sinks)


def test_far_sums_of_more_threads_than_a_launch_takes():
    """2^32 threads and more are no launch: such a call, allowed by its limits, goes
    without sums of far queries, and the largest workspace holds the calls below."""
    window, sinks = 10000, 10000
    for H, Hkv, dk, dv in ((32, 32, 128, 128), (32, 32, 192, 128), (64, 32, 128, 128)):
        need = lambda t, n, s: kda.kda_attn_window_backward_workspace_bytes(t, n, H, Hkv, dk, dv, BF16, 0, window, s)  # noqa: E731
        reach, width = window + 128, Hkv * (dk + dv)
        most = (2**32 - 256) // (width // 4) // sinks  # sequences whose sums are few enough
        T = (2**28 - 1) // H
        assert T // reach > most
        for n in (most + 1, T // reach, 2 * T // reach):
            assert need(T, n, sinks) == need(T, n, 0), n
        sums = need(T, most, sinks) - need(T, most, 0)
        assert sums == 2 * most * sinks * width * 4
        top = kda.kda_attn_window_backward_max_workspace_bytes(T, H, Hkv, dk, dv, BF16, 0, window, sinks)
        assert max(need(t, n, sinks) for t in (T, T // 2, (most + 1) * reach - 1) for n in (1, most, most + 1, T // reach)) <= top


@pytest.mark.parametrize("H,Hkv", [(32, 8), (1, 1), (64, 1)])
def test_workspaces_of_weights(H, Hkv):
    """(1,024 + N) KiB hold every call of N sequences."""
    for N in (1, 2, 3, 7, 300, 1000, 1023, 1024, 1025, 5000):
        need = max(kda.kda_cache_weigh_workspace_bytes(T, N, H, Hkv) for T in (0, 1, N, 40 * N, 1 << 20))
        assert 0 < need <= (1024 + N) * 1024


def test_bad_sizes_need_nothing():
    good = (8, 8, 64, 64, BF16)
    assert kda.kda_attn_window_backward_workspace_bytes(100, 1, *good, 0, 0, 0) == 0
    assert kda.kda_attn_window_backward_workspace_bytes(1 << 29, 1, *good, 0, 5, 0) == 0
    assert kda.kda_attn_window_backward_max_workspace_bytes(100, *good, 0, 5, -1) == 0
    assert kda.kda_attn_window_tree_workspace_bytes(1, 1, *good, 1 << 29, 5, 0) == 0
    assert kda.kda_attn_window_tree_max_workspace_bytes(1, 1, *good, 1 << 16, 0, 0) == 0
    for bad in A.HEAD_REFUSALS[:1]:
        assert kda.kda_cache_weigh_workspace_bytes(8, 1, bad[0]["H"], 1) == 0
    assert kda.kda_cache_weigh_workspace_bytes(8, 0, 8, 8) == kda.kda_cache_weigh_workspace_bytes(8, 1, 8, 3) == 0
    assert kda.kda_cache_evict_workspace_bytes(1 << 16, 8) == kda.kda_cache_evict_workspace_bytes(4, 0) == 0
    assert kda.kda_cache_evict_workspace_bytes(4, 100) >= 4 * 100 * 4
