"""The attention and cache calls refuse bad arguments on the host, before any
device work (CPU only)."""

import ctypes

import pytest

from gated_delta_rule_64_amd import _lib

P = ctypes.c_void_p
FAKE = 1 << 40  # an aligned, never-dereferenced address
M = 1 << 24
BAD, UNSUP, SMALL = _lib.KDA_ERR_INVALID_ARGUMENT, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def _at(names):
    return {n: FAKE + i * M for i, n in enumerate(names)}


def detail(lib):
    return lib.kda_last_error_detail().decode()


def prefill(lib, **kw):
    a = dict(T=64, H=4, Hkv=2, dk=64, dv=64, cu=None, N=1, x=1, scale=0.125, z=None, **_at(["q", "k", "v", "out", "lse"]))
    a.update(kw)
    return lib.kda_attn_prefill(a["T"], a["H"], a["Hkv"], a["dk"], a["dv"], P(a["cu"]), a["N"], a["x"], a["scale"], P(a["q"]),
                                P(a["k"]), P(a["v"]), P(a["z"]), P(a["out"]), P(a["lse"]), None)


HEAD_REFUSALS = [(dict(H=0), BAD, "H=0"), (dict(H=65536), BAD, "H="), (dict(Hkv=3), BAD, "does not divide"),
                 (dict(Hkv=0), BAD, "Hkv"), (dict(dk=96, dv=96), UNSUP, "dk=96"), (dict(dk=64, dv=128), UNSUP, "dv=128"),
                 (dict(x=2), BAD, "x_dtype"), (dict(scale=0.0), BAD, "scale"), (dict(scale=-1.0), BAD, "scale"),
                 (dict(scale=float("nan")), BAD, "scale"), (dict(scale=float("inf")), BAD, "scale"),
                 (dict(H=65534, Hkv=1, dk=192, dv=128, x=0), UNSUP, "2^25")]


@pytest.mark.parametrize("kw,status,word", HEAD_REFUSALS + [
    (dict(T=-1), BAD, "T_tot"), (dict(T=2**31), BAD, "T_tot"), (dict(N=0), BAD, "N=0"), (dict(N=2), BAD, "cu_seqlens"),
    (dict(q=None), BAD, "q is NULL"), (dict(v=FAKE + 2 * M + 8), BAD, "aligned"), (dict(out=FAKE + 64), BAD, "overlaps"),
    (dict(lse=FAKE + 3 * M + 16), BAD, "overlaps"), (dict(cu=FAKE + 9 * M + 2, N=2), BAD, "aligned"),
    (dict(lse=FAKE + 4 * M + 2), BAD, "aligned"), (dict(T=2**31 - 1, H=4096, Hkv=1), UNSUP, "workgroups")])
def test_prefill_refuses(lib, kw, status, word):
    assert prefill(lib, **kw) == status
    assert word in detail(lib)


def test_prefill_of_nothing(lib):
    assert prefill(lib, T=0, q=None, k=None, v=None, out=None, lse=None) == _lib.KDA_OK


def backward(lib, **kw):
    a = dict(T=64, H=4, Hkv=2, dk=64, dv=64, cu=None, N=1, x=1, scale=0.125, z=None, gz=None, ws=FAKE + (1 << 36), ws_bytes=None,
             **_at(["q", "k", "v", "out", "lse", "dy", "gq", "gk", "gv"]))
    a.update(kw)
    if a["ws_bytes"] is None:
        a["ws_bytes"] = lib.kda_attn_backward_workspace_bytes(a["T"], a["N"], a["H"], a["Hkv"], a["dk"], a["dv"], a["x"],
                                                              a["z"] is not None)
    return lib.kda_attn_prefill_backward(a["T"], a["H"], a["Hkv"], a["dk"], a["dv"], P(a["cu"]), a["N"], a["x"], a["scale"],
                                         P(a["q"]), P(a["k"]), P(a["v"]), P(a["z"]), P(a["out"]), P(a["lse"]), P(a["dy"]),
                                         P(a["gq"]), P(a["gk"]), P(a["gv"]), P(a["gz"]), P(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status,word", HEAD_REFUSALS + [
    (dict(z=FAKE + 20 * M), BAD, "grad_out_gate"), (dict(gz=FAKE + 20 * M), BAD, "grad_out_gate"),
    (dict(lse=None), BAD, "lse is NULL"), (dict(dy=None), BAD, "dy is NULL"), (dict(gk=FAKE + 6 * M + 32), BAD, "overlaps"),
    (dict(ws_bytes=8), SMALL, "workspace_bytes"), (dict(ws=FAKE + (1 << 36) + 16), BAD, "256-byte"),
    (dict(gq=FAKE), BAD, "overlaps"), (dict(ws=FAKE), BAD, "overlaps")])
def test_backward_refuses(lib, kw, status, word):
    assert backward(lib, **kw) == status
    assert word in detail(lib)


def test_backward_workspace(lib):
    w = lib.kda_attn_backward_workspace_bytes
    assert w(0, 1, 4, 2, 64, 64, 1, 1) == 0  # no tokens: nothing is needed
    assert w(64, 1, 4, 2, 64, 64, 1, 1) > w(64, 1, 4, 2, 64, 64, 1, 0) >= 64 * 4 * 4
    assert w(64, 1, 4, 3, 64, 64, 1, 0) == 0 and w(64, 1, 4, 2, 64, 32, 1, 0) == 0 and w(-1, 1, 4, 2, 64, 64, 1, 0) == 0


def tree(lib, **kw):
    a = dict(B=2, T=4, H=4, Hkv=2, dk=64, dv=64, x=1, scale=0.125, mask=None, z=None, pages=10, page=16, slots=2, width=4, idx=None,
             ws=FAKE + (1 << 36), ws_bytes=None, **_at(["q", "k", "v", "kc", "vc", "table", "lens", "out", "lse"]))
    a.update(kw)
    if a["ws_bytes"] is None:
        a["ws_bytes"] = 1 << 30
    return lib.kda_attn_tree(a["B"], a["T"], a["H"], a["Hkv"], a["dk"], a["dv"], a["x"], a["scale"], P(a["q"]), P(a["k"]), P(a["v"]),
                             P(a["mask"]), P(a["z"]), P(a["kc"]), P(a["vc"]), a["pages"], a["page"], P(a["table"]), a["slots"],
                             a["width"], P(a["lens"]), P(a["idx"]), P(a["out"]), P(a["lse"]), P(a["ws"]), a["ws_bytes"], None)


CACHE_REFUSALS = [(dict(pages=0), BAD, "num_pages"), (dict(pages=1 << 24), BAD, "num_pages"), (dict(slots=-1), BAD, "slots"),
                  (dict(width=0), BAD, "max_pages"), (dict(width=1 << 23), BAD, "max_pages")]
PAGE_REFUSALS = [(dict(page=24), UNSUP, "page_size"), (dict(page=8), UNSUP, "page_size"), (dict(page=2048), UNSUP, "page_size"),
                 (dict(page=0), UNSUP, "page_size"), (dict(page=-16), UNSUP, "page_size"),
                 (dict(width=(1 << 23) - 1, page=1024), UNSUP, "2^31")]


@pytest.mark.parametrize("kw,status,word", HEAD_REFUSALS + CACHE_REFUSALS + PAGE_REFUSALS + [
    (dict(T=65), BAD, "T=65"), (dict(T=-1), BAD, "T=-1"), (dict(B=-1), BAD, "B=-1"), (dict(slots=5), BAD, "slot_indices"),
    (dict(mask=FAKE + 20 * M + 4), BAD, "aligned"), (dict(kc=None), BAD, "k_cache is NULL"), (dict(table=None), BAD, "page_table"),
    (dict(idx=FAKE + 21 * M + 1), BAD, "aligned"), (dict(out=FAKE + 3 * M + 512), BAD, "overlaps"),
    (dict(width=600, ws_bytes=64), SMALL, "workspace_bytes"), (dict(width=600, ws=None), BAD, "256-byte"),
    (dict(B=1 << 22, T=64, H=16, Hkv=1, slots=1 << 22), UNSUP, "2^30")])
def test_tree_refuses(lib, kw, status, word):
    assert tree(lib, **kw) == status
    assert word in detail(lib)


def test_tree_of_nothing(lib):
    none = {n: None for n in ["q", "k", "v", "kc", "vc", "table", "lens", "out", "lse"]}
    assert tree(lib, B=0, slots=0, **none) == _lib.KDA_OK
    assert tree(lib, T=0, **none) == _lib.KDA_OK


def test_tree_workspace(lib):
    w = lib.kda_attn_tree_workspace_bytes
    assert w(256, 1, 32, 8, 128, 128, 1, 4096) == 0  # enough rows: no split
    assert w(1, 1, 32, 8, 128, 128, 1, 1 << 18) > 0
    assert w(1, 65, 32, 8, 128, 128, 1, 4096) == 0 and w(1, 1, 32, 8, 128, 128, 9, 4096) == 0


def append(lib, **kw):
    a = dict(T=8, N=1, cu=None, R=8, rows=None, Hkv=2, dk=64, dv=64, x=1, pages=10, page=16, slots=2, width=4, idx=None,
             **_at(["k", "v", "kc", "vc", "table", "lens"]))
    a.update(kw)
    return lib.kda_cache_append(a["T"], a["N"], P(a["cu"]), a["R"], P(a["rows"]), a["Hkv"], a["dk"], a["dv"], a["x"], P(a["k"]),
                                P(a["v"]), P(a["kc"]), P(a["vc"]), a["pages"], a["page"], P(a["table"]), a["slots"], a["width"],
                                P(a["lens"]), P(a["idx"]), None)


@pytest.mark.parametrize("kw,status,word", CACHE_REFUSALS[:2] + PAGE_REFUSALS + [
    (dict(T=-1), BAD, "T_tot"), (dict(N=0), BAD, "N=0"), (dict(N=2), BAD, "cu_seqlens"), (dict(R=7), BAD, "src_rows"),
    (dict(R=-1), BAD, "src_rows"), (dict(N=3, cu=FAKE + 9 * M), BAD, "slots=2"), (dict(k=FAKE + 2 * M), BAD, "overlaps"),
    (dict(vc=FAKE + 2 * M + 1024), BAD, "overlaps"), (dict(rows=FAKE + 30 * M + 2), BAD, "aligned"), (dict(x=3), BAD, "x_dtype"),
    (dict(Hkv=0), BAD, "Hkv"), (dict(dk=48, dv=48), UNSUP, "dk=48"), (dict(lens=None), BAD, "lens is NULL")])
def test_append_refuses(lib, kw, status, word):
    assert append(lib, **kw) == status
    assert word in detail(lib)


def pages_call(lib, which, **kw):
    a = dict(n=3, Hkv=2, dk=64, dv=64, x=1, pages=10, page=16, slots=2, width=4, ws=FAKE + (1 << 36), ws_bytes=1 << 20, status=None,
             **_at(["kc", "vc", "table", "lens", "refs", "a", "b", "live"]))
    a.update(kw)
    heads, pools = [a["Hkv"], a["dk"], a["dv"], a["x"]], [P(a["kc"]), P(a["vc"]), a["pages"], a["page"]]
    table, work = [P(a["table"]), a["slots"], a["width"]], [P(a["ws"]), a["ws_bytes"], None]
    if which == "free":
        return lib.kda_cache_free(a["n"], P(a["a"]), a["pages"], *table, P(a["lens"]), P(a["refs"]), None)
    if which == "fork":
        return lib.kda_cache_fork(a["n"], P(a["a"]), P(a["b"]), *heads, *pools, *table, P(a["lens"]), P(a["refs"]), P(a["status"]),
                                  *work)
    if which == "reserve":
        return lib.kda_cache_reserve(a["n"], P(a["a"]), P(a["b"]), a["pages"], a["page"], *table, P(a["lens"]), P(a["refs"]),
                                     P(a["status"]), *work)
    return lib.kda_cache_compact(*heads, *pools, *table, P(a["refs"]), P(a["live"]), *work)


@pytest.mark.parametrize("which", ["free", "fork", "reserve", "compact"])
@pytest.mark.parametrize("kw,status,word", CACHE_REFUSALS + [
    (dict(refs=None), BAD, "refs is NULL"), (dict(table=FAKE + 2 * M + 2), BAD, "aligned"), (dict(refs=FAKE + 2 * M + 8), BAD, "overlaps")])
def test_page_calls_refuse(lib, which, kw, status, word):
    assert pages_call(lib, which, **kw) == status
    assert word in detail(lib)


@pytest.mark.parametrize("which", ["fork", "reserve", "compact"])
@pytest.mark.parametrize("kw,status,word", PAGE_REFUSALS + [
    (dict(ws_bytes=16), SMALL, "workspace_bytes"), (dict(ws=None), BAD, "256-byte"), (dict(ws=FAKE + 2 * M), BAD, "overlaps")])
def test_page_calls_with_workspace_refuse(lib, which, kw, status, word):
    assert pages_call(lib, which, **kw) == status
    assert word in detail(lib)


@pytest.mark.parametrize("which", ["free", "fork", "reserve"])
def test_page_calls_of_nothing(lib, which):
    assert pages_call(lib, which, n=-1) == BAD
    assert pages_call(lib, which, n=0, table=None, lens=None, refs=None, a=None, b=None, kc=None, vc=None, ws=None, ws_bytes=0) == _lib.KDA_OK


def test_lists_refused(lib):
    assert pages_call(lib, "fork", a=None) == BAD and "src is NULL" in detail(lib)
    assert pages_call(lib, "fork", status=FAKE + 3 * M) == BAD and "overlaps" in detail(lib)
    assert pages_call(lib, "reserve", b=FAKE + 6 * M + 1) == BAD and "new_lens" in detail(lib)
    assert pages_call(lib, "compact", live=None) == BAD and "live is NULL" in detail(lib)


@pytest.mark.parametrize("kw,word", [(dict(row_bytes=24), "multiple of 16"), (dict(row_bytes=-16), "multiple of 16"), (dict(rows=-1), "rows"),
                                     (dict(n=-2), "n=-2"), (dict(pool=None), "pool is NULL"), (dict(pool=FAKE + 8), "aligned"),
                                     (dict(src=FAKE + 32), "overlaps"), (dict(row_bytes=1 << 50), "out of range")])
def test_copy_refuses(lib, kw, word):
    a = dict(pool=FAKE, row_bytes=64, rows=100, src=FAKE + M, dst=FAKE + 2 * M, n=3)
    a.update(kw)
    assert lib.kda_cache_copy(P(a["pool"]), a["row_bytes"], a["rows"], P(a["src"]), P(a["dst"]), a["n"], None) == BAD
    assert word in detail(lib)


def test_workspaces_hold_every_call(lib):
    w = lib.kda_cache_workspace_bytes
    assert w(10, 2, 3) >= 256 and w(0, 2, 3) == 0 and w(10, -1, 3) == 0 and w(10, 2, -1) == 0
    assert w(1000, 2, 0) >= 3 * 4000


# A launch holds fewer than 2^32 threads, so 2^24 workgroups of 256 are too
# many: each call just past its limit.  (Below the limit a call would launch.)
TOO_MANY = 1 << 24


@pytest.mark.parametrize("call,kw", [
    (prefill, dict(T=1 << 28, H=8, Hkv=1, dk=16, dv=16)),  # 2^21 tiles and one more of 8 heads
    (prefill, dict(T=TOO_MANY, N=TOO_MANY, H=1, Hkv=1, dk=16, dv=16, cu=FAKE + (1 << 37))),
    (backward, dict(T=1 << 26, H=16, Hkv=1, dk=16, dv=16)),  # tiles of both kinds of gradients
    (backward, dict(T=1 << 25, H=8, Hkv=1, dk=16, dv=16)),  # 2^28 rows, 16 a workgroup
    (tree, dict(B=TOO_MANY - 8, slots=TOO_MANY - 8, T=33, H=1, Hkv=1, dk=16, dv=16)),
    (tree, dict(B=TOO_MANY, slots=TOO_MANY, T=1, H=1, Hkv=1, dk=16, dv=16)),
    (append, dict(T=1 << 27, R=1 << 27))])
def test_launches_past_the_grid_are_refused(lib, call, kw):
    assert call(lib, **kw) == UNSUP
    assert "workgroups" in detail(lib)


@pytest.mark.parametrize("which", ["free", "fork", "reserve"])
def test_entry_lists_past_the_grid_are_refused(lib, which):
    assert pages_call(lib, which, n=TOO_MANY) == UNSUP
    assert "workgroups" in detail(lib)
