"""Every buffer that an attention or cache call writes is kept apart from every
other buffer of the call: each pair is laid over each other once and refused
on the host (CPU only)."""

import pytest

import test_attn_abi as A
from gated_delta_rule_64_amd import _lib

M, FAKE = A.M, A.FAKE


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def _pages(which):
    return lambda lib, **kw: A.pages_call(lib, which, **kw)


WS = FAKE + (1 << 36)
# call, its sizes, its buffers that are read, its buffers that are written
CALLS = {
    "prefill": (A.prefill, dict(N=2), "q k v z cu", "out lse"),
    "backward": (A.backward, dict(N=2, ws=WS), "q k v z out lse dy cu", "gq gk gv gz ws"),
    "tree": (A.tree, dict(width=600, ws=WS), "q k v mask z kc vc table lens idx", "out lse ws"),
    "append": (A.append, dict(N=2), "k v table lens cu rows idx", "kc vc"),
    "free": (_pages("free"), dict(), "a", "table lens refs"),
    "fork": (_pages("fork"), dict(ws=WS), "a b", "kc vc table lens refs status ws"),
    "reserve": (_pages("reserve"), dict(ws=WS), "a b lens", "table refs status ws"),
    "compact": (_pages("compact"), dict(ws=WS), "", "kc vc table refs live ws"),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_that_overlap(lib, name):
    call, sizes, read, written = CALLS[name]
    read, written = read.split(), written.split()
    at = {n: FAKE + (40 + i) * M for i, n in enumerate(read + written)}
    at.update(sizes)
    pairs = [(w, o) for i, w in enumerate(written) for o in read + written[i + 1:]]
    assert pairs
    for w, o in pairs:
        kw = dict(at)
        kw[w] = kw[o] = FAKE + (1 << 37)
        assert call(lib, **kw) == A.BAD, (w, o)
        assert "overlaps" in A.detail(lib), (w, o, A.detail(lib))
