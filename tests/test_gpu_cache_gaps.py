"""Slots that lack a page in front of their length."""

import math

import pytest
import torch

from test_gpu_cache import Device, Model, _ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


def _gap():
    """Slot 0: 40 tokens, the second and the last, partly filled page gone."""
    m = Model(12, 16, 4, 6)
    m.table[0, 0], m.refs[7], m.lens[0] = 7, 1, 40
    return m


def test_a_partly_filled_page_that_is_gone(K):
    """A fork keeps the gap, a reserve fills only what is behind the length, an
    append writes only what has a page, and no row attends what is gone."""
    m = _gap()
    d = Device(m, 1, 16, 16)
    d.kc.fill_(math.nan)
    d.vc.fill_(math.nan)
    d.kc[7], d.vc[7] = torch.randn(1, 16, 16, device="cuda"), torch.randn(1, 16, 16, device="cuda")
    got = K.kda_cache_fork(_ints([0]), _ints([2]), d.kc, d.vc, d.table, d.lens, d.refs)
    assert got.tolist() == m.fork([0], [2])[0] == [0]
    d.same(m)
    assert m.table[2, :4].tolist() == [7, -1, -1, -1]
    for slot in (0, 2):
        got = K.kda_cache_reserve(_ints([slot]), _ints([70]), 16, d.table, d.lens, d.refs)
        assert got.tolist() == m.reserve([slot], [70]) == [0]
    d.same(m)
    assert m.table[2, 1:3].tolist() == [-1, -1] and (m.table[2, 3:5] >= 0).all()
    k, v = torch.randn(30, 1, 16, device="cuda"), torch.randn(30, 1, 16, device="cuda")
    k0, v0 = d.kc.clone(), d.vc.clone()
    K.kda_cache_append(k, v, d.kc, d.vc, d.table, d.lens, slot_indices=_ints([2]))
    for i in range(8, 30):  # positions 48 and up have pages
        page = int(m.table[2, (40 + i) // 16])
        k0[page, :, (40 + i) % 16], v0[page, :, (40 + i) % 16] = k[i], v[i]
    assert torch.equal(d.kc.nan_to_num(9), k0.nan_to_num(9)) and torch.equal(d.vc.nan_to_num(9), v0.nan_to_num(9))
    d.lens[2] = 70
    q, kn, vn = (torch.randn(1, 1, 1, 16, device="cuda") for _ in range(3))
    out, lse = K.kda_attn_tree(q, kn, vn, d.kc, d.vc, d.table, d.lens, slot_indices=_ints([2]))
    keys = torch.cat([d.kc[7, 0], k[8:, 0], kn[0, 0]]).double()
    vals = torch.cat([d.vc[7, 0], v[8:, 0], vn[0, 0]]).double()
    s = (keys @ q[0, 0, 0].double()) * 0.25
    # 39 tokens in fp32: the sums are off by less than 2^-18 of values of a few units
    assert float((out[0, 0, 0].double() - torch.softmax(s, 0) @ vals).abs().max()) < 2.0 ** -16
    assert abs(float(lse[0, 0, 0]) - float(torch.logsumexp(s, 0))) < 2.0 ** -16
