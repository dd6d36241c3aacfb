"""Pools of several scan steps (more than 8,192 pages) whose pages move."""

import random

import pytest
import torch

from test_gpu_cache import Device, Model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from gated_delta_rule_64_amd import kda
    return kda


@pytest.mark.parametrize("pages,used", [(8192, 5000), (8193, 8000), (8193, 1), (20000, 11000), (20000, 19990), (30011, 300)])
def test_compact(K, pages, used):
    """Holes and pages in use on both sides of a scan step's end; every third
    page shared by two slots."""
    r = random.Random(pages + used)
    m = Model(pages, 16, 40, -(-pages // 30))
    live = r.sample(range(pages), used)
    for i, p in enumerate(live):
        m.table[i % 30, i // 30] = p
        m.refs[p] = 1
        if i % 3 == 0 and i // 30 < m.table.shape[1]:
            m.table[30 + i % 10, i // 30] = p
    m.refs[:] = 0
    for p in m.table[m.table >= 0]:
        m.refs[p] += 1
    d = Device(m, 1, 16, 16)
    k0, v0 = d.kc.clone(), d.vc.clone()
    print("compact", pages, used, flush=True)
    got = K.kda_cache_compact(d.kc, d.vc, d.table, d.refs)
    want, moves = m.compact()
    assert got.tolist() == [want] == [used]
    d.same(m)
    a, b = (torch.tensor([x[i] for x in moves], dtype=torch.long, device="cuda") for i in (0, 1))
    k0[b], v0[b] = k0[a], v0[a]
    assert torch.equal(d.kc, k0) and torch.equal(d.vc, v0)
