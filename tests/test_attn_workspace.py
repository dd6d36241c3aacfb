"""One workspace for every batch up to the largest: what a call needs does not
rise with its sizes, and the maximum over all smaller calls is asked for (CPU
only)."""

import random

import pytest

from gated_delta_rule_64_amd import kda

BF16, F32 = 1, 0


@pytest.mark.parametrize("H,Hkv,dk,dv,x", [(32, 8, 128, 128, BF16), (8, 1, 192, 128, F32), (4, 4, 16, 16, BF16), (64, 1, 64, 64, F32)])
@pytest.mark.parametrize("B,T,context", [(256, 1, 4096), (40, 9, 8192), (3, 64, 1 << 18), (1, 1, 64)])
def test_trees(B, T, context, H, Hkv, dk, dv, x):
    most = kda.kda_attn_tree_max_workspace_bytes(B, T, H, Hkv, dk, dv, x, context)
    every = [kda.kda_attn_tree_workspace_bytes(b, t, H, Hkv, dk, dv, x, c)
             for b in range(B + 1) for t in range(T + 1) for c in (0, context // 2, context - 1, context)]
    assert max(every) == most


def test_fewer_sequences_need_more():
    sizes = (1, 32, 8, 128, 128, BF16, 4096)
    assert kda.kda_attn_tree_workspace_bytes(127, *sizes) > kda.kda_attn_tree_workspace_bytes(256, *sizes)
    assert kda.kda_attn_tree_max_workspace_bytes(256, *sizes) >= kda.kda_attn_tree_workspace_bytes(127, *sizes)


@pytest.mark.parametrize("H,Hkv,dk,dv,x,gate", [(32, 8, 128, 128, BF16, 0), (32, 8, 128, 128, BF16, 1), (8, 1, 192, 128, F32, 1),
                                                (2, 2, 16, 16, F32, 0), (64, 64, 64, 64, BF16, 1), (1, 1, 32, 32, BF16, 0)])
@pytest.mark.parametrize("T", [0, 1, 127, 128, 1000, 5000, 16384, 200000])
def test_gradients(T, H, Hkv, dk, dv, x, gate):
    most = kda.kda_attn_backward_max_workspace_bytes(T, H, Hkv, dk, dv, x, gate)
    need = lambda t, n: kda.kda_attn_backward_workspace_bytes(t, n, H, Hkv, dk, dv, x, gate)  # noqa: E731
    r = random.Random(T)
    some = range(T + 1) if T <= 1000 else sorted({T, T - 1, *(r.randint(0, T) for _ in range(3000)),
                                                  *(t for i in range(T // 128 + 1) for t in (128 * i, 128 * i + 127) if t <= T)})
    every = [need(t, n) for t in some for n in (1, 2, 3, 17, 300)]
    assert max(every) == most


def test_fewer_tokens_need_more():
    sizes = (32, 8, 128, 128, BF16, 0)
    assert kda.kda_attn_backward_workspace_bytes(8192, 1, *sizes) > kda.kda_attn_backward_workspace_bytes(16384, 1, *sizes)
    assert kda.kda_attn_backward_max_workspace_bytes(16384, *sizes) >= kda.kda_attn_backward_workspace_bytes(8192, 1, *sizes)


HEADS = [(8, 3, 64, 64, BF16), (8, 8, 96, 96, BF16), (8, 8, 64, 64, 5)]


def test_bad_sizes_need_nothing():
    tree, gradients = kda.kda_attn_tree_max_workspace_bytes, kda.kda_attn_backward_max_workspace_bytes
    good = (8, 8, 64, 64, BF16)
    assert tree(4, 4, *good, 1 << 16) > 0 and gradients(100, *good, 0) > 0
    assert tree(-1, 4, *good, 1 << 16) == tree(4, 65, *good, 1 << 16) == tree(4, 4, *good, -1) == gradients(-1, *good, 0) == 0
    for bad in HEADS:
        assert tree(4, 4, *bad, 1 << 16) == 0 and gradients(100, *bad, 0) == 0
