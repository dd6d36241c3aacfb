"""The build refuses attention and cache kernels that keep registers in memory
(CPU only: compiles, runs nothing)."""

import os

import pytest

from gated_delta_rule_64_amd import build

# sums of as many values as `n`, all alive at once, for 1,024 threads a
# workgroup: up to 128 registers a lane
KERNEL = """
#include <hip/hip_runtime.h>
extern "C" __global__ __launch_bounds__(1024) void sums(const float* x, float* y) {
    float r[%d];
#pragma unroll
    for (int i = 0; i < %d; ++i) r[i] = x[i * 1024 + threadIdx.x];
    for (int k = 0; k < y[0]; ++k) {
#pragma unroll
        for (int i = 0; i < %d; ++i) r[i] = r[i] * r[(i + 7) %% %d] + x[k];
    }
#pragma unroll
    for (int i = 0; i < %d; ++i) y[i * 1024 + threadIdx.x] = r[i];
}
"""


def _compile(tmp_path, monkeypatch, name, n):
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    src = tmp_path / name
    src.write_text(KERNEL % ((n,) * 5))
    return build._compile(str(src))


@pytest.mark.parametrize("name", ["kda_attn_x.hip", "kda_cache.hip"])
def test_a_spilling_kernel_is_refused(tmp_path, monkeypatch, name):
    with pytest.raises(RuntimeError, match="sums: [1-9]"):
        _compile(tmp_path, monkeypatch, name, 200)
    assert not os.path.exists(tmp_path / (name + ".o"))


def test_others_are_built(tmp_path, monkeypatch):
    assert os.path.exists(_compile(tmp_path, monkeypatch, "kda_attn_x.hip", 20))
    assert os.path.exists(_compile(tmp_path, monkeypatch, "kda_other.hip", 200))


def test_the_sources_are_watched():
    names = [n for n in os.listdir(build.CSRC) if n.endswith(".hip") and n.startswith(build.NO_SPILL)]
    assert {"kda_attn_prefill.hip", "kda_attn_backward.hip", "kda_attn_tree.hip", "kda_cache.hip"} <= set(names)
