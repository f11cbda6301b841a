"""The tile loads that the product kernels share compile without warnings (no
GPU needed): each is instantiated hundreds of times, and a warning that matters
must not drown in theirs."""

import os
import subprocess

import pytest

from fp8_routed_expert_amd import build as lib_build

KERNEL = r"""
#include "gemm_tiles.hpp"
__global__ void loads(const uint8_t* p, uint8_t* out) {
  __shared__ __attribute__((aligned(1024))) uint8_t s[3 * 1024];
  const moe::v4i r = moe::make_rsrc(p, 4096);
  moe::dma16(r, s, threadIdx.x * 16);
  moe::dma16_add(r, s + 1024, threadIdx.x * 16, 1024);
  moe::dma16_split(r, s + 2048, threadIdx.x * 16, 16, 2048);
  moe::wait_vm<0>();
  moe::lds_barrier();
  out[threadIdx.x] = s[threadIdx.x] + s[threadIdx.x + 1024] + s[threadIdx.x + 2048];
}
"""


def test_tile_loads_compile_without_warnings(tmp_path):
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("hipcc not installed")
    src = tmp_path / "loads.hip"
    src.write_text(KERNEL)
    # (device code alone: the host pass does not know the device target's features)
    r = subprocess.run([lib_build.HIPCC, *lib_build.FLAGS, "--cuda-device-only", "-S", str(src), "-o", os.devnull],
                       check=True, capture_output=True, text=True)
    found = [line for line in r.stderr.split("\n") if "warning:" in line]
    assert not found, (len(found), found[:3])
