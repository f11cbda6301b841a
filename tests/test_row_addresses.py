"""Sizes that leave 31 or 32 bits, on the host (no GPU needed): the address of a
row's chunk, which the activation's kernels form with a helper that is compiled
for the host here and compared with exact integers, and the threads of a launch."""

import ctypes
import os
import subprocess

import pytest

from fp8_routed_expert_amd import _lib
from fp8_routed_expert_amd import build as lib_build

MAIN = r"""
#include <cstdio>
#include "row_chunks.hpp"
int main() {
  const int rows[] = {0, 1, (1 << 29) - 1, 1 << 29, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, 0x7fff0000 - 1};
  const size_t bytes[] = {16, 32, 4096, (size_t)1 << 30, (size_t)1 << 31};
  const unsigned chunks[] = {0, 1, 255, 0x7ffffff};
  for (int m : rows)
    for (size_t b : bytes)
      for (unsigned c : chunks) std::printf("%d %zu %u %zu\n", m, b, c, moe::chunk_at(m, b, c));
}
"""


def test_chunk_addresses(tmp_path):
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("hipcc not installed")
    src, exe = tmp_path / "rows.hip", tmp_path / "rows"
    src.write_text(MAIN)
    r = subprocess.run([lib_build.HIPCC, *lib_build.FLAGS, "--offload-host-only", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    lines = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert len(lines) == 8 * 5 * 4
    for m, b, c, at in lines:
        assert at == m * b + 16 * c, (m, b, c)


def test_norm_columns_of_one_launch():
    """The columns of the norm's weight and bias gradients are joined by one
    launch, which holds 2^32 threads, 256 for 32 columns of both."""
    P, most = ctypes.c_void_p(4096), (2 ** 32 // 256 - 1) * 32 // 2
    f = _lib.load().moe_layer_norm_grad
    for T in (0, 1, 4):
        for dw, db in ((P, P), (P, None), (None, P)):
            assert f(P, P, 1, T, most + 1, P, 0, P, P, P, dw, db, P, 1 << 50, None) == 2, (T, dw, db)
