"""The address of a row's chunk, in 64 bits for every row number that a call
takes, on the host (no GPU needed): the helper that the activation's kernels
form their addresses with is compiled for the host and compared with exact
integers."""

import os
import subprocess

import pytest

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
