"""The rule that chooses the tiles of the products in 32 and 16 bits and of
their gradients (no GPU needed): it is plain host code, compiled here and asked
about sizes.  Every kernel that the library holds is one that it chooses, and
one that a GPU test runs (test_gpu_float_tiles.py has the sizes)."""

import os
import re
import subprocess

import pytest

from fp8_routed_expert_amd import build as lib_build
from tests.float_tiles import CASES, rows_of

MAIN = r"""
#include <cstdio>
#include "float_tile.hpp"
int main() {
  int mode, f32, E, rows, N, K;
  while (std::scanf("%d %d %d %d %d %d", &mode, &f32, &E, &rows, &N, &K) == 6) {
    const int splits = mode == moe::kWeightsGrad ? moe::weight_splits(E, rows, N, K) : 1;
    const moe::FloatTile t = moe::float_tile(mode, f32, E, rows, N, K, splits);
    std::printf("%d %d %d %d\n", t.rows, t.cols, t.ahead, splits);
  }
}
"""
PRODUCT, ROWS, WEIGHTS = 0, 1, 2
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("hipcc not installed")
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(MAIN)
    subprocess.run(["/opt/rocm/lib/llvm/bin/clang++", "-std=c++17", "-O1", f"-I{lib_build.CSRC}", str(d / "rule.cpp"),
                    "-o", str(d / "rule")], check=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "rule")], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def kernel(mode, dtype, N, K, tile):
    """The name's arguments of the kernel that a size takes."""
    rows, cols, ahead, _ = tile
    if rows == 16:
        return "skinny", dtype, cols // 16
    ragged = mode != WEIGHTS and (K if mode == PRODUCT else N) % (32 if dtype == F32 else 64) != 0
    return "tile", dtype, mode, rows, cols, ahead, ragged


def test_every_kernel_is_chosen_and_run(rule, tmp_path):
    # (the device code's functions, as the compiler's front end has them)
    ir = tmp_path / "gemm_float.ll"
    subprocess.run([lib_build.HIPCC, *lib_build.FLAGS, "--cuda-device-only", "-emit-llvm", "-O1", "-Xclang",
                    "-disable-llvm-passes", "-S", os.path.join(lib_build.CSRC, "gemm_float.hip"), "-o", str(ir)],
                   check=True, capture_output=True)
    names = re.findall(r"^define .*amdgpu_kernel void @(\w+)\(", ir.read_text(), re.M)
    names = subprocess.run(["c++filt", *names], check=True, capture_output=True, text=True).stdout
    built = set()
    for m in re.finditer(r"moe::float_tile_kernel<(.*?)>", names):
        t, mode, bm, bn, _, _, _, ahead, ragged = [x.strip() for x in m.group(1).split(",")]
        built.add(("tile", int(t), int(mode), int(bm), int(bn), int(ahead), ragged == "true"))
    for m in re.finditer(r"moe::skinny_float_kernel<(\d+), (\d+)>", names):
        built.add(("skinny", int(m.group(1)), int(m.group(2))))
    asked = [(mode, dtype, len(counts), rows_of(counts, align), N, K)
             for counts, align, N, K, dtypes in CASES for dtype in dtypes for mode in (PRODUCT, ROWS, WEIGHTS)]
    tiles = rule([(mode, int(dtype == F32), *size) for mode, dtype, *size in asked])
    run = {kernel(mode, dtype, N, K, t) for (mode, dtype, _, _, N, K), t in zip(asked, tiles)}
    assert built - run == set(), "built, and reached by no case"
    assert run - built == set() and len(built) == 56
    assert any(t[3] > 1 for t in tiles) and any(t[3] == 1 for t in tiles)


def test_few_rows_of_one_expert(rule):
    """Rows that fill less than half of a tile count as a tile, not as none: 256
    x 256 tiles of 4096 channels would leave 240 CUs idle."""
    rows = [49, 60, 100, 101, 176, 200, 228]
    for mode, N, K in ((PRODUCT, 4096, 7168), (PRODUCT, 7168, 2048), (ROWS, 7168, 2048), (ROWS, 4096, 7168)):
        tiles = rule([(mode, 0, 1, R, N, K) for R in rows])
        assert all(t[:2] == (128, 128) for t in tiles), (mode, N, K, tiles)


@pytest.mark.parametrize("E,N,K", [(4, 4096, 7168), (8, 2048, 7168), (8, 4096, 7168), (2, 8192, 2048)])
def test_buffers_of_128_rows_to_an_expert(rule, E, N, K):
    """They may be contiguous ones of few rows, or full segments: the product
    without tiles, which reads the weights once for every 16 rows, is for buffers
    that hold no more, or for too few channels for 64 x 64 tiles."""
    tiles = rule([(PRODUCT, 0, E, E * rows, N, K) for rows in (16, 128, 143)])
    assert all(t[:2] == (64, 64) for t in tiles[1:]) and tiles[0][0] == 16, tiles
    assert all(t[0] == 16 for t in rule([(PRODUCT, 0, 1, 128, 7168, 2048), (PRODUCT, 0, 1, 143, 4096, 7168)]))
