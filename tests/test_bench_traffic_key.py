"""The stored counter record that bench.py reports belongs to one build of the
gate/up kernel: its key covers every source the kernel is compiled from (no GPU
needed)."""

import json
import os
import re
import shutil

import bench
from fp8_routed_expert_amd import build as lib_build


def included(path, seen):
    """The repository's files that path includes, itself first."""
    seen.append(path)
    for name in re.findall(r'#include "(\w+\.hpp)"', open(path).read()):
        p = os.path.join(os.path.dirname(path), name)
        if p not in seen:
            included(p, seen)
    return seen


def test_key_covers_the_kernel_and_its_headers(tmp_path, monkeypatch):
    names = [os.path.basename(p) for p in included(os.path.join(lib_build.CSRC, "gemm.hip"), [])]
    assert "gemm_tiles.hpp" in names
    for n in names:
        shutil.copy(os.path.join(lib_build.CSRC, n), tmp_path / n)
    monkeypatch.setattr(bench, "GEMM_SRC", str(tmp_path / "gemm.hip"))
    key = bench.gemm_source_hash()
    for n in names:
        text = (tmp_path / n).read_bytes()
        (tmp_path / n).write_bytes(text + b"\n")
        assert bench.gemm_source_hash() != key, n
        (tmp_path / n).write_bytes(text)
    assert bench.gemm_source_hash() == key


def test_stored_record_is_of_these_sources():
    rec = json.load(open(bench.TRAFFIC_FILE))
    assert bench.stored_traffic(rec["launch"]) == rec["hbm_bytes_per_launch"] > 0
