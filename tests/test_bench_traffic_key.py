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


def test_record_of_other_sources_is_not_used(tmp_path, monkeypatch):
    rec = json.load(open(bench.TRAFFIC_FILE))
    assert {"gemm_source_sha", "launch", "hbm_bytes_per_launch"} <= set(rec)
    path = tmp_path / "record.json"
    monkeypatch.setattr(bench, "TRAFFIC_FILE", str(path))
    assert bench.stored_traffic(rec["launch"]) is None
    for key, want in ((bench.gemm_source_hash(), rec["hbm_bytes_per_launch"]), ("0" * 16, None)):
        path.write_text(json.dumps({**rec, "gemm_source_sha": key}))
        assert bench.stored_traffic(rec["launch"]) == want
        assert bench.stored_traffic("another launch") is None
