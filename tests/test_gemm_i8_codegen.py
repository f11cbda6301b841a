"""Code-generation invariants of the 8-bit integer products (no GPU needed):
from the first tile load to the last multiplication the compiler waits for no
vector memory (a wait would serialise loads and multiplications), M0 has no
user but the tile loads, and nothing spills."""

import os
import re
import subprocess

import pytest

from fp8_routed_expert_amd import build as lib_build

SRC = os.path.join(lib_build.CSRC, "gemm_i8.hip")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("hipcc not installed")
    out = tmp_path_factory.mktemp("gemm_i8_asm") / "gemm_i8.s"
    subprocess.run([lib_build.HIPCC, *lib_build.FLAGS, "--cuda-device-only", "-S", SRC, "-o",
                    str(out)], check=True, capture_output=True)
    res, name, in_asm = {}, None, False
    for line in out.read_text().split("\n"):
        m = re.match(r"^(_ZN3moe\w*i8\w*kernel\w*):", line)
        if m:
            name, in_asm = m.group(1), False
            res[name] = []
        elif name and line.startswith(".Lfunc_end"):
            name = None
        elif name:
            s = line.strip()
            if s.startswith(";;#ASM"):
                in_asm = s.startswith(";;#ASMSTART")
            elif s and s[0] not in ";.":
                res[name].append((s, in_asm))
    assert len(res) >= 8
    return res


def test_no_compiler_waits_in_the_pipeline(kernels):
    tiled = 0
    for name, body in kernels.items():
        loads = [i for i, (s, _) in enumerate(body) if re.match(r"buffer_load_dwordx4 .* lds$", s)]
        if not loads:
            continue
        tiled += 1
        last = max(i for i, (s, _) in enumerate(body) if s.startswith("v_mfma"))
        extra = [s for s, in_asm in body[loads[0]:last]
                 if s.startswith("s_waitcnt") and "vmcnt" in s and not in_asm]
        assert not extra, (name, extra[:3])
    assert tiled >= 8


def test_m0_and_spills(kernels):
    for name, body in kernels.items():
        assert not [s for s, in_asm in body if re.search(r"\bm0\b", s) and not in_asm], name
        assert not [s for s, _ in body if s.startswith("scratch_")], name


def test_walking_kernels_count_their_accesses(kernels):
    """The kernels that walk several tiles wait for a tile's loads by counting
    what was issued behind them: 16 stores of a tile in each 16-bit type, and
    the scales' 8 + 4 loads, before the walk and within it (gathered or ragged:
    8, the channels' 4 once, after the K loop); none under a branch of its
    own."""
    walking = {n: b for n, b in kernels.items() if "Li256ELi256ELi128ELi64ELi2ELi0ELb1E" in n}
    assert len(walking) == 3
    for name, body in walking.items():
        ins = [s for s, _ in body]
        stores = [i for i, s in enumerate(ins) if s.startswith("buffer_store_dwordx4")]
        loads = [i for i, s in enumerate(ins) if s.startswith("buffer_load") and not s.endswith(" lds")]
        late = "ELb1ELb0ELb0E" not in name
        assert len(stores) == 2 * 16 and len(loads) == (2 * 8 + 4 if late else 2 * 12), name
        assert not [s for s in ins if s.startswith("global_store")], name
        if late:   # the channels' loads, 16 bytes each, stand apart
            sw = [i for i in loads if ins[i].startswith("buffer_load_dwordx4")]
            assert len(sw) == 4, name
            rows = [i for i in loads if i not in sw]
            runs = [stores[:16], stores[16:], rows[:8], rows[8:]]
        else:
            runs = [stores[:16], stores[16:], loads[:12], loads[12:]]
        for run in runs:
            between = ins[run[0]:run[-1] + 1]
            assert not [s for s in between if s.startswith(("s_cbranch", "s_branch", "s_and_saveexec"))], name
            other = [s for s in between if s.startswith(("global_", "buffer_", "flat_", "scratch_"))]
            assert len(other) == len(run), name
