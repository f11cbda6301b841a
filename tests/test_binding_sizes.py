"""CPU checks that the binding of the row and int8 calls refuses sizes past 31
bits, which a C int would take as some other size.  The tensors have no
memory of their own (expanded from one element), and nothing is launched."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from fp8_routed_expert_amd import ops

BIG = 2 ** 32 + 16      # as a C int: 16


def wide(*shape, dtype=torch.int8):
    return torch.zeros((), dtype=dtype).expand(shape)


I32 = torch.int32


@pytest.fixture(autouse=True)
def no_device_needed(monkeypatch):
    """The other checks pass, and a call says what size the library would get."""
    monkeypatch.setattr(ops, "_arg", lambda t, *a: 4096)

    def call(name, stream, dev, *args):
        raise AssertionError(f"{name} called with {args}")
    monkeypatch.setattr(ops, "_call", call)


def refused():
    return pytest.raises(ValueError, match="past 2147483647|at most 2147483647")


def test_quantize():
    for shape in ((1, BIG), (BIG, 16), (2, BIG // 2, 16)):
        x = wide(*shape, dtype=torch.bfloat16)
        with refused():
            fre.moe_quantize_int8(x, wide(*shape), wide(*shape[:-1], dtype=torch.float32))


@pytest.mark.parametrize("shape", [(BIG, 16, 16), (2, BIG, 16), (2, 16, BIG)])
def test_experts(shape):
    E, n, k = shape
    s = wide(1, dtype=torch.float32)
    with refused():
        fre.moe_grouped_gemm_int8(wide(4, k), s, wide(*shape), s, s, s, s, s)
    with refused():
        fre.moe_grouped_gemm_int8_gather(wide(4, k), s, wide(4, dtype=I32), wide(*shape), s, s, s, s, s)


def test_gathered_rows():
    s = wide(1, dtype=torch.float32)
    with refused():
        fre.moe_grouped_gemm_int8_gather(wide(4, 16), s, wide(BIG, dtype=I32), wide(2, 16, 16), s, s, s, s, s)


def test_act_experts():
    with refused():
        fre.moe_act_requant_int8(wide(4, 64, dtype=torch.float32), wide(BIG + 1, dtype=I32), wide(BIG, dtype=I32),
                                 wide(4, 32), wide(4, dtype=torch.float32), wide(1, dtype=I32))


@pytest.mark.parametrize("what", ["E", "rows", "align_m"])
def test_sort(what):
    n = dict(E=4, rows=64, align_m=128)
    n[what] = BIG
    idx, s = wide(4, 2, dtype=I32), wide(1, dtype=I32)
    with refused():
        fre.moe_sort_tokens(idx, n["E"], fre.LAYOUT_CONTIGUOUS, n["align_m"], n["rows"], s, s, s, s, s, s, s)
