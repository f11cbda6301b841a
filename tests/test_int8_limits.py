"""CPU checks of the 8-bit integer calls at their largest sizes: what does not
fit the kernels' index arithmetic is refused before any launch (there is no
GPU here, so a call that launches returns the HIP error 3; the pointers are
never followed)."""

import ctypes

from fp8_routed_expert_amd import _lib

P = ctypes.c_void_p(4096)
N = None


def test_quantize_row_length():
    """A row is walked with a 31-bit index in steps of 2048 values: it may not
    come within a step of 2^31."""
    f = _lib.load().moe_quantize_int8
    for dtype in (0, 1, 2):
        for cols in (0x7ffff010, 0x7ffffff0):
            assert f(P, dtype, 1, cols, P, P, N) == 2, hex(cols)
        assert f(N, dtype, 1, 0x7ffff000, P, P, N) == 1     # taken: the pointer is what it lacks


def test_product_channels():
    """The tile counts of a product are formed in 31 bits, with up to 255
    channels added."""
    lib = _lib.load()
    big = 0x7fffff10
    for n in (big, 0x7ffffff0):
        for m in (1, 20, 300):
            assert lib.moe_gemm_int8(P, P, P, P, m, n, 16, P, 1, N) == 2, (m, hex(n))
            assert lib.moe_linear_int8(P, 1, P, P, m, n, 16, P, 1, P, 1 << 20, N) == 2, (m, hex(n))
            assert lib.moe_grouped_gemm_int8(P, P, P, P, P, P, 1, m, n, 16, P, 1, P, N) == 2
            assert lib.moe_grouped_gemm_int8_gather(P, P, 9, P, P, P, P, P, 1, m, n, 16, P, 1, P, N) == 2
    assert lib.moe_gemm_int8(N, P, P, P, 1, 0x7fffff00, 16, P, 1, N) == 1    # taken so far


def test_linear_refuses_before_it_quantises():
    """A row count that the product cannot take is refused before the rows'
    quantisation is launched into the workspace."""
    f = _lib.load().moe_linear_int8
    m = 0x1ffffc01
    assert f(P, 1, P, P, m, 16, 16, P, 1, P, m * 20, N) == 2
    assert f(N, 1, P, P, m - 1, 16, 16, P, 1, P, m * 20, N) == 1


def test_scales_are_aligned():
    """Scales are 4-byte aligned, as the header asks, in every call."""
    lib = _lib.load()
    odd = ctypes.c_void_p(4098)
    assert lib.moe_quantize_int8(P, 1, 4, 48, P, odd, N) == 2
    assert lib.moe_act_requant_int8(P, 1, P, P, 4, 64, 48, P, odd, P, N) == 2
    for m, wsb in ((1, 64), (40, 4096)):     # one launch, two launches
        assert lib.moe_linear_int8(P, 1, P, odd, m, 32, 48, P, 1, P, wsb, N) == 2
    assert lib.moe_gemm_int8(P, odd, P, P, 4, 32, 48, P, 1, N) == 2
    assert lib.moe_gemm_int8(P, P, P, odd, 4, 32, 48, P, 1, N) == 2
