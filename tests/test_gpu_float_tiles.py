"""GPU tests of every kernel that the products in 32 and 16 bits and their
gradients choose (test_float_tile_rule.py checks that the sizes reach them all),
and of sums past 2^32 bytes.  The inputs are small whole numbers, whose sums
are exact in fp32 in any order: results are compared bit by bit."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.float_tiles import CASES, rows_of
from tests.trained_util import Guarded, table, valid_mask

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = ["f32", "bf16", "f16"]


def whole(g, most, *shape, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


def run_case(counts, rows, layout, align, N, K, dt, zero_rest, dw_type):
    E = len(counts)
    c, o, R, seg = table(counts, rows, layout, align)
    g = torch.Generator(device="cuda").manual_seed(N + K + R)
    # sums of up to 7176 products of at most 4: below 65504, fp16's largest
    a, w, dc = (whole(g, 2, *s, dtype=dt) for s in ((R, K), (E, N, K), (R, N)))
    rest = ~valid_mask(seg, R).cuda()
    a[rest], dc[rest] = float("nan"), float("nan")
    gd = Guarded()
    out, da = gd.new(R, N, dtype=dt, fill=9.0), gd.new(R, K, dtype=dt, fill=9.0)
    dw = gd.new(E, N, K, dtype=dw_type)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, fre.moe_grouped_gemm_float_workspace_bytes(E, R, N, K)), dtype=torch.uint8, device="cuda")
    fre.moe_grouped_gemm_float(a, w, o, c, out, st, zero_rest)
    fre.moe_grouped_gemm_float_grad_rows(dc, w, o, c, da, st, zero_rest)
    fre.moe_grouped_gemm_float_grad_weights(dc, a, o, c, dw, ws, st)
    gd.check()
    assert int(st) == 0
    left = 0.0 if zero_rest else 9.0
    assert (out[rest] == left).all() and (da[rest] == left).all()
    for e, (b, n) in enumerate(seg):
        A, W, D = a[b:n].double(), w[e].double(), dc[b:n].double()
        assert torch.equal(out[b:n], (A @ W.t().contiguous()).to(dt)), ("product", e)
        assert torch.equal(da[b:n], (D @ W).to(dt)), ("rows' gradient", e)
        assert torch.equal(dw[e], (D.t().contiguous() @ A).to(dw_type)), ("weights' gradient", e)


@pytest.mark.parametrize("counts,align,N,K,dt", [(c, al, n, k, d) for c, al, n, k, dts in CASES for d in dts],
                         ids=[f"{len(c)}x{rows_of(c, al)}-{n}x{k}-{NAMES[d]}" for c, al, n, k, dts in CASES
                              for d in dts])
def test_every_kernel(gpu, counts, align, N, K, dt):
    run_case(counts, rows_of(counts, align), 0, align, N, K, TYPES[dt], False, TYPES[dt])
    run_case(counts, rows_of(counts, align) + 40, 0, align, N, K, TYPES[dt], True, torch.float32)


@pytest.mark.parametrize("dt", TYPES, ids=NAMES)
def test_weights_gradient_past_4_gb(gpu, dt):
    """Rows past 2^32 bytes, and a segment whose sum is split: every element."""
    R, K, N = (150000 if dt == torch.float32 else 300000), 8192, 72
    c, o, _, seg = table([1000, R - 1040], R, 0, 1)
    g = torch.Generator(device="cuda").manual_seed(5)
    a, dc = whole(g, 2, R, K, dtype=dt), whole(g, 2, R, N, dtype=dt)
    dw = torch.full((2, N, K), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = fre.moe_grouped_gemm_float_workspace_bytes(2, R, N, K)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    fre.moe_grouped_gemm_float_grad_weights(dc, a, o, c, dw, ws, st)
    assert int(st) == 0
    for e, (b, n) in enumerate(seg):
        ref = torch.zeros(N, K, dtype=torch.float64, device="cuda")
        for i in range(b, n, 20000):
            s = slice(i, min(n, i + 20000))
            ref += dc[s].double().t().contiguous() @ a[s].double()
        assert torch.equal(dw[e].double(), ref), e


@pytest.mark.parametrize("rows", [127, 128, 143, 160])
def test_full_segments(gpu, rows):
    """Fixed-capacity segments that are all full, on both sides of the buffers
    that a contiguous layout of few rows has too."""
    for E, N, K in ((8, 2048, 520), (1, 4096, 264)):
        run_case([rows] * E, rows, 1, 1, N, K, torch.bfloat16, False, torch.float32)
