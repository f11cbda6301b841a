"""GPU tests of the experts' products in 32 and 16 bits with their gradients,
and of the gated activation, against 64-bit sums with counted roundings."""

import math

import numpy as np
import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.trained_util import TYPES, U, Guarded, close, rounding, table, valid_mask, values

pytestmark = pytest.mark.gpu

# counts, rows (of the buffer; masked: of an expert's segment), layout, N, K:
# one row, no rows, experts without rows, ends inside a tile, clipped segments
# (of the buffer and of a capacity), sizes no tile divides, one step and many
CASES = [
    ([1], 128, 0, 8, 8), ([0], 128, 0, 16, 8), ([3, 0, 1], 16, 1, 40, 72), ([1] * 8, 16, 1, 128, 256),
    ([5, 130, 0, 64, 257], 900, 0, 136, 200), ([16, 17, 40], 16, 1, 64, 64), ([100, 128, 129], 300, 0, 64, 48),
    ([300], 300, 0, 512, 264), ([33, 1, 31, 65], 640, 0, 520, 1032), ([700, 90], 900, 0, 256, 512),
    ([0, 0, 0], 0, 0, 64, 64), ([2] * 70, 4, 1, 24, 136), ([64, 500, 7, 3], 640, 1, 264, 320),
    ([40, 41], 48, 1, 1000, 2056), ([1000], 1024, 0, 128, 136), ([260, 100, 513], 1152, 0, 264, 328),
    ([13] * 3, 16, 1, 2048, 520),
]
IDS = [f"{len(c[0])}x{sum(c[0])}x{c[3]}x{c[4]}" for c in CASES]


def inputs(case, dt):
    counts, rows, layout, N, K = case
    c, o, R, seg = table(counts, rows, layout)
    E = len(counts)
    a, a64 = values([1, R, K], (R, K), TYPES[dt])
    w, w64 = values([2, N, K], (E, N, K), TYPES[dt], 0.3)
    dc, dc64 = values([3, R, N], (R, N), TYPES[dt])
    # rows that are not valid are never read
    other = ~valid_mask(seg, R)
    a[other.cuda()] = math.nan
    dc[other.cuda()] = math.nan
    return c, o, R, seg, a, a64, w, w64, dc, dc64


def check_rows(got, seg, R, zeroed, ref, mag, L, t, what):
    valid = valid_mask(seg, R)
    rest = got.cpu()[~valid]
    assert (rest == 0).all() if zeroed else rest.isnan().all(), what
    close(got.cpu()[valid], ref[valid], (L + 2) * U * mag[valid] + rounding(ref[valid], t), what)


@pytest.mark.parametrize("zero", [False, True], ids=["left", "zeroed"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_product(gpu, case, dt, zero):
    c, o, R, seg, a, a64, w, w64, _, _ = inputs(case, dt)
    N, K = case[3:]
    ref, mag = torch.zeros(R, N, dtype=torch.float64), torch.zeros(R, N, dtype=torch.float64)
    for e, (b, n) in enumerate(seg):
        ref[b:n] = a64[b:n] @ w64[e].t()
        mag[b:n] = a64[b:n].abs() @ w64[e].abs().t()
    g = Guarded()
    out, st = g.new(R, N, dtype=TYPES[dt]), torch.zeros(1, dtype=torch.int32, device="cuda")
    fre.moe_grouped_gemm_float(a, w, o, c, out, st, zero)
    g.check()
    assert int(st) == 0
    check_rows(out, seg, R, zero, ref, mag, K, TYPES[dt], "product")


@pytest.mark.parametrize("zero", [False, True], ids=["left", "zeroed"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_rows_gradient(gpu, case, dt, zero):
    c, o, R, seg, _, _, w, w64, dc, dc64 = inputs(case, dt)
    N, K = case[3:]
    ref, mag = torch.zeros(R, K, dtype=torch.float64), torch.zeros(R, K, dtype=torch.float64)
    for e, (b, n) in enumerate(seg):
        ref[b:n] = dc64[b:n] @ w64[e]
        mag[b:n] = dc64[b:n].abs() @ w64[e].abs()
    g = Guarded()
    out, st = g.new(R, K, dtype=TYPES[dt]), torch.zeros(1, dtype=torch.int32, device="cuda")
    fre.moe_grouped_gemm_float_grad_rows(dc, w, o, c, out, st, zero)
    g.check()
    assert int(st) == 0
    check_rows(out, seg, R, zero, ref, mag, N, TYPES[dt], "rows' gradient")


@pytest.mark.parametrize("out_f32", [False, True], ids=["own", "f32"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_weights_gradient(gpu, case, dt, out_f32):
    c, o, R, seg, a, a64, _, _, dc, dc64 = inputs(case, dt)
    N, K = case[3:]
    E = len(seg)
    t = torch.float32 if out_f32 else TYPES[dt]
    ref, mag = torch.zeros(E, N, K, dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64)
    for e, (b, n) in enumerate(seg):
        ref[e] = dc64[b:n].t() @ a64[b:n]
        mag[e] = dc64[b:n].abs().t() @ a64[b:n].abs()
    g = Guarded()
    out, st = g.new(E, N, K, dtype=t), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = g.new(fre.moe_grouped_gemm_float_workspace_bytes(E, R, N, K), dtype=torch.uint8)
    fre.moe_grouped_gemm_float_grad_weights(dc, a, o, c, out, ws, st)
    g.check()
    assert int(st) == 0
    L = torch.tensor([n - b for b, n in seg], dtype=torch.float64)[:, None, None]
    close(out, ref, (L + 2) * U * mag + rounding(ref, t), "weights' gradient")
    for e, (b, n) in enumerate(seg):
        if n == b:
            assert (out[e] == 0).all()


def test_infinities_stay_in_their_rows(gpu):
    """An infinity or a NaN of one row or one weight reaches no other output."""
    c, o, R, seg = table([70, 50], 256)
    N, K = 72, 136
    a, _ = values([7], (R, K), torch.bfloat16)
    w, _ = values([8], (2, N, K), torch.bfloat16)
    a[3, 5], a[128 + 49, K - 1] = math.inf, math.nan
    w[1, 9, 0] = math.nan
    out, st = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    fre.moe_grouped_gemm_float(a, w, o, c, out, st)
    bad = ~out.isfinite().cpu()
    want = torch.zeros(R, N, dtype=torch.bool)
    want[3], want[128 + 49] = True, True
    want[128:128 + 50, 9] = True
    assert torch.equal(bad, want)


def test_bad_tables(gpu):
    """Tables that do not describe segments set the status bit, and nothing is
    read or written outside the buffer."""
    N, K, R = 64, 64, 256
    a, _ = values([9], (R, K), torch.bfloat16)
    w, _ = values([10], (3, N, K), torch.bfloat16)
    h, _ = values([11], (R, 2 * K), torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for off, cnt in (((0, 128, 64, 256), (10, 10, 10)), ((0, 128, 256, 256), (10, -1, 0)),
                     ((-64, 0, 128, 256), (64, 10, 10)), ((0, 2 ** 31 - 1, -2 ** 31, 256), (2 ** 31 - 1, 5, 5))):
        for call in range(5):
            g, st = Guarded(), i32(0)
            if call == 0:
                fre.moe_grouped_gemm_float(a, w, i32(*off), i32(*cnt), g.new(R, N, dtype=torch.bfloat16), st, True)
            elif call == 1:
                fre.moe_grouped_gemm_float_grad_rows(a, w, i32(*off), i32(*cnt), g.new(R, K, dtype=torch.bfloat16), st)
            elif call == 2:
                ws = g.new(fre.moe_grouped_gemm_float_workspace_bytes(3, R, N, K), dtype=torch.uint8)
                fre.moe_grouped_gemm_float_grad_weights(a, a, i32(*off), i32(*cnt), g.new(3, N, K), ws, st)
            elif call == 3:
                fre.moe_gated_act(h, i32(*off), i32(*cnt), g.new(R, K, dtype=torch.bfloat16), st, True)
            else:
                fre.moe_gated_act_grad(a, h, i32(*off), i32(*cnt), g.new(R, 2 * K, dtype=torch.bfloat16), st, True)
            g.check()
            assert int(st) == fre.ERR_BAD_INDEX, (off, call)


def act64(h):
    gate, up = h.chunk(2, 1)
    return gate * torch.sigmoid(gate) * up


ACT = [([1], 128, 0, 8), ([0, 3], 16, 1, 40), ([100, 0, 77], 300, 0, 2048), ([5, 9, 40], 16, 1, 264),
       ([700, 300], 1100, 0, 1032)]


@pytest.mark.parametrize("zero", [False, True], ids=["left", "zeroed"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("case", ACT, ids=[f"{len(c[0])}x{sum(c[0])}x{c[3]}" for c in ACT])
def test_act(gpu, case, dt, zero):
    counts, rows, layout, I = case
    t = TYPES[dt]
    c, o, R, seg = table(counts, rows, layout)
    h, h64 = values([21, R, I], (R, 2 * I), t, 3.0)
    dq, dq64 = values([22, R, I], (R, I), t)
    if R and I > 16:
        # the ends of the sigmoid
        ends = torch.tensor([0.0, -0.0, 20.0, -20.0, 60.0, -60.0, 87.0, -87.0, 88.5, -88.5, -100.0, 300.0, -300.0])
        h64[:, :13] = ends.to(t).double()
        h[:, :13] = ends.to(t).cuda()
    valid = valid_mask(seg, R)
    g, st = Guarded(), torch.zeros(1, dtype=torch.int32, device="cuda")
    q, dh = g.new(R, I, dtype=t), g.new(R, 2 * I, dtype=t)
    fre.moe_gated_act(h, o, c, q, st, zero)
    fre.moe_gated_act_grad(dq, h, o, c, dh, st, zero)
    g.check()
    assert int(st) == 0
    for out in (q, dh):
        rest = out.cpu()[~valid]
        assert (rest == 0).all() if zero else rest.isnan().all()
    # the sigmoid: base-2 exponential 1 ulp of fp32 squared (4 U and 2 of its
    # products), its argument's two parts (U), one addition, the reciprocal's
    # ulp (2 U) and a product: 12 U; then two to four products and a sum.  A
    # sigmoid below 2^-149 is 0.
    s = torch.sigmoid(h64[:, :I])
    gate, up = h64.chunk(2, 1)
    ref = act64(h64)
    low = 2.0 ** -148 * (1 + gate.abs()) * (1 + up.abs())
    close(q.cpu()[valid], ref[valid], (16 * U * ref.abs() + low + rounding(ref, t))[valid], "act")
    x = h64.clone().requires_grad_()
    act64(x).backward(dq64)
    part = (dq64 * up * s).abs() * (1 + (gate * (1 - s)).abs())
    tol = torch.cat([32 * U * part, 16 * U * (dq64 * gate * s).abs()], 1)
    # a subnormal sigmoid is off by up to two steps of 2^-149 in itself, and both
    # halves multiply it by the gate (dh of up: dq g s; of gate: dq up s g), the
    # first by up as well
    low = (2.0 ** -147 * (1 + gate.abs()) * (1 + up.abs()) * (1 + dq64.abs())).repeat(1, 2)
    close(dh.cpu()[valid], x.grad[valid], (tol + low + rounding(x.grad, t))[valid], "act gradient")


def test_act_of_infinities(gpu):
    """Infinite and NaN gates give what the formula gives."""
    c, o, R, _ = table([2], 2)
    h = torch.ones(R, 16, device="cuda")
    h[0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1e30])
    h[1, 8:10] = torch.tensor([math.inf, math.nan])
    q, st = torch.zeros(R, 8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    fre.moe_gated_act(h, o, c, q, st)
    q = q.cpu()
    assert q[0, 0] == math.inf and q[0, 1].isnan() and q[0, 2].isnan() and q[0, 3] == np.float32(1e30)
    assert q[1, 0] == math.inf and q[1, 1].isnan() and q[1, 2:].isfinite().all()
