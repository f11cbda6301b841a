"""GPU tests of the gated activation and its gradient on buffers of more than
2^30 rows, and on more experts than a wave has lanes."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.trained_util import TYPES, U, Guarded, close, rounding, table, valid_mask, values

pytestmark = pytest.mark.gpu


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def test_rows_past_30_bits(gpu):
    """Segments at the start, around row 2^30 and at the end of the narrowest
    buffer come out as the same rows do in a small one; rows that no expert has
    are left as they were."""
    R, I = (1 << 30) + 5000, 8
    starts, counts = [0, (1 << 30) - 40, R - 77], [100, 90, 77]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    off, cnt, st = i32(starts + [R]), i32(counts), status()
    h = torch.empty(R, 2 * I, dtype=torch.bfloat16, device="cuda")
    small = torch.randn(sum(counts), 2 * I, device="cuda").bfloat16()
    dq_small = torch.randn(sum(counts), I, device="cuda").bfloat16()
    pieces = [slice(s, s + n) for s, n in zip(starts, counts)]
    for piece, rows in zip(pieces, small.split(counts)):
        h[piece] = rows
    c1, o1 = i32(counts), i32([0, 100, 190, 267])
    want = torch.empty_like(dq_small)
    fre.moe_gated_act(small, o1, c1, want, st)
    q = torch.full((R, I), 7.0, dtype=torch.bfloat16, device="cuda")
    fre.moe_gated_act(h, off, cnt, q, st)
    near = [slice(100, 3000), slice((1 << 30) - 3000, (1 << 30) - 40), slice((1 << 30) + 50, (1 << 30) + 3000),
            slice(R - 1000, R - 77)]
    assert torch.equal(torch.cat([q[p] for p in pieces]), want)
    assert all((q[n] == 7.0).all() for n in near)
    dh_small = torch.empty_like(small)
    fre.moe_gated_act_grad(dq_small, small, o1, c1, dh_small, st)
    dq = q
    for piece, rows in zip(pieces, dq_small.split(counts)):
        dq[piece] = rows
    dh = torch.full((R, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    fre.moe_gated_act_grad(dq, h, off, cnt, dh, st)
    assert torch.equal(torch.cat([dh[p] for p in pieces]), dh_small)
    assert all((dh[n] == 7.0).all() for n in near)
    assert int(st) == 0


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("zero_rest", [False, True])
@pytest.mark.parametrize("E,I,layout", [(70, 40, 0), (300, 264, 0), (70, 8, 1), (1024, 24, 1)])
def test_many_experts(gpu, E, I, layout, zero_rest, dt):
    """Segments of none to many rows; rows that no expert has hold NaN."""
    counts = [(7 * e) % 23 if e % 5 else 0 for e in range(E)]
    counts[E - 1] = 150 if not layout else 22
    c, o, R, seg = table(counts, 22 if layout else sum(-(-n // 16) * 16 for n in counts) + 37, layout, 16)
    valid = valid_mask(seg, R)
    h, h64 = values([20, E], (R, 2 * I), TYPES[dt], 2.0)
    dq, dq64 = values([21, E], (R, I), TYPES[dt])
    h[~valid.cuda()] = float("nan")
    dq[~valid.cuda()] = float("nan")
    g, st = Guarded(), status()
    q, dh = g.new(R, I, dtype=TYPES[dt], fill=9.0), g.new(R, 2 * I, dtype=TYPES[dt], fill=9.0)
    fre.moe_gated_act(h, o, c, q, st, zero_rest)
    fre.moe_gated_act_grad(dq, h, o, c, dh, st, zero_rest)
    g.check()
    assert int(st) == 0
    rest = 0.0 if zero_rest else 9.0
    assert (q[~valid.cuda()] == rest).all() and (dh[~valid.cuda()] == rest).all()
    h64, dq64 = h64[valid], dq64[valid]
    gate, up = h64[:, :I], h64[:, I:]
    s = torch.sigmoid(gate)
    # 1 - sigmoid: e = exp(-|g|) from the hardware's exponential of half the
    # argument (2 U), squared, and its correction (7 U in all), 1 + e (U), the
    # reciprocal (2 U) and a product (U): 11 U, and as many for sigmoid.  q adds
    # two products; dh's first half two products, the sum 1 + g (1 - s) (U, and
    # 11 U of its second term) and another product, its second half two
    ref = gate * s * up
    close(q[valid.cuda()], ref, 13 * U * ref.abs() + rounding(ref, TYPES[dt]), "q")
    ref = torch.cat([dq64 * up * s * (1 + gate * (1 - s)), dq64 * gate * s], 1)
    mag = torch.cat([26 * (dq64 * up * s).abs() * (1 + gate.abs() * (1 - s)), 13 * (dq64 * gate * s).abs()], 1)
    close(dh[valid.cuda()], ref, U * mag + rounding(ref, TYPES[dt]), "dh")
