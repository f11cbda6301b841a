"""GPU tests of the row and int8 calls on more units than one launch has
workgroups (2^22): the kernels walk them, and the last ones are right.  And of
the differentiable calls with nothing to do."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.test_gpu_int8 import i32

pytestmark = pytest.mark.gpu

WORKGROUPS = 1 << 22


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def test_quantiser_walks(gpu):
    """Four rows to a workgroup."""
    R = 4 * WORKGROUPS + 4099
    torch.manual_seed(1)
    x = torch.randn(R, 16, device="cuda", dtype=torch.float16)
    q, s = torch.full((R, 16), 99, dtype=torch.int8, device="cuda"), torch.full((R,), 99.0, device="cuda")
    fre.moe_quantize_int8(x, q, s)
    want = x.float().abs().amax(1).double()
    assert ((s.double() * 127 - want).abs() <= want * 2.0 ** -24).all()
    assert torch.equal(q.double(), torch.round(x.double() / s.double()[:, None]))
    # the activation: rows of 2 x 16, the last 5 outside the segment
    h = torch.randn(R, 32, device="cuda", dtype=torch.float16)
    q.fill_(99)
    s.fill_(99)
    st = i32(1)
    fre.moe_act_requant_int8(h, torch.tensor([0, R], dtype=torch.int32, device="cuda"),
                             torch.tensor([R - 5], dtype=torch.int32, device="cuda"), q, s, st)
    gate, up = h[:-5].double().split(16, dim=1)
    v = gate / (1 + torch.exp(-gate)) * up
    rel = (gate.abs().amax() + 6) * 2.0 ** -23
    sd = s[:-5].double()
    assert ((sd - v.abs().amax(1) / 127).abs() <= 2 * rel * sd).all()
    assert ((q[:-5].double() * sd[:, None] - v).abs() <= (sd * (0.5 + 128 * rel) * (1 + 1e-12))[:, None]).all()
    assert (q[-5:] == 99).all() and (s[-5:] == 99).all() and int(st) == 0


# (T, K, H): sixteen short rows, four rows of a wave each, one row of a
# workgroup (K: more than 16 picks take a wave)
WALKS = [(16 * WORKGROUPS + 1025, 1, 8), (4 * WORKGROUPS + 1025, 17, 8), (WORKGROUPS + 1025, 1, 2064)]


@pytest.mark.parametrize("shape", WALKS, ids=["short", "wave", "workgroup"])
def test_rows_walk(gpu, shape):
    """Few tokens have a row, the last ones among them: all four row calls."""
    T, K, H = shape
    R = 64
    torch.manual_seed(T)
    tok = torch.cat([torch.randint(0, T, (40,)), torch.arange(T - 24, T)]).cuda()
    tok = torch.unique(tok)
    n = tok.numel()
    slot = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    slot[tok, K - 1] = torch.randperm(R, device="cuda")[:n].int()
    at = slot[tok, K - 1].long()
    st, x = i32(1), torch.empty(T, H, device="cuda", dtype=torch.bfloat16)
    x.fill_(1.5)
    x[tok] = torch.randn(n, H, device="cuda").bfloat16()
    a = torch.zeros(R, H, device="cuda", dtype=torch.bfloat16)
    fre.moe_permute_rows(x, slot, a, st)
    assert torch.equal(a[at], x[tok])
    w = torch.zeros(T, K, device="cuda")
    w[tok, K - 1] = 2.0
    out = torch.full_like(x, float("nan"))
    fre.moe_permute_rows_grad(a, slot, out, st)
    assert torch.equal(out[tok], a[at])
    out[tok] = 0
    assert not out.any()               # (a NaN counts as true)
    out.fill_(float("nan"))
    fre.moe_combine_rows(a, slot, w, out, st)
    assert torch.equal(out[tok], 2 * a[at])
    out[tok] = 0
    assert not out.any()
    del out
    dy, dw = torch.zeros_like(a), torch.full((T, K), float("nan"), device="cuda")
    fre.moe_combine_rows_grad(x, a, slot, w, dy, dw, st)
    assert torch.equal(dy[at], 2 * x[tok])
    ref = (x[tok].double() * a[at].double()).sum(1)
    mag = (x[tok].double() * a[at].double()).abs().sum(1)
    # a lane's products, 6 levels of lanes, the waves (as in the row calls' tests)
    n_roundings = 16 + 6 + 2 + -(-H // 2048) + 8
    assert ((dw[tok, K - 1].double() - ref).abs() <= (n_roundings + 1) * 2.0 ** -24 * mag).all()
    dw[tok, K - 1] = 0
    assert not dw.any() and int(st) == 0


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", ["no tokens", "no rows", "no picks"])
def test_routing_with_nothing_to_do(gpu, case, dt):
    """No tokens, a buffer without rows, and tokens whose experts are all
    elsewhere: zeros of the right shapes, forward and backward."""
    T, K, E, H, R = (0 if case == "no tokens" else 7), 2, 3, 40, (0 if case == "no rows" else 500)
    idx = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    if case == "no rows":
        idx[3, 1] = 2                    # dropped
    t = fre.sort_tokens(idx, E, R)
    x = torch.randn(T, H, device="cuda").to(dt).requires_grad_()
    w = torch.rand(T, K, device="cuda").requires_grad_()
    a = fre.permute_tokens(x, t)
    out = fre.combine_tokens(a * 1, w, t)
    out.backward(torch.ones_like(out))
    assert a.shape == (R, H) and out.shape == (T, H) and not a.any() and not out.any()
    assert x.grad.shape == x.shape and not x.grad.any() and w.grad.shape == w.shape and not w.grad.any()
    assert int(t.status) == (fre.ERR_OVERFLOW if case == "no rows" else 0)
    assert int(t.counts.sum()) == (case == "no rows")
