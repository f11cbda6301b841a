"""GPU tests of the RoutedExperts module inside a training program: activation
checkpoints."""

import pytest
import torch
from torch.utils.checkpoint import checkpoint

import fp8_routed_expert_amd as fre

pytestmark = pytest.mark.gpu


def grads(m, x, scores_of):
    m.zero_grad()
    x.grad = None
    out, scores = scores_of(m, x)
    (out.float().square().mean() + 10 * scores.mean(0).square().sum()).backward()
    return {"x": x.grad.clone(), **{k: v.grad.clone() for k, v in m.named_parameters()}}


@pytest.mark.parametrize("reentrant", [False, True])
def test_balancing_loss_through_a_checkpoint(gpu, reentrant):
    """The scores that a call returns carry their gradient through a checkpoint
    of either kind (a re-entrant one runs the module without a graph first, so
    that the scores that the module keeps have none)."""
    torch.manual_seed(3)
    m = fre.RoutedExperts(E=6, H=128, I=64, K=2)
    x = torch.randn(50, 128, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    plain = grads(m, x, lambda m, x: (m(x), m.scores))
    returned = grads(m, x, lambda m, x: m(x, with_scores=True))
    saved = grads(m, x, lambda m, x: checkpoint(m, x, True, use_reentrant=reentrant))
    none = grads(m, x, lambda m, x: (m(x), m.scores.detach()))
    for k, v in plain.items():
        scale = v.double().norm()
        # the same calls on the same inputs; room for a library product whose
        # sums have another order (64 sums' roundings of a leaf's type)
        tol = 64 * torch.finfo(v.dtype).eps * scale
        assert (returned[k].double() - v.double()).norm() <= tol, k
        assert (saved[k].double() - v.double()).norm() <= tol, k
    # (the loss does have a gradient of its own to lose)
    lost = (none["router"].double() - plain["router"].double()).norm()
    assert lost > 1000 * 64 * torch.finfo(torch.float32).eps * plain["router"].double().norm()


def test_returned_scores_are_the_kept_ones(gpu):
    m = fre.RoutedExperts(E=4, H=64, I=32, K=2)
    x = torch.randn(9, 64, device="cuda", dtype=torch.bfloat16)
    out, scores = m(x, with_scores=True)
    assert scores is m.scores and scores.shape == (9, 4) and torch.equal(out, m(x))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_converted_module(gpu, dt):
    """A module that its program converted as a whole: the router's product and
    the bias are still float32, from the converted values."""
    m = fre.RoutedExperts(E=6, H=64, I=32, K=2, score=fre.SCORE_SIGMOID)
    m.bias[2] = 0.25
    m.to(dt)
    x = torch.randn(40, 64, device="cuda", dtype=dt, requires_grad=True)
    out, scores = m(x, with_scores=True)
    assert out.dtype == dt and scores.dtype == torch.float32
    xn = fre.layer_norm(x, m.norm_weight, m.norm_bias)
    idx, _, want = fre.route_tokens(torch.nn.functional.linear(xn.float(), m.router.float()), 2,
                                    m.bias.float(), score=fre.SCORE_SIGMOID)
    assert torch.equal(scores, want) and int(m.route_status) == 0
    (out.float().square().sum() + scores.square().sum()).backward()
    for k, v in m.named_parameters():
        assert v.grad.dtype == dt and v.grad.isfinite().all() and v.grad.abs().sum() > 0, k
