"""What combine_tokens keeps for its backward pass (no GPU: the row calls are
replaced by plain sums)."""

import pytest
import torch

from fp8_routed_expert_amd import routing


@pytest.fixture
def plain(monkeypatch):
    calls = {}

    def combine(y, slot, w, out, status):
        out.copy_((y[slot.long()] * w[..., None]).sum(1))

    def grad(dout, y, slot, w, dy, dw, status, row_src=None):
        calls["y"], calls["w"] = y is not None, w is not None
        if dy is not None:
            dy.zero_()
            dy[slot.long()] = dout[:, None] * w[..., None]
        if dw is not None:
            dw.copy_((y[slot.long()] * dout[:, None]).sum(-1))
    monkeypatch.setattr(routing.ops, "moe_combine_rows", combine)
    monkeypatch.setattr(routing.ops, "moe_combine_rows_grad", grad)
    return calls


@pytest.mark.parametrize("needs", [(True, False), (False, True), (True, True)], ids=["y", "weights", "both"])
def test_saved_for_backward(plain, needs):
    """Only what a gradient that is asked for reads: y's needs the weights, the
    weights' needs y (a buffer of all routed rows)."""
    T, K, R, H = 3, 2, 7, 5
    t = routing.SortedTokens()
    t.T, t.K, t.E, t.rows_total, t.status, t.row_src = T, K, 2, R, None, None
    t.slot_of = torch.tensor([[0, 4], [2, 1], [6, 3]], dtype=torch.int32)
    y = torch.randn(R, H, requires_grad=needs[0])
    w = torch.rand(T, K, requires_grad=needs[1])
    out = routing.combine_tokens(y * 1 if needs[0] else y, w * 1 if needs[1] else w, t)
    saved = [v for v in out.grad_fn.saved_tensors if v is not None]
    assert any(v.shape == (R, H) for v in saved) == needs[1]
    assert any(v.shape == (T, K) for v in saved) == needs[0]
    g = torch.randn(T, H)
    got = torch.autograd.grad(out, [v for v, n in zip((y, w), needs) if n], g)
    yd, wd = y.detach().clone().requires_grad_(), w.detach().clone().requires_grad_()
    want = torch.autograd.grad((yd[t.slot_of.long()] * wd[..., None]).sum(1), (yd, wd), g)
    for a, b in zip(got, [v for v, n in zip(want, needs) if n]):
        assert torch.allclose(a, b)
    assert plain == {"y": needs[1], "w": needs[0]}


def test_refusals():
    """What a gradient reads may not be left out."""
    g, y, slot, w = torch.zeros(3, 5), torch.zeros(7, 5), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    for args in ((g, None, slot, w, None, w), (g, None, slot, w, y, w), (g, y, slot, None, y, None)):
        with pytest.raises(ValueError, match="needs"):
            routing.ops.moe_combine_rows_grad(*args, slot)
    with pytest.raises(ValueError, match="neither"):
        routing.ops.moe_combine_rows_grad(g, None, slot, None, None, None, slot)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
def test_one_gradient_at_a_time(gpu, dt):
    """Either gradient alone, without what it does not read, equals the two
    together, and the rows of y are free once no gradient needs them."""
    torch.manual_seed(4)
    T, K, E, H = 500, 4, 6, 1000
    idx = torch.stack([torch.randperm(E + 2)[:K] for _ in range(T)]).int()
    idx[idx >= E] = -1
    t = routing.sort_tokens(idx.cuda(), E, T * K + 127 * E)
    y, w = torch.randn(t.rows_total, H, device="cuda").to(dt), torch.rand(T, K, device="cuda")
    g = torch.randn(T, H, device="cuda").to(dt)
    yb, wb = y.clone().requires_grad_(), w.clone().requires_grad_()
    want = torch.autograd.grad(routing.combine_tokens(yb, wb, t), (yb, wb), g)
    for i in range(2):
        ya, wa = y.clone().requires_grad_(i == 0), w.clone().requires_grad_(i == 1)
        out = routing.combine_tokens(ya, wa, t)
        assert torch.equal(torch.autograd.grad(out, (ya, wa)[i], g)[0], want[i])
    ya = y.clone().requires_grad_()
    kept = ya * 1                        # (its backward keeps nothing)
    before = torch.cuda.memory_allocated()
    out = routing.combine_tokens(kept, w, t)
    size = kept.numel() * kept.element_size()
    del kept
    # (the allocator may give out a block of up to 1 MB more than was asked for)
    assert size > 5 << 20
    assert torch.cuda.memory_allocated() <= before - size + out.numel() * out.element_size() + (2 << 20)
    assert torch.equal(torch.autograd.grad(out, ya, g)[0], want[0])
    assert int(t.status) == 0
