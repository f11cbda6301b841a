"""GPU tests of the norm, the router, the sorting, the experts' products and the
activation together, as a trained block uses them: against the block written
out in 64 bits, captured in a graph, on another stream, and under autograd's
own rules (unused outputs, strided inputs, frozen weights)."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.gpu_util import log
from tests.trained_util import values

pytestmark = pytest.mark.gpu

KEYS = ("x", "nw", "nb", "wr", "w13", "w2")


def leaves(T, E, H, I, dt, seed=0):
    """Parameters and input, on the device, and in 64 bits."""
    shapes = dict(x=(T, H), nw=(H,), nb=(H,), wr=(E, H), w13=(E, 2 * I, H), w2=(E, H, I))
    scale = dict(x=1.0, nw=0.2, nb=0.2, wr=H ** -0.5, w13=H ** -0.5, w2=I ** -0.5)
    d, d64 = {}, {}
    for n, (k, s) in enumerate(shapes.items()):
        d[k], d64[k] = values([seed, n], s, torch.float32 if k == "wr" else dt, scale[k], 1.0 if k == "nw" else 0.0)
    return d, d64


def block(p, K, E, **route):
    T = p["x"].shape[0]
    xn = fre.layer_norm(p["x"], p["nw"], p["nb"])
    idx, w, scores = fre.route_tokens(xn.float() @ p["wr"].t(), K, **route)
    t = fre.sort_tokens(idx, E, fre.contiguous_rows(T * K, E))
    a = fre.permute_tokens(xn, t)
    q = fre.gated_act(fre.grouped_linear(a, p["w13"], t), t)
    return fre.combine_tokens(fre.grouped_linear(q, p["w2"], t), w, t), scores, idx, t


def block64(p, idx, E, softmax, renorm, scale):
    """The block with the picks given, expert by expert, in 64 bits."""
    x = p["x"]
    xn = (x - x.mean(1, keepdim=True)) / torch.sqrt(x.var(1, correction=0, keepdim=True) + 1e-5) * p["nw"] + p["nb"]
    l = xn @ p["wr"].t()
    s = torch.softmax(l, 1) if softmax else torch.sigmoid(l)
    w = torch.where(idx >= 0, s.gather(1, idx.clamp(min=0)), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        h = xn[t] @ p["w13"][e].t()
        gate, up = h.chunk(2, 1)
        out = out.index_add(0, t, scale * w[t, k, None] * ((gate * torch.sigmoid(gate) * up) @ p["w2"][e].t()))
    return out, s


@pytest.mark.parametrize("dt,tol", [(torch.float32, 2e-5), (torch.float16, 8e-3), (torch.bfloat16, 6e-2)],
                         ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", [fre.SCORE_SOFTMAX, fre.SCORE_SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,H,I,K", [(1, 4, 64, 32, 2), (77, 5, 136, 72, 3), (300, 16, 264, 128, 4)])
def test_block(gpu, T, E, H, I, K, score, dt, tol):
    """Outputs and every gradient, by their norm.  A tensor of the chain carries
    the roundings of the ones before it: eight roundings to the rows' type (x's
    norm, the rows, h, q, y and their gradients) of half a step each, that the
    sums average; tol is 8 steps of the type (fp32: 160 steps of the sums)."""
    d, d64 = leaves(T, E, H, I, dt)
    p = {k: v.clone().requires_grad_() for k, v in d.items()}
    out, scores, idx, t = block(p, K, E, score=score, scale=1.5)
    assert int(t.status) == 0
    dout, dout64 = values([9], (T, H), dt)
    ds, ds64 = values([10], (T, E), torch.float32)
    torch.autograd.backward([out, scores], [dout, ds])
    p64 = {k: v.clone().requires_grad_() for k, v in d64.items()}
    out64, scores64 = block64(p64, idx.cpu().long(), E, score == fre.SCORE_SOFTMAX, True, 1.5)
    torch.autograd.backward([out64, scores64], [dout64, ds64])
    for k, got, want in [("out", out, out64), ("scores", scores, scores64)] + [(k, p[k].grad, p64[k].grad) for k in KEYS]:
        rel = float((got.detach().double().cpu() - want).norm() / want.norm())
        log(f"{k}: {rel:.2e}")
        assert rel <= tol, (k, rel)


def test_module_and_unused_outputs(gpu):
    torch.manual_seed(1)
    m = fre.RoutedExperts(E=6, H=128, I=64, K=2, score=fre.SCORE_SIGMOID, groups=3, top_groups=2, group_best=2)
    x = torch.randn(50, 128, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    m.bias[0] = -float("inf")
    out = m(x)
    assert not (m.table.slot_of < 0).any() and int(m.table.counts[0]) == 0 and int(m.route_status) == 0
    (out.float().square().mean() + 0.01 * m.scores.mean(0).square().sum()).backward()
    assert x.grad.isfinite().all()
    for k, v in m.named_parameters():
        assert v.grad is not None and v.grad.isfinite().all() and v.grad.abs().sum() > 0, k
    assert (m.w13.grad[0] == 0).all() and (m.w2.grad[0] == 0).all()
    # only the scores, only the weights, neither
    l = torch.randn(7, 6, device="cuda", requires_grad=True)
    idx, w, s = fre.route_tokens(l, 2)
    g1, = torch.autograd.grad(s[:, 0].sum(), l, retain_graph=True)
    g2, = torch.autograd.grad(w[:, 0].sum(), l)
    assert g1.abs().sum() > 0 and g2.abs().sum() > 0 and not idx.requires_grad
    # frozen weights: their gradients are not computed, the rows' is
    m.requires_grad_(False)
    x.grad = None
    m(x).float().sum().backward()
    assert x.grad.isfinite().all() and m.w2.grad is not None


def test_strided_and_broadcast(gpu):
    """Transposed, sliced and expanded inputs and gradients give what their
    contiguous copies give."""
    E, H, I, T = 3, 64, 40, 30
    big = torch.randn(T, 2 * H, device="cuda")
    x = big[:, ::2]
    w = torch.randn(H, device="cuda")
    assert torch.equal(fre.layer_norm(x, w), fre.layer_norm(x.contiguous(), w))
    x3 = torch.randn(2, 5, H, device="cuda", requires_grad=True)
    y = fre.layer_norm(x3.transpose(0, 1), w)
    y.backward(torch.ones(1, device="cuda").expand(5, 2, H))
    g = x3.grad.clone()
    x3.grad = None
    fre.layer_norm(x3.transpose(0, 1).contiguous(), w).sum().backward()
    assert torch.equal(g, x3.grad)
    idx = torch.randint(0, E, (T, 2), dtype=torch.int32, device="cuda")
    t = fre.sort_tokens(idx, E, fre.contiguous_rows(2 * T, E))
    a = fre.permute_tokens(x.contiguous(), t).detach()
    wt = torch.randn(E, H, I, device="cuda").requires_grad_()
    c = fre.grouped_linear(a, wt.transpose(1, 2), t)
    c.sum().backward()
    w2 = wt.detach().transpose(1, 2).contiguous().requires_grad_()
    c2 = fre.grouped_linear(a, w2, t)
    c2.sum().backward()
    assert torch.equal(c, c2) and torch.equal(wt.grad.transpose(1, 2), w2.grad)
    # rows of the buffer that no token has are zeros
    empty = (t.row_src < 0)
    assert (c[empty] == 0).all()
    s = torch.randn(T, E, device="cuda")
    a1 = fre.route_tokens(s.t().contiguous().t(), 2)
    a2 = fre.route_tokens(s, 2)
    assert all(torch.equal(u, v) for u, v in zip(a1, a2))


def test_captured_block(gpu):
    """Forward and backward captured in a graph and replayed on other inputs,
    with eager passes (on their own leaves) between the replays."""
    T, E, H, I, K = 96, 8, 128, 64, 2
    d, _ = leaves(T, E, H, I, torch.bfloat16)
    dout = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)

    def step(p):
        out, scores, idx, t = block(p, K, E)
        return [out, idx, *torch.autograd.grad([out, scores.square().sum()], [p[k] for k in KEYS], [dout, None])]

    p = {k: v.clone().requires_grad_() for k, v in d.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(p)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(p)
    for i in range(4):
        with torch.no_grad():
            p["x"].copy_(torch.randn(T, H, device="cuda") * (i + 1))
            p["w2"].mul_(1.1)
        graph.replay()
        torch.cuda.synchronize()
        eager = {k: v.detach().clone().requires_grad_() for k, v in p.items()}
        want = step(eager)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_two_streams(gpu):
    """Two blocks at once on two streams give what each gives alone."""
    T, E, H, I, K = 200, 8, 256, 128, 2
    runs = [{k: v.clone().requires_grad_() for k, v in leaves(T, E, H, I, torch.float16, s)[0].items()} for s in (1, 2)]

    def step(p):
        out, scores, _, _ = block(p, K, E)
        return [out, *torch.autograd.grad([out.float().sum() + scores.sum()], [p[k] for k in KEYS])]
    alone = [step(p) for p in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for p, s in zip(runs, streams):
            with torch.cuda.stream(s):
                got.append(step(p))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_captured_module(gpu):
    """A module's training step captured after an eager one of the same
    parameters, replayed with eager passes of a copy between the replays."""
    torch.manual_seed(4)
    kw = dict(E=6, H=128, I=64, K=2)
    m, other = fre.RoutedExperts(**kw), fre.RoutedExperts(**kw)
    other.load_state_dict(m.state_dict())
    x = torch.randn(70, 128, device="cuda", dtype=torch.bfloat16)

    def step(m):
        out = m(x)
        (out.float().square().mean() + m.scores.square().mean()).backward()
        return out.detach()
    step(m)
    m.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(m)
    for i in range(3):
        with torch.no_grad():
            x.copy_(torch.randn(70, 128, device="cuda") * (i + 1))
        for v in m.parameters():
            v.grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        other.zero_grad(set_to_none=True)
        assert torch.equal(got, step(other)), i


def test_router_in_float32_under_autocast(gpu):
    torch.manual_seed(5)
    m = fre.RoutedExperts(E=16, H=128, I=64, K=4)
    x = torch.randn(40, 128, device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        want = m(x), m.scores
        with torch.autocast("cuda", dtype=torch.bfloat16):
            got = m(x), m.scores
    assert got[0].dtype == want[0].dtype and all(torch.equal(a, b) for a, b in zip(got, want))
