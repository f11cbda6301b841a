"""GPU tests of the router, the norm, the experts' products and the activation
on buffers past 2^32 bytes, on other streams, captured in graphs that run at
once, and on rows that nothing is to touch."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.gpu_util import log
from tests.trained_util import U, table

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def normal(*shape, dtype=BF16):
    return torch.randn(*shape, device="cuda", dtype=dtype)


def test_norm_past_4_gb(gpu):
    """The last rows come out as the same rows alone do."""
    T, H = 310000, 7168
    x, w = normal(T, H), normal(H)
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fre.moe_layer_norm(x, w, None, 1e-5, y, mean, rstd)
    tail = slice(T - 700, T)
    y2, m2, r2 = torch.empty_like(y[tail]), torch.empty(700, device="cuda"), torch.empty(700, device="cuda")
    fre.moe_layer_norm(x[tail].clone(), w, None, 1e-5, y2, m2, r2)
    assert torch.equal(y[tail], y2) and torch.equal(mean[tail], m2) and torch.equal(rstd[tail], r2)
    dy = y        # (as good as any)
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda", dtype=BF16)
    ws = torch.empty(fre.moe_layer_norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    fre.moe_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, None, ws)
    d2 = torch.empty_like(y2)
    fre.moe_layer_norm_grad(dy[tail].clone(), x[tail].clone(), w, m2, r2, d2, None, None, ws)
    assert torch.equal(dx[tail], d2)
    ref = torch.zeros(H, dtype=torch.float64, device="cuda")
    mag = torch.zeros(H, dtype=torch.float64, device="cuda")
    for b in range(0, T, 31000):
        s = slice(b, min(T, b + 31000))
        v = dy[s].double() * (x[s].double() - mean[s, None].double()) * rstd[s, None].double()
        ref += v.sum(0)
        mag += v.abs().sum(0)
    # T / 256 rows of a workgroup one after the other, then the workgroups' sums
    tol = (T / 256 + 100) * U * mag + 2.0 ** -8 * ref.abs()
    assert ((dw.double() - ref).abs() <= tol).all()


def test_act_past_4_gb(gpu):
    R, I = 560000, 2048
    c, o, _, _ = table([R - 300000, 299000], R, 0, 1)
    h, st = normal(R, 2 * I), status()
    q, dh = torch.zeros(R, I, device="cuda", dtype=BF16), torch.zeros_like(h)
    fre.moe_gated_act(h, o, c, q, st)
    fre.moe_gated_act_grad(q, h, o, c, dh, st)
    tail = slice(R - 1500, R)
    c2, o2, _, _ = table([500], 1500, 0, 1)
    h2 = h[tail].clone()
    q2, d2 = torch.zeros(1500, I, device="cuda", dtype=BF16), torch.zeros_like(h2)
    fre.moe_gated_act(h2, o2, c2, q2, st)
    fre.moe_gated_act_grad(q2, h2, o2, c2, d2, st)
    assert int(st) == 0 and torch.equal(q[tail], q2) and torch.equal(dh[tail], d2)
    assert (q[R - 1000:] == 0).all() and (q[R - 1500:R - 1000] != 0).any()


@pytest.mark.parametrize("dt", [BF16, torch.float32], ids=["bf16", "f32"])
def test_products_past_4_gb(gpu, dt):
    """Rows, and a segment, past 2^32 bytes, against 64 bits at the ends."""
    R, K, N = (300000, 8192, 72) if dt == BF16 else (150000, 8192, 72)
    first = 1000
    c, o, _, seg = table([first, R - first - 40], R, 0, 1)
    a, w, st = normal(R, K, dtype=dt), normal(2, N, K, dtype=dt), status()
    out, da = torch.zeros(R, N, device="cuda", dtype=dt), torch.zeros_like(a)
    dw = torch.zeros(2, N, K, device="cuda")
    fre.moe_grouped_gemm_float(a, w, o, c, out, st)
    half = torch.finfo(dt).eps / 2 if dt != torch.float32 else 0.0
    for e, rows in ((0, slice(0, 300)), (1, slice(first, first + 300)), (1, slice(R - 340, R - 40))):
        ref = a[rows].double() @ w[e].double().t()
        mag = a[rows].double().abs() @ w[e].double().abs().t()
        assert ((out[rows].double() - ref).abs() <= (K + 2) * U * mag + half * ref.abs()).all()
    assert (out[R - 40:] == 0).all()
    dc = normal(R, N, dtype=dt)
    fre.moe_grouped_gemm_float_grad_rows(dc, w, o, c, da, st)
    rows = slice(R - 340, R - 40)
    ref, mag = dc[rows].double() @ w[1].double(), dc[rows].double().abs() @ w[1].double().abs()
    assert ((da[rows].double() - ref).abs() <= (N + 2) * U * mag + half * ref.abs()).all()
    assert (da[R - 40:] == 0).all()
    del da
    ws = torch.empty(max(1, fre.moe_grouped_gemm_float_workspace_bytes(2, R, N, K)), dtype=torch.uint8, device="cuda")
    fre.moe_grouped_gemm_float_grad_weights(dc, a, o, c, dw, ws, st)
    for e, (b, n) in enumerate(seg):
        ref, mag = (torch.zeros(N, K, dtype=torch.float64, device="cuda") for _ in range(2))
        for i in range(b, n, 20000):
            s = slice(i, min(n, i + 20000))
            ref += dc[s].double().t() @ a[s].double()
            mag += dc[s].double().abs().t() @ a[s].double().abs()
        assert ((dw[e].double() - ref).abs() <= (n - b + 2) * U * mag).all(), e
    assert int(st) == 0


def test_router_past_4_gb(gpu):
    T, E, K = 2 ** 23 + 77, 288, 8
    l = normal(T, E)
    b = torch.randn(E, device="cuda") * 0.05
    kw = dict(bias=b, score=fre.SCORE_SIGMOID, groups=9, top_groups=4, group_best=2)
    idx, w, st = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda"), status()
    fre.moe_route_tokens(l, idx, w, st, **kw)
    tail = slice(T - 500, T)
    i2, w2 = torch.empty(500, K, dtype=torch.int32, device="cuda"), torch.empty(500, K, device="cuda")
    fre.moe_route_tokens(l[tail].clone(), i2, w2, st, **kw)
    assert torch.equal(idx[tail], i2) and torch.equal(w[tail], w2) and int(st) == 0
    dl = torch.empty_like(l)
    fre.moe_route_tokens_grad(l, idx, w, dl, st, fre.SCORE_SIGMOID)
    d2 = torch.empty(500, E, device="cuda", dtype=BF16)
    fre.moe_route_tokens_grad(l[tail].clone(), i2, w2, d2, st, fre.SCORE_SIGMOID)
    assert torch.equal(dl[tail], d2)


def calls(seed):
    """One of each call on its own buffers: a function that makes them, and the
    outputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s, dt=BF16: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    E, N, K, H, T = 4, 136, 264, 264, 700
    c, o, R, _ = table([300, 0, 77, 200], 800)
    a, w, dc, h = new(R, K), new(E, N, K), new(R, N), new(R, 2 * K)
    x, wt, l = new(T, H), new(H), new(T, 40, dt=torch.float32)
    z = lambda *s, dt=BF16: torch.zeros(*s, device="cuda", dtype=dt)  # noqa: E731
    st = status()
    out = dict(c=z(R, N), da=z(R, K), dw=z(1, 64, 64), dw2=z(E, N, K), q=z(R, K), dh=z(R, 2 * K), y=z(T, H),
               dx=z(T, H), dwt=z(H), mean=z(T, dt=torch.float32), rstd=z(T, dt=torch.float32),
               idx=z(T, 6, dt=torch.int32), tw=z(T, 6, dt=torch.float32), dl=z(T, 40, dt=torch.float32))
    # (a long segment, split)
    R1 = 8192
    c1, o1, _, _ = table([R1 - 5], R1)
    a1, d1 = new(R1, 64), new(R1, 64)
    n1, n2 = fre.moe_grouped_gemm_float_workspace_bytes(1, R1, 64, 64), fre.moe_layer_norm_workspace_bytes(T, H)
    assert n1 > 0 and n2 > 0
    ws1, ws2 = z(n1, dt=torch.uint8), z(n2, dt=torch.uint8)

    def run(stream=None):
        s = dict(stream=stream)
        fre.moe_grouped_gemm_float(a, w, o, c, out["c"], st, **s)
        fre.moe_grouped_gemm_float_grad_rows(dc, w, o, c, out["da"], st, **s)
        fre.moe_grouped_gemm_float_grad_weights(d1, a1, o1, c1, out["dw"], ws1, st, **s)
        fre.moe_grouped_gemm_float_grad_weights(dc, a, o, c, out["dw2"], z(1, dt=torch.uint8), st, **s)
        fre.moe_gated_act(h, o, c, out["q"], st, **s)
        fre.moe_gated_act_grad(a, h, o, c, out["dh"], st, **s)
        fre.moe_layer_norm(x, wt, None, 1e-5, out["y"], out["mean"], out["rstd"], **s)
        fre.moe_layer_norm_grad(x, x, wt, out["mean"], out["rstd"], out["dx"], out["dwt"], None, ws2, **s)
        fre.moe_route_tokens(l, out["idx"], out["tw"], st, **s)
        fre.moe_route_tokens_grad(l, out["idx"], out["tw"], out["dl"], st, **s)
    return run, out, (a, x, l, dc, h)


def test_streams_and_graphs_at_once(gpu):
    """Two sets of calls on two streams at once, then as two graphs that are
    replayed at once, on changed inputs, give what each gives alone."""
    sets = [calls(1), calls(2)]
    alone = []
    for run, out, _ in sets:
        run()
        torch.cuda.synchronize()
        alone.append({k: v.clone() for k, v in out.items()})
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (run, out, _), s in zip(sets, streams):
            for v in out.values():
                v.zero_()
        torch.cuda.synchronize()
        for (run, _, _), s in zip(sets, streams):
            run(s)
        torch.cuda.synchronize()
        for want, (_, out, _) in zip(alone, sets):
            for k in want:
                assert torch.equal(want[k], out[k]), k
    graphs = []
    for run, _, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for i in range(4):
        for _, _, inputs in sets:
            for v in inputs:
                v.mul_(0.5 + 0.25 * i)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        got = [{k: v.clone() for k, v in out.items()} for _, out, _ in sets]
        for (run, out, _), g in zip(sets, got):
            run()
            torch.cuda.synchronize()
            for k in g:
                assert torch.equal(g[k], out[k]), (i, k)


def test_every_tile_rule(gpu):
    """One product of every kernel that the sizes choose, each with segments
    that end inside its tiles, against 64 bits."""
    for counts, N, K in (([1], 264, 520), ([3, 9, 16], 7168, 136), ([5] * 40, 1032, 264), ([700] * 3, 2056, 1032),
                         ([130, 90, 200, 61], 776, 392), ([300, 511, 257, 129], 2048, 264),
                         ([2000, 1900], 4096, 136), ([1500] * 2, 264, 7176)):
        for dt in (BF16, torch.float16):
            c, o, R, seg = table(counts, sum(-(-n // 128) * 128 for n in counts))
            a, w, dc, st = normal(R, K, dtype=dt), normal(len(counts), N, K, dtype=dt) * 0.1, normal(R, N, dtype=dt), status()
            out, da = torch.zeros(R, N, device="cuda", dtype=dt), torch.zeros(R, K, device="cuda", dtype=dt)
            dw = torch.zeros(len(counts), N, K, device="cuda", dtype=dt)
            ws = torch.empty(max(1, fre.moe_grouped_gemm_float_workspace_bytes(len(counts), R, N, K)),
                             dtype=torch.uint8, device="cuda")
            fre.moe_grouped_gemm_float(a, w, o, c, out, st)
            fre.moe_grouped_gemm_float_grad_rows(dc, w, o, c, da, st)
            fre.moe_grouped_gemm_float_grad_weights(dc, a, o, c, dw, ws, st)
            half = torch.finfo(dt).eps / 2
            tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
            for e, (b, n) in enumerate(seg):
                A, W, D = a[b:n].double(), w[e].double(), dc[b:n].double()
                for got, ref, mag, L in ((out[b:n], A @ W.t(), A.abs() @ W.abs().t(), K),
                                         (da[b:n], D @ W, D.abs() @ W.abs(), N),
                                         (dw[e], D.t() @ A, D.abs().t() @ A.abs(), n - b)):
                    off = (got.double() - ref).abs() - ((L + 2) * U * mag + half * ref.abs() + tiny)
                    assert (off <= 0).all(), (counts, N, K, dt, e, float(off.max()))
            log(f"tiles {counts} {N} {K} {dt}")


def test_no_tokens(gpu):
    """The block on no token at all: empty outputs, zero gradients of weights."""
    m = fre.RoutedExperts(E=4, H=64, I=32, K=2)
    x = torch.zeros(0, 64, device="cuda", dtype=BF16, requires_grad=True)
    out = m(x)
    assert out.shape == (0, 64)
    out.sum().backward()
    assert x.grad.shape == (0, 64)
    for k, v in m.named_parameters():
        assert v.grad is not None and (v.grad == 0).all(), k
