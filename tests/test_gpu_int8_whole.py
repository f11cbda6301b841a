"""GPU tests of the 8-bit integer products and the quantiser over their whole
outputs and at their largest sizes: every valid row of every grouped shape
against exact sums (float64 on the device; the integer sums are below 2^31),
gathered rows from a source that fills its descriptor, and the longest row.

Tolerances are those of the sampled tests: the sum, the product of the scales
and the multiplication are rounded to fp32 once each, the output once."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.gpu_util import log
from tests.test_gpu_int8 import FEW_EACH, GROUPED, TYPES, U, codes, i32, scales, segments

pytestmark = pytest.mark.gpu


def check_all(got, a, sa, w, sw, what):
    """Every element of got [M, N] against a [M, K], w [N, K], on the device."""
    if not got.shape[0]:
        return
    ref = (a.double() @ w.double().t().contiguous()) * sa.double()[:, None] * sw.double()
    f = torch.finfo(got.dtype)
    half = 0.0 if got.dtype == torch.float32 else f.eps / 2
    assert ref.abs().max() < f.max
    tol = (4 * U * (1 + half) + half) * ref.abs() + f.smallest_normal * f.eps / 2
    worst = float(((got.double() - ref).abs() / tol).max())
    log(f"{what}: {got.numel()} values, largest error over tolerance {worst:.2f}")
    assert worst <= 1, what          # (a NaN fails as well)


SHAPES = GROUPED + FEW_EACH


@pytest.mark.parametrize("gather", [False, True], ids=["plain", "gather"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s[:3])) + f"_{i}" for i, s in enumerate(SHAPES)])
def test_grouped_every_row(gpu, shape, gather):
    E, N, K = shape[:3]
    g, counts, offsets, R = segments(shape)
    w, sw = codes(g, E, N, K).cuda(), scales(g, E, N).cuda()
    tab = (torch.from_numpy(offsets).cuda(), torch.from_numpy(counts).cuda())
    if gather:
        T = max(1, R // 2)
        x, sx = codes(g, T, K).cuda(), scales(g, T).cuda()
        src = torch.from_numpy(g.integers(-1, T, R)).cuda()
        src[::17] = T + 1
        known = (src >= 0) & (src < T)
        at = src.clamp(0, T - 1)
        a, sa = x[at] * known[:, None], sx[at] * known
        src = src.int()
    else:
        a, sa = codes(g, R, K).cuda(), scales(g, R).cuda()
    valid = torch.zeros(R, dtype=torch.bool, device="cuda")
    for b, n in zip(offsets, counts):
        valid[int(b):int(b) + int(n)] = True
    for name, t in TYPES.items():
        c, st = torch.full((R, N), float("nan"), dtype=t, device="cuda"), i32(1)
        if gather:
            fre.moe_grouped_gemm_int8_gather(x, sx, src, w, sw, *tab, c, st)
        else:
            fre.moe_grouped_gemm_int8(a, sa, w, sw, *tab, c, st)
        for e in range(E):
            b, n = int(offsets[e]), int(counts[e])
            check_all(c[b:b + n], a[b:b + n], sa[b:b + n], w[e], sw[e], f"{shape[:3]} {name} expert {e}")
        assert c[~valid].isnan().all() and int(st) == 0


LIMIT = 0x7ffff000      # T * K of a gathered call

# (E, N, counts): the few-row kernels, each height of staged tiles, the walking
# tiles (K a multiple of 128) and the others
FAR = [(2, 272, [5, 9]), (1, 4096, [30]), (2, 272, [70, 33]), (3, 4096, [300, 1, 420]), (2, 4096, [1200, 1190]),
       (2, 4096, [2900, 2700])]


@pytest.fixture(scope="module", params=[4096, 4112, 144], ids=["K4096", "K4112", "K144"])
def far_source(request):
    K = request.param
    T = LIMIT // K
    torch.manual_seed(K)
    x = torch.randint(-128, 128, (T, K), dtype=torch.int8, device="cuda")
    sx = torch.rand(T, device="cuda") / 64 + 0.005
    yield x, sx
    del x, sx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("shape", FAR, ids=["x".join(map(str, s[2])) for s in FAR])
def test_gather_from_a_full_descriptor(gpu, far_source, shape):
    """Source rows up to the last one that a call may have, next to rows
    without a source: byte offsets up to 2^31, beside the out-of-range one."""
    x, sx = far_source
    T, K = x.shape
    E, N, counts = shape
    torch.manual_seed(sum(counts))
    w = torch.randint(-128, 128, (E, N, K), dtype=torch.int8, device="cuda")
    sw = torch.rand(E, N, device="cuda") / 64 + 0.005
    R = sum(counts)
    offsets = [sum(counts[:e]) for e in range(E + 1)]
    src = torch.randint(T - T // 8, T, (R,), device="cuda")
    edge = torch.tensor([T - 1, 0, -1, T - 2, T, 2 ** 31 - 1, -2 ** 31, T - 1], device="cuda")
    for b, n in zip(offsets, counts):
        m = min(n, 8)
        src[b:b + m], src[b + n - m:b + n] = edge[:m], edge.flip(0)[:m]
    known = (src >= 0) & (src < T)
    at = src.clamp(0, T - 1)
    a, sa = x[at] * known[:, None], sx[at] * known
    for name, t in TYPES.items():
        c, st = torch.full((R, N), float("nan"), dtype=t, device="cuda"), i32(1)
        fre.moe_grouped_gemm_int8_gather(x, sx, src.int(), w, sw, torch.tensor(offsets, dtype=torch.int32).cuda(),
                                         torch.tensor(counts, dtype=torch.int32).cuda(), c, st)
        assert (c[~known] == 0).all() and int(st) == 0
        for e in range(E):
            b, n = offsets[e], counts[e]
            check_all(c[b:b + n], a[b:b + n], sa[b:b + n], w[e], sw[e], f"far {K} {shape} {name} expert {e}")


def test_quantize_longest_row(gpu):
    """One row of the most values a call takes: its largest magnitude near the
    end, codes exact throughout, nothing outside the row written."""
    n = 0x7ffff000
    torch.manual_seed(1)
    x = torch.randn(1, n, device="cuda", dtype=torch.bfloat16)
    x[0, n - 3] = -23.5                     # past every normal value of 2^31
    buf = torch.full((n + 128,), 99, dtype=torch.int8, device="cuda")
    q, s = buf[64:-64].view(1, n), torch.zeros(1, device="cuda")
    fre.moe_quantize_int8(x, q, s)
    want = torch.tensor(23.5) / 127
    assert s.cpu()[0] == want
    for b in range(0, n, 1 << 27):
        v = x[0, b:b + (1 << 27)].double().div_(want.double().cuda()).round_()
        assert torch.equal(q[0, b:b + (1 << 27)], v.to(torch.int8)), b
    assert (buf[:64] == 99).all() and (buf[-64:] == 99).all()


@pytest.mark.parametrize("K", [128, 144])
@pytest.mark.parametrize("shape", FAR, ids=["x".join(map(str, s[2])) for s in FAR])
def test_gather_with_non_finite_scales(gpu, shape, K):
    """A row without a source is a row of zeros with the scale 0: NaN in a
    channel whose scale is not finite, 0 in all others.  Other rows take the
    channel's NaN, or its infinity times their sum."""
    E, N, counts = shape
    torch.manual_seed(K + N)
    T, R = 60, sum(counts)
    x, sx = torch.randint(1, 128, (T, K), dtype=torch.int8, device="cuda"), torch.rand(T, device="cuda") + 0.5
    w, sw = torch.randint(1, 128, (E, N, K), dtype=torch.int8, device="cuda"), torch.rand(E, N, device="cuda") + 0.5
    sw[:, 3], sw[:, N - 1] = float("nan"), float("inf")
    src = torch.randint(-1, T, (R,), device="cuda")
    src[0], src[R - 1], src[R // 2] = -1, T, 5
    known = (src >= 0) & (src < T)
    offsets = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32).cuda()
    finite = torch.ones(N, dtype=torch.bool, device="cuda")
    finite[3], finite[N - 1] = False, False
    for name, t in TYPES.items():
        c, st = torch.full((R, N), 77.0, dtype=t, device="cuda"), i32(1)
        fre.moe_grouped_gemm_int8_gather(x, sx, src.int(), w, sw, offsets,
                                         torch.tensor(counts, dtype=torch.int32).cuda(), c, st)
        assert c[:, 3].isnan().all() and c[~known][:, N - 1].isnan().all()
        assert (c[known][:, N - 1] == float("inf")).all()
        assert (c[~known][:, finite] == 0).all() and (c[known][:, finite] > 0).all() and int(st) == 0


def test_act_of_far_gates(gpu):
    """Down to -87.3 as accurate as any gate ((|g| + 6) 2^-23, as in the
    activation's other test), below that 0; infinite values make the row NaN."""
    gates = torch.tensor([-80.0, -86, -87, -87.25, -87.5, -89, -104, -1e30, 88, 1e4, float("-inf"), float("inf")])
    n, I = gates.numel(), 16
    h = torch.cat([gates[:, None].expand(n, I), torch.full((n, I), 1e30)], dim=1).contiguous()
    q, s, st = torch.full((n, I), 99, dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda"), i32(1)
    fre.moe_act_requant_int8(h.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                             torch.tensor([n], dtype=torch.int32).cuda(), q, s, st)
    q, s, g = q.cpu().double(), s.cpu().double(), gates.double()
    near = (g > -87.3) & (g < 1e5)
    v = (g / (1 + torch.exp(-g)) * 1e30)[near]
    rel = (g[near].abs() + 6) * 2.0 ** -23
    assert (q[near] == 127 * v.sign()[:, None]).all()
    assert ((s[near] - v.abs() / 127).abs() <= 2 * rel * s[near]).all()
    far = (g <= -87.3) & g.isfinite()
    assert (q[far] == 0).all() and (s[far] == 1).all()
    assert s[g.isinf()].isnan().all() and (q[g.isinf()] == 0).all() and int(st) == 0
