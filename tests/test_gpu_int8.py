"""GPU tests of the products in 8-bit integers: quantising rows, dense and
grouped products, the gated activation, the linear and the layer, against
64-bit arithmetic on the CPU.

Tolerances count roundings: the integer sums are exact, so an output is
float(sum) (one fp32 rounding), times the product of two scales (one), the
multiplication (one) and, in 16 bits, one rounding of half a step more."""

import numpy as np
import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


def i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def codes(g, *shape):
    return torch.from_numpy(g.integers(-128, 128, shape, dtype=np.int64).astype(np.int8))


def scales(g, *shape):
    return torch.from_numpy(g.uniform(0.5, 2, shape).astype(np.float32) / 64)


def check(got, a, sa, w, sw, what):
    """got against the 64-bit product of codes a [M, K] and w [N, K]."""
    ref = (a.double() @ w.double().T) * sa.double()[:, None] * sw.double()
    f = torch.finfo(got.dtype)
    half = 0.0 if got.dtype == torch.float32 else f.eps / 2
    fits = ref.abs() < f.max
    tol = (4 * U * (1 + half) + half) * ref.abs() + f.smallest_normal * f.eps / 2
    d = (got.double().cpu() - ref).abs()
    log(f"{what}: largest error over tolerance {float((d / tol)[fits].max()) if d.numel() else 0:.2f}")
    assert fits.all() and (d <= tol).all(), what


def exact_codes(v64, s):
    """The integers nearest v / s, ties to even, for fp32 scales s."""
    return torch.round(v64 / s.double()[..., None])


def exact_scale(amax):
    s = torch.clamp((amax.float() / 127), min=2.0 ** -126)
    return torch.where(amax == 0, torch.ones(()), s)


# ------------------------------------------------------------- quantiser
def test_quantize_rows(gpu):
    """Every length class (in registers, past them), type and magnitude; the
    codes and scales are exact."""
    g = np.random.default_rng(0)
    for cols in (16, 32, 48, 1000 * 16, 2048, 7168, 8192, 8208):
        for name, dt in TYPES.items():
            mag = 10.0 ** g.uniform(-4, 4, (5, 1))
            x = torch.from_numpy(g.standard_normal((5, cols)) * mag).to(dt)
            q, s = torch.zeros(5, cols, dtype=torch.int8, device="cuda"), torch.zeros(5, device="cuda")
            fre.moe_quantize_int8(x.cuda(), q, s)
            want = exact_scale(x.double().abs().amax(1))
            assert torch.equal(s.cpu(), want), (cols, name)
            assert torch.equal(q.cpu().double(), exact_codes(x.double(), want)), (cols, name)


def test_quantize_ties_zeros_and_extremes(gpu):
    f = torch.finfo(torch.float32)
    n = torch.arange(-126, 126).float() + 0.5
    rows = torch.zeros(9, 256)
    rows[0, :252], rows[0, 255] = n, 127.0                      # ties: scale 1
    rows[1, :252], rows[1, 255] = n * 2.0 ** 60, 127 * 2.0 ** 60
    rows[2, :252], rows[2, 255] = n * 3, 381.0                  # scale 3
    rows[4, :252], rows[4, 255] = n * 2.0 ** -126, 127 * 2.0 ** -126
    rows[5, 3], rows[5, 7] = f.smallest_normal * 2.0 ** -23, -f.smallest_normal * 2.0 ** -23
    rows[6, 0], rows[6, 1] = f.max, -f.max
    rows[7, ::2], rows[7, 1::2] = 1.0, -1.0
    rows[8] = torch.nextafter(n.new_full((256,), 0.5), n.new_zeros(())) * 2   # just under 1
    rows[8, 0] = 254.0                                         # scale 2: just under a tie
    q, s = torch.zeros(9, 256, dtype=torch.int8, device="cuda"), torch.zeros(9, device="cuda")
    fre.moe_quantize_int8(rows.cuda(), q, s)
    want = exact_scale(rows.double().abs().amax(1))
    assert torch.equal(s.cpu(), want)
    assert torch.equal(q.cpu().double(), exact_codes(rows.double(), want))
    assert s[3] == 1 and (q[3] == 0).all()
    # random values within a few last places of every border
    g = np.random.default_rng(1)
    s32 = np.float32(g.uniform(1, 2, 4000))
    x = np.zeros((4000, 16), np.float32)
    for j in range(15):
        k = g.integers(-126, 126, 4000) + 0.5
        x[:, j] = (s32.astype(np.float64) * k).astype(np.float32) * (1 + g.integers(-2, 3, 4000) * 2.0 ** -23)
    x[:, 15] = s32 * np.float32(127)
    x = torch.from_numpy(x)
    q, s = torch.zeros(4000, 16, dtype=torch.int8, device="cuda"), torch.zeros(4000, device="cuda")
    fre.moe_quantize_int8(x.cuda(), q, s)
    want = exact_scale(x.double().abs().amax(1))
    assert torch.equal(s.cpu(), want) and torch.equal(q.cpu().double(), exact_codes(x.double(), want))


@pytest.mark.parametrize("dt", list(TYPES))
def test_quantize_non_finite(gpu, dt):
    """A row with an infinity or a NaN: scale NaN, codes 0; others as ever."""
    x = torch.randn(6, 64).to(TYPES[dt])
    x[1, 5], x[3, 0], x[4, 63] = float("inf"), float("nan"), float("-inf")
    q, s = torch.ones(6, 64, dtype=torch.int8, device="cuda"), torch.ones(6, device="cuda")
    fre.moe_quantize_int8(x.cuda(), q, s)
    bad = torch.tensor([False, True, False, True, True, False])
    assert torch.equal(s.cpu().isnan(), bad) and (q.cpu()[bad] == 0).all()
    ok = x[~bad].double()
    want = exact_scale(ok.abs().amax(1))
    assert torch.equal(s.cpu()[~bad], want) and torch.equal(q.cpu()[~bad].double(), exact_codes(ok, want))


# ------------------------------------------------------------- dense
DENSE = [(1, 16, 16), (1, 128, 128), (2, 4096, 7168), (3, 48, 80), (16, 272, 144), (17, 272, 144),
         (33, 7168, 2048), (64, 144, 4112), (65, 144, 4112), (130, 144, 4112), (300, 256, 256),
         (257, 528, 1040), (700, 1040, 7168), (1500, 768, 16), (8448, 1296, 272), (8200, 4096, 384),
         (32, 16400, 48), (31, 6160, 80), (96, 7168, 2048), (200, 7168, 272), (1000, 4096, 400), (2400, 4096, 144),
         (2048, 4096, 1040), (2048, 4112, 128), (40, 16384, 656), (129, 80, 896), (16640, 4096, 256), (16400, 4112, 128),
         (12300, 4096, 144)]


@pytest.mark.parametrize("shape", DENSE, ids=["x".join(map(str, s)) for s in DENSE])
def test_gemm(gpu, shape):
    M, N, K = shape
    g = np.random.default_rng([2, *shape])
    a, w, sa, sw = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    d = [v.cuda() for v in (a, sa, w, sw)]
    pick = np.unique(np.r_[0, M - 1, g.integers(0, M, 60)])     # rows that the CPU checks
    for name, t in TYPES.items():
        c = torch.full((M + 2, N), 77.0, dtype=t, device="cuda")
        fre.moe_gemm_int8(*d, c[1:-1])
        assert (c[0] == 77).all() and (c[-1] == 77).all(), "wrote past its rows"
        check(c[1:-1].cpu()[pick], a[pick], sa[pick], w, sw, f"gemm {shape} {name}")
        ref = (d[0].float() @ d[2].float().T) * (d[1][:, None] * d[3])      # every element
        assert ((c[1:-1].float() - ref).abs() <= 0.01 * ref.abs() + 0.5).all()


def test_gemm_largest_sum(gpu):
    """-128 times -128 over the largest K: 2^31 - 262,144 does not overflow."""
    K = 131056
    a = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((16, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = torch.ones(16, device="cuda")
    c = torch.zeros(3, 16, device="cuda")
    fre.moe_gemm_int8(a, one[:3].contiguous(), w, one, c)
    assert (c[:, 0] == 128 * 128 * K).all() and (c[:, 1] == -128 * 127 * K).all()


# ------------------------------------------------------------- grouped
# (E, N, K, counts or None for random, gaps between segments, rows left over)
GROUPED = [(1, 16, 16, [1], 0, 0), (4, 128, 256, [3, 0, 130, 1], 5, 7), (3, 272, 1040, [64, 65, 1], 1, 0),
           (8, 4096, 512, [0, 1, 16, 17, 33, 48, 100, 128], 0, 30), (2, 528, 144, [300, 257], 127, 1),
           (70, 64, 48, None, 0, 3), (300, 32, 32, None, 2, 0), (3, 4096, 400, [2900, 1, 2700], 60, 0),
           (2, 784, 7168, [513, 700], 0, 0), (16, 4096, 4112, [40, 0, 64, 65, 128, 1, 17, 90] * 2, 3, 0),
           (40, 2064, 272, [20, 33, 0, 1, 31] * 8, 0, 0), (4, 4096, 256, [600, 640, 580, 700], 10, 0),
           (3, 1040, 144, [300, 200, 129], 0, 5), (3, 4096, 384, [2900, 1, 2700], 60, 0),
           (3, 4096, 128, [5900, 0, 6100], 1, 9), (70, 256, 128, [260] * 70, 0, 0)]


def segments(shape):
    E, N, K, counts, gap, extra = shape
    g = np.random.default_rng([3, E, N, K])
    counts = np.array(counts if counts else g.integers(0, 9, E), np.int32)
    offsets = np.r_[0, np.cumsum(counts + gap)].astype(np.int32)
    return g, counts, offsets, int(offsets[-1]) + extra


@pytest.mark.parametrize("gather", [False, True], ids=["plain", "gather"])
@pytest.mark.parametrize("shape", GROUPED, ids=["x".join(map(str, s[:3])) for s in GROUPED])
def test_grouped(gpu, shape, gather):
    """Every valid row, and no other, is written; an expert without rows, odd
    segment starts, rows without a source."""
    E, N, K = shape[:3]
    g, counts, offsets, R = segments(shape)
    w, sw = codes(g, E, N, K), scales(g, E, N)
    tab = (torch.from_numpy(offsets).cuda(), torch.from_numpy(counts).cuda())
    T = 50
    if gather:
        src = g.integers(0, T, R).astype(np.int32)
        src[g.random(R) < 0.1] = -1
        src[g.random(R) < 0.05] = T + 3
        x, sx = codes(g, T, K), scales(g, T)
        known = torch.from_numpy((src >= 0) & (src < T))
        at = torch.from_numpy(np.clip(src, 0, T - 1)).long()
        a = torch.where(known[:, None], x[at], torch.zeros((), dtype=torch.int8))
        sa = torch.where(known, sx[at], torch.zeros(()))
    else:
        a, sa = codes(g, R, K), scales(g, R)
    for name, t in TYPES.items():
        c, st = torch.full((R, N), 77.0, dtype=t, device="cuda"), i32(1)
        if gather:
            fre.moe_grouped_gemm_int8_gather(x.cuda(), sx.cuda(), torch.from_numpy(src).cuda(), w.cuda(),
                                             sw.cuda(), *tab, c, st)
        else:
            fre.moe_grouped_gemm_int8(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), *tab, c, st)
        got, written = c.cpu(), torch.zeros(R, dtype=torch.bool)
        for e in range(E):
            b, n = offsets[e], counts[e]
            written[b:b + n] = True
            if n:
                rows = np.unique(np.r_[b, b + n - 1, g.integers(b, b + n, 40)])
                check(got[rows], a[rows], sa[rows], w[e], sw[e], f"grouped {shape[:3]} {name} expert {e}")
        assert (got[~written] == 77).all() and int(st) == 0
        assert not (got[written] == 77).all(-1).any()


# Few rows with many channels, or of many experts: the tiles' borders.
FEW = [(9, 7184, 272), (7, 7184, 1040), (3, 16400, 144), (2, 33040, 1040), (16, 16400, 2064), (20, 16384, 144),
       (5, 40016, 256), (30, 8208, 144), (64, 16400, 144), (100, 33040, 80)]


@pytest.mark.parametrize("shape", FEW, ids=["x".join(map(str, s)) for s in FEW])
def test_gemm_of_few_rows(gpu, shape):
    test_gemm(gpu, shape)


FEW_EACH = [(20, 1040, 144, None, 1, 0), (40, 1040, 144, None, 0, 2), (520, 144, 2064, None, 0, 3),
            (30, 272, 144, [16, 0, 9] * 10, 0, 0), (24, 272, 2064, [2, 1, 0] * 8, 0, 1), (70, 1040, 144, [64, 33] * 35, 0, 0),
            (70, 1040, 128, [70, 96] * 35, 1, 0), (40, 1040, 144, [150, 190, 129, 0] * 10, 3, 0),
            (40, 1040, 256, [150, 250, 129, 256] * 10, 0, 9)]


@pytest.mark.parametrize("gather", [False, True], ids=["plain", "gather"])
@pytest.mark.parametrize("shape", FEW_EACH, ids=["x".join(map(str, s[:3])) for s in FEW_EACH])
def test_grouped_of_few_rows(gpu, shape, gather):
    test_grouped(gpu, shape, gather)


@pytest.mark.parametrize("R", [300, 5000])
def test_grouped_clipped_and_corrupt_tables(gpu, R):
    """Counts past their segment or the buffer are clipped; a table that is
    none is reported, and no row outside the buffer is touched."""
    N, K, E = 256, 128, 3
    g = np.random.default_rng(R)
    a, sa, w, sw = codes(g, R, K), scales(g, R), codes(g, E, N, K), scales(g, E, N)
    d = [v.cuda() for v in (a, sa, w, sw)]
    for offs, counts, bad in (([0, 100, 200, R], [150, 20, 10 ** 6], 0), ([0, 100, 100, R + 900], [100, 50, R + 5], 0),
                              ([0, 100, 50, R], [10, 10, 10], fre.ERR_BAD_INDEX),
                              ([-8, 100, 200, R], [50, -1, 10], fre.ERR_BAD_INDEX)):
        c, st = torch.full((R + 2, N), 77.0, device="cuda"), i32(1)
        fre.moe_grouped_gemm_int8(*d, torch.tensor(offs, dtype=torch.int32).cuda(),
                                  torch.tensor(counts, dtype=torch.int32).cuda(), c[1:-1], st)
        assert int(st) == bad and (c[0] == 77).all() and (c[-1] == 77).all()
        if not bad:
            for e in range(E):
                lo, hi = offs[e], min(offs[e] + counts[e], offs[e + 1], R)
                check(c[1:-1][lo:hi].cpu(), a[lo:hi], sa[lo:hi], w[e], sw[e], f"clipped expert {e}")


# ------------------------------------------------------------- activation
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("I", [16, 48, 2048, 8208])
def test_act(gpu, I, dt):
    """Codes are the nearest integers of a value whose fp32 error is at most
    (|g| + 6) 2^-23 of itself: the exponent's argument is off by half a step
    of |g| / ln 2, the two hardware functions, the sum and the two products
    by a step or less each.  The scale's maximum has the same error."""
    g = np.random.default_rng([4, I])
    counts, offsets, R = np.array([3, 0, 9], np.int32), np.array([0, 5, 5, 16], np.int32), 18
    h = torch.from_numpy(g.standard_normal((R, 2 * I)) * 3).to(TYPES[dt])
    h[1] = 0
    h[6, 0] = float("nan")
    q = torch.full((R, I), 99, dtype=torch.int8, device="cuda")
    s = torch.full((R,), 99.0, device="cuda")
    st = i32(1)
    fre.moe_act_requant_int8(h.cuda(), torch.from_numpy(offsets).cuda(), torch.from_numpy(counts).cuda(), q, s, st)
    q, s, h64 = q.cpu(), s.cpu(), h.double()
    live = [0, 1, 2, 5, 6, 7, 8, 9, 10, 11, 12, 13]
    rest = [r for r in range(R) if r not in live]
    assert (q[rest] == 99).all() and (s[rest] == 99).all() and int(st) == 0
    assert s[6].isnan() and (q[6] == 0).all() and s[1] == 1 and (q[1] == 0).all()
    for r in live:
        if r == 6:
            continue
        gate, up = h64[r, :I], h64[r, I:]
        v = gate / (1 + torch.exp(-gate)) * up
        rel = (gate.abs().max() + 6) * 2.0 ** -23
        if r != 1:
            assert abs(s[r] - v.abs().max() / 127) <= 2 * rel * s[r]
        sd = s[r].double()
        assert ((q[r].double() * sd - v).abs() <= sd * (0.5 + 128 * rel) * (1 + 1e-12)).all()
        assert q[r].abs().max() <= 127


def test_act_corrupt_table(gpu):
    h = torch.randn(8, 64, device="cuda")
    q, s, st = torch.zeros(8, 32, dtype=torch.int8, device="cuda"), torch.zeros(8, device="cuda"), i32(1)
    fre.moe_act_requant_int8(h, torch.tensor([0, 6, 3], dtype=torch.int32).cuda(),
                             torch.tensor([2, 2], dtype=torch.int32).cuda(), q, s, st)
    assert int(st) == fre.ERR_BAD_INDEX


@pytest.mark.parametrize("rows,I,dt", [(66000, 2048, "bf16"), (16500, 8208, "f16"), (66000, 1040, "f32"),
                                       (8300, 8208, "f32")])
def test_act_of_many_rows(gpu, rows, I, dt):
    """An h larger than the caches is read past them, with the same bits as
    its parts; rows behind the last segment are left as they were."""
    h = torch.randn(rows, 2 * I, device="cuda").to(TYPES[dt])
    end = rows - 7

    def act(lo, hi):
        q = torch.full((hi - lo, I), 99, dtype=torch.int8, device="cuda")
        s, st = torch.full((hi - lo,), 99.0, device="cuda"), i32(1)
        fre.moe_act_requant_int8(h[lo:hi], torch.tensor([0, hi - lo], dtype=torch.int32).cuda(),
                                 torch.tensor([min(hi, end) - lo], dtype=torch.int32).cuda(), q, s, st)
        assert int(st) == 0
        return q, s

    q, s = act(0, rows)
    cuts = [0, rows // 5, rows // 2, rows * 3 // 4, rows]
    parts = [act(lo, hi) for lo, hi in zip(cuts, cuts[1:])]
    assert torch.equal(q, torch.cat([p[0] for p in parts])) and torch.equal(s, torch.cat([p[1] for p in parts]))
    assert (q[end:] == 99).all() and (s[end:] == 99).all()


# ------------------------------------------------------------- linear
LINEAR = [(1, 16, 16), (1, 4096, 7168), (2, 256, 128), (4, 272, 400), (5, 144, 2064), (8, 512, 7168), (16, 1040, 1040),
          (17, 64, 64), (40, 7168, 2048), (96, 528, 2048), (300, 272, 1040), (1, 48, 20000), (3, 32, 131056),
          (4, 16, 15344), (1, 32, 61424), (1, 32, 61440), (3, 272, 208)]


@pytest.mark.parametrize("shape", [(1, 12288, 256), (1, 12304, 256), (3, 40016, 144), (17, 40016, 48)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_of_many_channels(gpu, shape):
    """Either side of the channels that one launch takes."""
    test_linear(gpu, shape, "bf16")


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("shape", LINEAR, ids=["x".join(map(str, s)) for s in LINEAR])
def test_linear(gpu, shape, dt):
    """Equal to the quantiser followed by the product, bit for bit, and near
    the 64-bit product of the exact codes; a NaN stays in its own row."""
    M, N, K = shape
    g = np.random.default_rng([5, *shape])
    x = torch.from_numpy(g.standard_normal((M, K))).to(TYPES[dt])
    if M > 2:
        x[1, K // 2] = float("nan")
        x[2] = 0
    w, sw = codes(g, N, K), scales(g, N) / 64
    xd, wd, swd = x.cuda(), w.cuda(), sw.cuda()
    c = torch.full((M, N), 77.0, dtype=TYPES[dt], device="cuda")
    ws = torch.full((fre.moe_linear_int8_workspace_bytes(M, K) + 64,), 0xa5, dtype=torch.uint8, device="cuda")
    fre.moe_linear_int8(xd, wd, swd, c, ws[:-64])
    assert (ws[-64:] == 0xa5).all()
    q, s = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    two = torch.zeros_like(c)
    fre.moe_quantize_int8(xd, q, s)
    fre.moe_gemm_int8(q, s, wd, swd, two)
    fine = torch.ones(M, dtype=torch.bool)
    if M > 2:
        fine[1] = False
        assert c[1].isnan().all() and two[1].isnan().all() and (c[2] == 0).all()
    assert torch.equal(c.cpu()[fine], two.cpu()[fine])
    s64 = exact_scale(x[fine].double().abs().amax(1))
    check(c.cpu()[fine], exact_codes(x[fine].double(), s64), s64, w, sw, f"linear {shape} {dt}")


@pytest.mark.parametrize("M", [1, 3, 20, 100, 700])
def test_linear_captured(gpu, M):
    """Replayed with other inputs and with eager calls between."""
    N, K = 528, 1040
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    sw = torch.rand(N, device="cuda") / 100
    x, c = torch.randn(M, K, device="cuda").bfloat16(), torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(fre.moe_linear_int8_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    fre.moe_linear_int8(x, w, sw, c, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fre.moe_linear_int8(x, w, sw, c, ws)
    for _ in range(4):
        x.copy_(torch.randn(M, K, device="cuda"))
        fre.moe_linear_int8(x, w, sw, c, ws)
        want = c.clone()
        c.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)


def test_two_linears_at_once(gpu):
    """On two streams, with workspaces of their own, each repeated."""
    N, K, M = 4096, 2048, 300
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    sw = torch.rand(N, device="cuda") / 100
    xs = [torch.randn(M, K, device="cuda").half() for _ in range(2)]
    n = fre.moe_linear_int8_workspace_bytes(M, K)
    wss = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cs = [torch.zeros(6, M, N, dtype=torch.float16, device="cuda") for _ in range(2)]
    want = []
    for x, ws in zip(xs, wss):
        c = torch.zeros(M, N, dtype=torch.float16, device="cuda")
        fre.moe_linear_int8(x, w, sw, c, ws)
        want.append(c)
    torch.cuda.synchronize()
    for i in range(6):
        for x, ws, c, s in zip(xs, wss, cs, streams):
            fre.moe_linear_int8(x, w, sw, c[i], ws, stream=s)
    torch.cuda.synchronize()
    for c, v in zip(cs, want):
        assert all(torch.equal(c[i], v) for i in range(6))


# ------------------------------------------------------------- the layer
@pytest.mark.parametrize("gather", [True, False], ids=["gather", "copy"])
@pytest.mark.parametrize("layout", [0, 1], ids=["contiguous", "masked"])
def test_layer(gpu, layout, gather):
    """MoELayer(scale_fmt="int8") against its stages in 64 bits.  The stages'
    own codes are compared from the device's own h, as borders move with h's
    bf16 rounding; the output then has y's and its own rounding."""
    E, H, I, T, K = 5, 400, 208, 90, 3
    g = np.random.default_rng(6)
    idx = np.stack([g.permutation(E + 2)[:K] for _ in range(T)]).astype(np.int32)
    idx[idx >= E] = -1
    rows = 64 if layout else int((idx >= 0).sum()) + E * 127
    x, sx = codes(g, T, H), scales(g, T)
    w13, s13, w2, s2 = codes(g, E, 2 * I, H), scales(g, E, 2 * I) / 200, codes(g, E, H, I), scales(g, E, H)
    tw = torch.from_numpy(g.random((T, K)).astype(np.float32))
    layer = fre.MoELayer(E, H, I, T, K, layout, rows, scale_fmt="int8", gather=gather)
    dev = [v.cuda() for v in (torch.from_numpy(idx), x, sx, tw, w13, s13, w2, s2)]
    out = layer.forward(*dev).clone()
    assert int(layer.status) == 0
    slot, src, exp = layer.slot_of.cpu(), layer.row_src.cpu().long(), layer.row_expert.cpu().long()
    live = src >= 0
    assert int(live.sum()) == int((idx >= 0).sum())
    h, q, qs, y = layer.h.cpu(), layer.q2.cpu(), layer.q2_scale.cpu(), layer.y.cpu()
    for e in range(E):
        r = (exp == e) & live
        check(h[r], x[src[r]], sx[src[r]], w13[e], s13[e], f"h {e}")
        check(y[r], q[r], qs[r], w2[e], s2[e], f"y {e}")
    gate, up = h[live].double().split(I, 1)
    v = gate / (1 + torch.exp(-gate)) * up
    rel = (gate.abs().amax(1) + 6) * 2.0 ** -23
    sd = qs[live].double()
    assert ((sd - v.abs().amax(1) / 127).abs() <= 2 * rel * sd).all()
    assert ((q[live].double() * sd[:, None] - v).abs() <= (sd * (0.5 + 128 * rel))[:, None]).all()
    ok = slot >= 0
    terms = (tw.double() * ok)[..., None] * y.double()[slot.clamp(min=0).long()]
    ref = terms.sum(1)
    tol = (K + 1) * U * terms.abs().sum(1) + 2.0 ** -8 * ref.abs() + 1e-38
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    # captured, replayed with other tokens, and with eager work between
    other = codes(g, T, H).cuda()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.forward(*dev)
    for v in (other, x.cuda(), other):
        dev[1].copy_(v)
        want = layer.forward(*dev).clone()
        layer.out.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, want)


# ------------------------------------------------------------- trained tokens
@pytest.mark.parametrize("dt", list(TYPES))
def test_differentiable_routing(gpu, dt):
    """sort_tokens, permute_tokens and combine_tokens around a per-expert
    product, against autograd through the dense 64-bit form."""
    E, T, K, H, t = 4, 70, 2, 72, TYPES[dt]
    g = np.random.default_rng(8)
    idx = np.stack([g.permutation(E + 1)[:K] for _ in range(T)]).astype(np.int32)
    idx[idx >= E] = -1
    x = torch.from_numpy(g.standard_normal((T, H))).to(t)
    wt = torch.from_numpy(g.random((T, K)).astype(np.float32))
    gain = torch.from_numpy(g.standard_normal(E))
    xd, wd = x.cuda().requires_grad_(), wt.cuda().requires_grad_()
    tab = fre.sort_tokens(torch.from_numpy(idx).cuda(), E, 16, layout=1)
    small = int(tab.status)                     # capacity 16: some rows are dropped
    assert small == fre.ERR_OVERFLOW
    tab = fre.sort_tokens(torch.from_numpy(idx).cuda(), E, T * K + 127 * E)
    a = fre.permute_tokens(xd, tab)
    assert (a[tab.row_src < 0] == 0).all()
    y = a * gain.to(t).cuda()[tab.row_expert.clamp(min=0).long()][:, None]
    out = fre.combine_tokens(y, wd, tab)
    c = torch.from_numpy(g.standard_normal((T, H))).to(t)
    out.backward(c.cuda())
    x64, w64 = x.double().requires_grad_(), wt.double().requires_grad_()
    gk = gain.to(t).double()[np.clip(idx, 0, E - 1)] * torch.from_numpy(idx >= 0)
    ref = ((w64 * gk).sum(1))[:, None] * x64
    ref.backward(c.double())
    u = torch.finfo(t).eps / 2 + 8 * U
    mag = (wt.double() * gk.abs()).sum(1)[:, None]
    # y and out are rounded once each; dy, dy * gain and dx once each
    assert ((out.detach().cpu().double() - ref).abs() <= 2.1 * u * mag * x.double().abs() + 1e-7).all()
    assert ((xd.grad.cpu().double() - x64.grad).abs() <= 3.1 * u * mag * c.double().abs() + 1e-7).all()
    mag = gk.abs() * (x.double().abs() * c.double().abs()).sum(1)[:, None]
    assert ((wd.grad.cpu().double() - w64.grad).abs() <= (1.1 * u + 20 * U) * mag + 1e-7).all()


def test_rows_that_are_not_the_tables(gpu):
    idx = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    tab = fre.sort_tokens(idx, 1, 256)
    with pytest.raises(ValueError, match="256"):
        fre.combine_tokens(torch.zeros(255, 4, device="cuda"), torch.ones(3, 1, device="cuda"), tab)
    with pytest.raises(ValueError):
        fre.permute_tokens(torch.zeros(4, 4, device="cuda"), tab)


def test_more_tiles_than_a_launch_holds(gpu):
    """1024 experts of one row with 131,072 channels: past 2^22 tiles of 16."""
    E, N, K = 1024, 131072, 16
    g = np.random.default_rng(9)
    w = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    a, sa, sw = codes(g, E, K), scales(g, E), scales(g, N)
    sws = sw.cuda().expand(E, N).contiguous()
    offs = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    c, st = torch.full((E, N), 77.0, dtype=torch.bfloat16, device="cuda"), i32(1)
    picked = {e: codes(g, N, K) for e in (0, 511, 1023)}
    for e, v in picked.items():
        w[e] = v.cuda()
    fre.moe_grouped_gemm_int8(a.cuda(), sa.cuda(), w, sws, offs, torch.ones(E, dtype=torch.int32, device="cuda"), c, st)
    for e, v in picked.items():
        check(c[e:e + 1].cpu(), a[e:e + 1], sa[e:e + 1], v, sw, f"expert {e}")
    assert int((c != 0).any(1).sum()) == 3 and int(st) == 0


def test_only_one_gradient(gpu):
    """Weights or rows alone; an expanded gradient; a table sorted in between."""
    idx = torch.tensor([[0, 1], [1, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    tab = fre.sort_tokens(idx, 2, 256)
    x, w = torch.randn(3, 10, device="cuda"), torch.rand(3, 2, device="cuda")
    a = fre.permute_tokens(x, tab)
    wr = w.clone().requires_grad_()
    o = fre.combine_tokens(a, wr, tab)
    fre.sort_tokens(idx.flip(0).contiguous(), 2, 256)
    o.sum().backward()
    want = x.double().sum(1)[:, None] * (idx >= 0)
    assert torch.allclose(wr.grad.double(), want, atol=1e-5)
    xr = x.clone().requires_grad_()
    fre.combine_tokens(fre.permute_tokens(xr, tab), w, tab).sum().backward()
    want = (w * (idx >= 0)).sum(1)[:, None].expand(3, 10)
    assert torch.allclose(xr.grad, want, atol=1e-6)
