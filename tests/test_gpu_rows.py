"""GPU tests of tokens sorted by expert and back, with the gradients
(moe_sort_tokens, moe_permute_rows[_grad], moe_combine_rows[_grad]), against
plain 64-bit sums on the CPU.

Tolerances count roundings.  A sum of n terms in fp32 is off by at most
n * 2^-24 of the sum of the terms' magnitudes (one rounding per addition or
fused multiply-add, to first order; the second order is covered by counting
n + 1), and a value rounded to a type t by at most half a step,
finfo(t).eps / 2 of itself, or half the smallest subnormal."""

import numpy as np
import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24

# (T, K, E, H, layout, rows): sizes from one element to several pieces of a
# row, rows shorter than 16 bytes, rows of no multiple of 16 bytes, more picks
# than a wave has halves, buffers too small for every row, and no token at all
SHAPES = [
    (1, 1, 1, 1, 0, 128), (1, 8, 8, 7168, 0, 1024), (3, 2, 2, 5, 0, 256), (64, 2, 4, 256, 0, 636),
    (77, 3, 5, 509, 0, 900), (200, 4, 6, 1000, 1, 40), (33, 8, 9, 7168, 0, 1500),
    (5, 64, 70, 130, 0, 9100), (77, 16, 40, 130, 0, 6000), (78, 17, 40, 40, 0, 6000), (301, 4, 6, 2048, 0, 2000),
    (20, 3, 4, 18000, 0, 600), (130, 5, 300, 9, 1, 3), (19, 2, 3, 4099, 0, 30), (0, 3, 4, 64, 0, 16),
]
IDS = ["x".join(map(str, s)) for s in SHAPES]


def routing(T, K, E, seed=0, none=0.3):
    """Distinct picks per token, some elsewhere (-1), one token with none."""
    g = np.random.default_rng([seed, T, K, E])
    idx = np.full((T, K), -1, np.int32)
    for t in range(T):
        n = min(K, E)
        idx[t, g.permutation(K)[:n]] = g.permutation(E)[:n]
    idx[g.random((T, K)) < none] = -1
    if T > 2:
        idx[T // 2] = -1
    w = g.random((T, K)).astype(np.float32)
    w[idx < 0] = np.nan                     # never used
    return idx, w


def brute_sort(idx, E, layout, align, rows):
    T, K = idx.shape
    R = E * rows if layout else rows
    counts = [int((idx == e).sum()) for e in range(E)]
    offsets = [0]
    for e in range(E):
        offsets.append(offsets[-1] + (rows if layout else -(-counts[e] // align) * align))
    slot_of = np.full((T, K), -1, np.int32)
    src, exp = np.full(R, -1, np.int32), np.full(R, -1, np.int32)
    seen, dropped = [0] * E, False
    for t in range(T):
        for k in range(K):
            e = idx[t, k]
            if 0 <= e < E:
                s = offsets[e] + seen[e]
                if (seen[e] < rows) if layout else (s < R):
                    slot_of[t, k], src[s], exp[s] = s, t, e
                else:
                    dropped = True
                seen[e] += 1
    return (np.array(counts, np.int32), np.array(offsets, np.int32), slot_of, src, exp), dropped


def new_i32(*shape, fill=-7):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def sort(idx, E, layout, align, rows, stream=None):
    """Through the library; outputs start from a value none of them takes."""
    T, K = idx.shape
    R = E * rows if layout else rows
    o = [new_i32(E), new_i32(E + 1), new_i32(T, K), new_i32(R), new_i32(R)]
    ws = torch.full((max(1, fre.moe_layout_workspace_bytes(T, K, E)),), 0xa5, dtype=torch.uint8,
                    device="cuda")
    st = new_i32(1, fill=0)
    fre.moe_sort_tokens(idx, E, layout, align, rows, *o, ws, st, stream)
    return o, st


def values(g, shape, dt, offset=0):
    """Device values of type dt and the same in 64 bits; offset shifts the
    buffer by that many elements off its allocation."""
    n = int(np.prod(shape))
    v = torch.from_numpy(g.standard_normal(n + offset)).to(dt)
    d = v.cuda()[offset:].view(shape)
    return d, v[offset:].view(shape).double()


def near(got, ref, mag, n, dt, what):
    """got (type dt) within n fp32 roundings of sums of magnitude mag, then
    one rounding to dt, of the 64-bit ref."""
    f = torch.finfo(dt)
    half = 0.0 if dt == torch.float32 else f.eps / 2
    got, ref, mag = got.double().cpu(), torch.as_tensor(ref), torch.as_tensor(mag)
    tol = (n + 1) * U * mag * (1 + half) + half * ref.abs() + f.smallest_normal * f.eps / 2
    off = (got - ref).abs() - tol
    log(f"{what}: {got.numel()} values, largest error over tolerance "
        f"{float(((got - ref).abs() / tol).max()) if got.numel() else 0:.2f}")
    assert not got.isnan().any(), what
    assert (off <= 0).all(), (what, float(off.max()))


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_sort(gpu, shape):
    T, K, E, H, layout, rows = shape
    for align in (1, 128):
        idx, _ = routing(T, K, E)
        want, dropped = brute_sort(idx, E, layout, align, rows)
        got, st = sort(torch.from_numpy(idx).cuda(), E, layout, align, rows)
        for a, b, name in zip(got, want, ("counts", "offsets", "slot_of", "row_src", "row_expert")):
            assert np.array_equal(a.cpu().numpy(), b), name
        assert int(st) == (fre.ERR_OVERFLOW if dropped else 0)


def test_sort_bad_ids(gpu):
    """Ids outside [-1, E) are skipped and reported."""
    idx, _ = routing(50, 4, 6)
    idx[3, 1], idx[7, 0], idx[9, 2] = 6, -2, 2 ** 31 - 1
    want, _ = brute_sort(idx, 6, 0, 128, 1000)
    got, st = sort(torch.from_numpy(idx).cuda(), 6, 0, 128, 1000)
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert int(st) == fre.ERR_BAD_EXPERT


@pytest.mark.parametrize("T,K,E", [(1024, 1, 7), (1025, 1, 7), (341, 3, 1024), (4096, 8, 32), (70000, 2, 300)])
def test_sort_equals_dispatch(gpu, T, K, E):
    """Around one chunk of picks, with many experts, and where the scan is a
    launch of its own: the dispatch's indices bit for bit."""
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32).cuda()
    x = torch.zeros(T, 128, dtype=torch.uint8, device="cuda")
    xs = torch.zeros(T, 1, device="cuda")
    for layout, rows in ((0, T * K + 127 * E), (1, T * K // E + 2)):
        R = E * rows if layout else rows
        want = [new_i32(E), new_i32(E + 1), new_i32(T, K), new_i32(R), new_i32(R)]
        ws = torch.zeros(fre.moe_layout_workspace_bytes(T, K, E), dtype=torch.uint8, device="cuda")
        st2 = new_i32(1, fill=0)
        fre.moe_dispatch_layout(idx, x, xs, E, layout, 128, rows, *want, None,
                                torch.zeros(1, R, device="cuda"), ws, st2)
        got, st = sort(idx, E, layout, 128, rows)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(st, st2)


@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "shifted"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_rows(gpu, shape, dt, offset):
    """All four row calls.  Rows that no token has hold NaN and are neither
    read nor (without row_src) written."""
    T, K, E, H, layout, rows = shape
    t = TYPES[dt]
    g = np.random.default_rng([1, T, H])
    idx, w = routing(T, K, E)
    (_, _, slot_of, src, _), _ = brute_sort(idx, E, layout, 128, rows)
    R = src.size
    slot, wd = torch.from_numpy(slot_of).cuda(), torch.from_numpy(w).cuda()
    srcd = torch.from_numpy(src).cuda()
    st = new_i32(1, fill=0)
    live, empty = torch.from_numpy(src >= 0), torch.from_numpy(src < 0)
    tok = torch.from_numpy(src[src >= 0]).long()

    def out(*s):
        return torch.full((int(np.prod(s)) + offset,), float("nan"), dtype=t, device="cuda")[offset:].view(s)

    x, x64 = values(g, (T, H), t, offset)
    # permute: exact; empty rows untouched, then zero
    a = out(R, H)
    fre.moe_permute_rows(x, slot, a, st)
    assert torch.equal(a.cpu()[live].double(), x64[tok])
    assert a.cpu()[empty].isnan().all()
    a = out(R, H)
    fre.moe_permute_rows(x, slot, a, st, row_src=srcd)
    assert torch.equal(a.cpu()[live].double(), x64[tok])
    assert (a.cpu()[empty] == 0).all()

    y, y64 = values(g, (R, H), t, offset)
    y[srcd < 0] = float("nan")
    picked = torch.from_numpy(slot_of).long()
    ok = picked >= 0
    rows64 = y64[picked.clamp(min=0)] * ok[..., None] if R else torch.zeros(T, K, H, dtype=torch.float64)
    # its gradient
    dx = out(T, H)
    fre.moe_permute_rows_grad(y, slot, dx, st)
    near(dx, rows64.sum(1), rows64.abs().sum(1), K, t, "permute grad")
    # combine
    w64 = torch.from_numpy(w).double().masked_fill(~ok, 0)[..., None]
    o = out(T, H)
    fre.moe_combine_rows(y, slot, wd, o, st)
    near(o, (w64 * rows64).sum(1), (w64 * rows64).abs().sum(1), K, t, "combine")
    # its gradients: together, with zeroed rows, and one at a time
    gd, g64 = values(g, (T, H), t, offset)
    dy, dw = out(R, H), torch.full((T, K), float("nan"), device="cuda")
    fre.moe_combine_rows_grad(gd, y, slot, wd, dy, dw, st)
    wrow = torch.zeros(R, dtype=torch.float64)
    wrow[picked[ok]] = torch.from_numpy(w).double()[ok]
    ref = g64[tok] * wrow[live][:, None]
    near(dy.cpu()[live], ref, ref.abs(), 1, t, "dy")
    assert dy.cpu()[empty].isnan().all()
    dots, mag = (g64[:, None] * rows64).sum(-1), (g64[:, None] * rows64).abs().sum(-1)
    # a lane's products of one part of a row (at most 2 chunks of 8), 6 levels
    # of lanes, the parts (a wave's 128 chunks of a row of up to 256, or a
    # workgroup's 512, of at least 4), 8 waves
    near(dw, dots, mag, 16 + 6 + 2 + -(-H // 2048) + 8, torch.float32, "dw")
    dy2, dw2 = out(R, H), torch.full((T, K), float("nan"), device="cuda")
    fre.moe_combine_rows_grad(gd, y, slot, wd, dy2, None, st, row_src=srcd)
    fre.moe_combine_rows_grad(gd, y, slot, wd, None, dw2, st)
    assert torch.equal(dy2.cpu()[live], dy.cpu()[live]) and (dy2.cpu()[empty] == 0).all()
    assert torch.equal(dw2, dw)
    assert int(st) == 0


@pytest.mark.parametrize("H", [1, 7, 16, 130, 7168])
def test_bytes(gpu, H):
    """8-bit rows move as bytes."""
    idx, _ = routing(60, 4, 6)
    (_, _, slot_of, src, _), _ = brute_sort(idx, 6, 0, 16, 400)
    x = torch.randint(0, 256, (60, H), dtype=torch.uint8)
    for view in (torch.uint8, torch.int8, torch.float8_e4m3fn):
        a = torch.full((400, H), 0x5a, dtype=torch.uint8, device="cuda")
        fre.moe_permute_rows(x.cuda().view(view), torch.from_numpy(slot_of).cuda(), a.view(view),
                             new_i32(1, fill=0))
        want = torch.full((400, H), 0x5a, dtype=torch.uint8)
        want[torch.from_numpy(src >= 0)] = x[torch.from_numpy(src[src >= 0]).long()]
        assert torch.equal(a.cpu(), want)


def test_bad_slots(gpu):
    """A slot past the buffer is skipped and reported by every row call."""
    T, K, R, H = 9, 3, 20, 40
    slot = torch.full((T, K), -1, dtype=torch.int32)
    slot[2, 1], slot[4, 0], slot[5, 2] = 7, 20, 2 ** 31 - 1
    sd, w = slot.cuda(), torch.ones(T, K, device="cuda")
    x, y = torch.randn(T, H, device="cuda"), torch.randn(R, H, device="cuda")
    for call in ("permute", "permute_grad", "combine", "combine_grad"):
        st, a = new_i32(1, fill=0), torch.zeros(R, H, device="cuda")
        o, dw = torch.full((T, H), 9.0, device="cuda"), torch.full((T, K), 9.0, device="cuda")
        if call == "permute":
            fre.moe_permute_rows(x, sd, a, st)
            want = torch.zeros(R, H, device="cuda")
            want[7] = x[2]
            assert torch.equal(a, want)
        elif call == "combine_grad":
            fre.moe_combine_rows_grad(x, y, sd, w, a, dw, st)
            want = torch.zeros(R, H, device="cuda")
            want[7] = x[2]
            assert torch.equal(a, want) and int((dw != 0).sum()) == 1
        else:
            if call == "combine":
                fre.moe_combine_rows(y, sd, w, o, st)
            else:
                fre.moe_permute_rows_grad(y, sd, o, st)
            want = torch.zeros(T, H, device="cuda")
            want[2] = y[7]
            assert torch.equal(o, want)
        assert int(st) == fre.ERR_BAD_INDEX, call


def test_infinities_and_overflow(gpu):
    """Infinite and NaN values of a row that is used come through; an fp16 sum
    past the largest value rounds to infinity."""
    slot = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    w = torch.ones(2, 2, device="cuda")
    y = torch.tensor([[60000.0, float("inf"), float("nan"), 1.0], [60000.0, 1.0, 1.0, -1.0],
                      [float("-inf"), 65504.0, 2.0 ** -24, 0.0]], dtype=torch.float16, device="cuda")
    o, st = torch.zeros(2, 4, dtype=torch.float16, device="cuda"), new_i32(1, fill=0)
    fre.moe_combine_rows(y, slot, w, o, st)
    want = torch.tensor([[float("inf"), float("inf"), float("nan"), 0.0],
                         [float("-inf"), 65504.0, 2.0 ** -24, 0.0]], dtype=torch.float16)
    assert torch.equal(o.cpu().nan_to_num(nan=7), want.nan_to_num(nan=7))


def test_combine_equals_moe_combine(gpu):
    idx, w = routing(300, 8, 9)
    (_, _, slot_of, src, _), _ = brute_sort(idx, 9, 0, 128, 3000)
    slot, wd = torch.from_numpy(slot_of).cuda(), torch.from_numpy(w).cuda()
    y = torch.randn(3000, 1152, device="cuda").bfloat16()
    o1, o2, st = torch.zeros(300, 1152, dtype=torch.bfloat16, device="cuda"), None, new_i32(1, fill=0)
    o2 = torch.zeros_like(o1)
    fre.moe_combine(y, slot, wd, o1, st)
    fre.moe_combine_rows(y, slot, wd, o2, st)
    assert torch.equal(o1, o2)


def test_gradients_against_differences(gpu):
    """A loss through sort, permute and combine moves by gradient . step."""
    T, K, E, H, R = 40, 3, 5, 24, 800
    idx, w = routing(T, K, E, none=0.2)
    w = np.nan_to_num(w, nan=0.5)
    (_, _, slot_of, src, _), _ = brute_sort(idx, E, 0, 128, R)
    slot, st = torch.from_numpy(slot_of).cuda(), new_i32(1, fill=0)
    x = torch.randn(T, H, dtype=torch.float64)
    wt = torch.from_numpy(w).double()
    c = torch.randn(T, H, dtype=torch.float64)                 # loss = <c, out>

    def out64(x, wt):
        y = torch.zeros(R, H, dtype=torch.float64)
        live = torch.from_numpy(src >= 0)
        y[live] = x[torch.from_numpy(src[src >= 0]).long()] ** 2       # the "experts"
        p = torch.from_numpy(slot_of).long()
        return ((wt * (p >= 0))[..., None] * y[p.clamp(min=0)]).sum(1)

    xd, wd, cd = x.float().cuda(), wt.float().cuda(), c.float().cuda()
    a = torch.zeros(R, H, device="cuda")
    fre.moe_permute_rows(xd, slot, a, st)
    dy, dw, dx = torch.zeros(R, H, device="cuda"), torch.zeros(T, K, device="cuda"), torch.zeros(T, H, device="cuda")
    fre.moe_combine_rows_grad(cd, a * a, slot, wd, dy, dw, st)
    fre.moe_permute_rows_grad(2 * a * dy, slot, dx, st)
    h = 1e-4
    for _ in range(4):
        vx, vw = torch.randn(T, H, dtype=torch.float64), torch.randn(T, K, dtype=torch.float64)
        num = ((c * out64(x + h * vx, wt + h * vw)).sum() - (c * out64(x - h * vx, wt - h * vw)).sum()) / (2 * h)
        ana = (dx.double().cpu() * vx).sum() + (dw.double().cpu() * vw).sum()
        # fp32 sums of ~1e3 terms of size 1: far under 1e-4; differences h^2
        assert abs(num - ana) < 1e-3 * (1 + abs(num))


@pytest.mark.parametrize("dt", list(TYPES))
def test_captured_step(gpu, dt):
    """Sort, permute, combine and both gradients in one graph, replayed with
    new inputs and with eager work between; every replay equals eager."""
    T, K, E, H = 700, 4, 6, 520
    R = T * K + 127 * E
    t = TYPES[dt]
    torch.manual_seed(3)
    ins = lambda: (torch.from_numpy(routing(T, K, E, seed=int(torch.randint(1 << 20, (1,))))[0]).cuda(),  # noqa: E731
                   torch.randn(T, H, device="cuda").to(t), torch.rand(T, K, device="cuda"),
                   torch.randn(T, H, device="cuda").to(t))
    idx, x, w, g = ins()
    ws = torch.zeros(fre.moe_layout_workspace_bytes(T, K, E), dtype=torch.uint8, device="cuda")
    tab = [new_i32(E), new_i32(E + 1), new_i32(T, K), new_i32(R), new_i32(R)]
    z = lambda *s: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    a, o, dy, dx, dw = z(R, H), z(T, H), z(R, H), z(T, H), torch.zeros(T, K, device="cuda")
    st = new_i32(1, fill=0)

    def step():
        fre.moe_sort_tokens(idx, E, 0, 128, R, *tab, ws, st)
        fre.moe_permute_rows(x, tab[2], a, st, row_src=tab[3])
        fre.moe_combine_rows(a, tab[2], w, o, st)
        fre.moe_combine_rows_grad(g, a, tab[2], w, dy, dw, st, row_src=tab[3])
        fre.moe_permute_rows_grad(dy, tab[2], dx, st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for d, s in zip((idx, x, w, g), ins()):
            d.copy_(s)
        step()
        want = [v.clone() for v in (*tab, a, o, dy, dx, dw)]
        for v in (a, o, dy, dx, dw):
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for v, u in zip((*tab, a, o, dy, dx, dw), want):
            assert torch.equal(v, u)
    assert int(st) == 0


def test_captured_autograd(gpu):
    """The differentiable calls, forward and backward in one graph (gradients
    asked for by name, so that no leaf accumulates), against eager passes."""
    T, K, E, H = 300, 3, 5, 264
    R = T * K + 127 * E
    torch.manual_seed(8)
    idx = torch.from_numpy(routing(T, K, E, seed=1)[0]).cuda()
    x = torch.randn(T, H, device="cuda", requires_grad=True)
    w = torch.rand(T, K, device="cuda", requires_grad=True)
    g = torch.randn(T, H, device="cuda")

    def step():
        t = fre.sort_tokens(idx, E, R)
        out = fre.combine_tokens(fre.permute_tokens(x, t) * 1.5, w, t)
        return (out.detach(), *torch.autograd.grad(out, (x, w), g), t.status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in range(4):
        idx.copy_(torch.from_numpy(routing(T, K, E, seed=10 + n)[0]))
        with torch.no_grad():
            for v in (x, w, g):
                v.copy_(torch.randn_like(v))
        want = [v.clone() for v in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once(gpu):
    """Two calls that share nothing but the library, on two streams."""
    res, keep = [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    idxs = [torch.from_numpy(routing(3000, 4, 9, seed=s)[0]).cuda() for s in range(2)]
    xs = [torch.randn(3000, 512, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for idx, x, s in zip(idxs, xs, streams):
        with torch.cuda.stream(s):
            tab, st = sort(idx, 9, 0, 128, 14000)
            a = torch.zeros(14000, 512, device="cuda")
            fre.moe_permute_rows(x, tab[2], a, st)
            res.append((tab, a, st))
    torch.cuda.synchronize()
    for (tab, a, st), idx, x in zip(res, idxs, xs):
        want, _ = brute_sort(idx.cpu().numpy(), 9, 0, 128, 14000)
        assert np.array_equal(tab[2].cpu().numpy(), want[2]) and int(st) == 0
        live = torch.from_numpy(want[3] >= 0).cuda()
        assert torch.equal(a[live], x[tab[3][live].long()])
