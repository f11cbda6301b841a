"""GPU tests of the layer norm and its gradient against the formulas in 64 bits,
with tolerances that count fp32 roundings, and against differences."""

import math

import numpy as np
import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.trained_util import TYPES, U, Guarded, close, rounding, values

pytestmark = pytest.mark.gpu

# T, H: rows from one element to more than registers hold, lengths that are no
# multiple of a chunk, at the borders of a wave's and a workgroup's chunks, and
# numbers of rows around a workgroup's and the partial sums'
SHAPES = [(1, 1), (3, 5), (2, 7), (1, 64), (5, 509), (9, 512), (4, 513), (7, 1000), (1, 7168), (33, 7168), (6, 2047),
          (6, 2048), (5, 2056), (4, 4096), (4, 4100), (3, 8191), (3, 8192), (2, 8200), (3, 16384), (2, 16392),
          (3, 40001), (0, 128), (513, 72), (1200, 264), (700, 2048), (515, 1024)]
IDS = [f"{t}x{h}" for t, h in SHAPES]


def depth(n):
    """Additions that a value goes through in a row's sum: a lane's own values,
    the lanes of a wave, the waves (rows past the registers: n / 256 and more
    of a lane's own)."""
    return 64 + n / 128


def moments64(x, eps):
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    return mean, var, 1 / torch.sqrt(var + eps)


def norm(x, w, b, eps, offset=0):
    g = Guarded()
    T, H = x.shape
    y = g.new(T, H, dtype=x.dtype, offset=offset)
    mean, rstd = g.new(T), g.new(T)
    fre.moe_layer_norm(x, w, b, eps, y, mean, rstd)
    g.check()
    return y, mean, rstd


@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "shifted"])
@pytest.mark.parametrize("wt", ["own", "f32"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_norm(gpu, shape, dt, wt, offset):
    T, H = shape
    t = TYPES[dt]
    w_t = t if wt == "own" else torch.float32
    x, x64 = values([1, T, H], (T, H), t, 1.5, 0.7, offset)
    w, w64 = values([2, H], (H,), w_t, 0.3, 1.0, offset)
    b, b64 = values([3, H], (H,), w_t, 0.5, 0.0, offset)
    eps = 1e-5
    for weight, bias in ((w, b), (w, None), (None, None)):
        y, mean, rstd = norm(x, weight, bias, eps, offset)
        if not T:
            continue
        m64, v64, r64 = moments64(x64, eps)
        d = depth(H)
        dm = (d + 2) * U * x64.abs().mean(1, keepdim=True)
        close(mean, m64[:, 0], dm[:, 0] + U * m64[:, 0].abs(), "mean")
        # the squares' sum, and the mean's error squared; half of it in the root
        dv = (d + 6) * U * v64 + dm ** 2
        dr = 0.5 * dv / (v64 + eps) + 4 * U
        close(rstd, r64[:, 0], (r64 * dr)[:, 0], "rstd")
        wv = w64 if weight is not None else torch.ones(H, dtype=torch.float64)
        z = (x64 - m64) * r64
        ref = z * wv + (b64 if bias is not None else 0)
        tol = wv.abs() * (r64 * (dm + 2 * U * (x64 - m64).abs()) + z.abs() * (dr + 3 * U)) + U * ref.abs()
        close(y, ref, tol + rounding(ref, t), "y")


@pytest.mark.parametrize("shift", [100.0, 3000.0])
def test_norm_of_rows_with_a_large_mean(gpu, shift):
    """The variance does not come from the difference of two large sums."""
    T, H = 8, 4096
    x, x64 = values([5], (T, H), torch.float32, 1.0, shift)
    y, mean, rstd = norm(x, None, None, 0.0)
    m64, v64, r64 = moments64(x64, 0.0)
    dm = (depth(H) + 2) * U * x64.abs().mean(1, keepdim=True)
    dv = (depth(H) + 6) * U * v64 + dm ** 2
    dr = 0.5 * dv / v64 + 4 * U
    close(rstd, r64[:, 0], (r64 * dr)[:, 0], "rstd")
    z = (x64 - m64) * r64
    close(y, z, r64 * (dm + 2 * U * (x64 - m64).abs()) + z.abs() * (dr + 3 * U) + 2 * U * z.abs(), "y")


def test_rows_apart(gpu):
    """A row with a NaN or an infinity is NaN, and no other is; constant rows
    and rows of one element give the bias."""
    for H in (24, 1000, 7168, 40000):
        x = torch.randn(6, H, device="cuda")
        x[1, H // 2], x[3, H - 1] = math.nan, math.inf
        x[4] = 2.5
        b = torch.randn(H, device="cuda")
        y, mean, _ = norm(x, None, b, 1e-5)
        bad = y.isnan().any(1).tolist()
        assert bad == [False, True, False, True, False, False] and y[1].isnan().all()
        assert torch.equal(y[4], b) and float(mean[4]) == 2.5
    x = torch.randn(5, 1, device="cuda").to(torch.bfloat16)
    y, _, _ = norm(x, None, torch.full((1,), 0.25, device="cuda"), 1e-5)
    assert (y == 0.25).all()


def grad(dy, x, w, mean, rstd, wants, w_t, offset=0):
    g = Guarded()
    T, H = x.shape
    dx = g.new(T, H, dtype=x.dtype, offset=offset) if wants[0] else None
    dw = g.new(H, dtype=w_t, offset=offset) if wants[1] else None
    db = g.new(H, dtype=w_t, offset=offset) if wants[2] else None
    ws = g.new(fre.moe_layer_norm_workspace_bytes(T, H), dtype=torch.uint8)
    fre.moe_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db, ws)
    g.check()
    return dx, dw, db


@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "shifted"])
@pytest.mark.parametrize("wt", ["own", "f32"])
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_norm_grad(gpu, shape, dt, wt, offset):
    T, H = shape
    t = TYPES[dt]
    w_t = t if wt == "own" else torch.float32
    x, x64 = values([11, T, H], (T, H), t, 1.5, 0.7, offset)
    dy, dy64 = values([12, T, H], (T, H), t, 1.0, 0.1, offset)
    w, w64 = values([13, H], (H,), w_t, 0.3, 1.0, offset)
    _, mean, rstd = norm(x, None, None, 1e-5)
    m64, r64 = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    z = (x64 - m64) * r64
    for weight, wants in ((w, (1, 1, 1)), (None, (1, 0, 0)), (w, (0, 1, 0)), (None, (0, 0, 1))):
        dx, dw, db = grad(dy, x, weight, mean, rstd, wants, w_t, offset)
        g = dy64 * (w64 if weight is not None else 1.0)
        d = depth(H)
        if wants[0] and T:
            c1, c2 = g.mean(1, keepdim=True), (g * z).mean(1, keepdim=True)
            ref = r64 * (g - c1 - z * c2)
            e1 = (d + 3) * U * g.abs().mean(1, keepdim=True)
            e2 = (d + 6) * U * (g * z).abs().mean(1, keepdim=True)
            tol = r64 * (e1 + z.abs() * (e2 + 4 * U * c2.abs()) + 5 * U * (g.abs() + c1.abs() + (z * c2).abs()))
            close(dx, ref, tol + rounding(ref, t), "dx")
        # a workgroup's rows one after the other, then the workgroups' sums
        n = T / 64 + 96
        if wants[1]:
            ref = (dy64 * z).sum(0)
            close(dw, ref, (n + 3) * U * (dy64 * z).abs().sum(0) + rounding(ref, w_t), "dweight")
        if wants[2]:
            ref = dy64.sum(0)
            close(db, ref, n * U * dy64.abs().sum(0) + rounding(ref, w_t), "dbias")


def test_norm_grad_against_differences(gpu):
    """Through autograd, against central differences of the 64-bit formula."""
    T, H = 3, 20
    x, x64 = values([21], (T, H), torch.float32)
    w, w64 = values([22], (H,), torch.float32, 0.3, 1.0)
    b, b64 = values([23], (H,), torch.float32)
    k64 = torch.from_numpy(np.random.default_rng(24).standard_normal((T, H)).astype(np.float32)).double()
    leaves = [v.clone().requires_grad_() for v in (x, w, b)]
    (fre.layer_norm(*leaves, 1e-5) * k64.float().cuda()).sum().backward()

    def f(x, w, b):
        m, _, r = moments64(x, 1e-5)
        return float((((x - m) * r * w + b) * k64).sum())
    h = 1e-5
    for i, v in enumerate((x64, w64, b64)):
        num = torch.zeros_like(v)
        for j in range(v.numel()):
            d = torch.zeros_like(v).view(-1)
            d[j] = h
            d = d.view(v.shape)
            args = [x64, w64, b64]
            num.view(-1)[j] = (f(*[a + d if n == i else a for n, a in enumerate(args)]) -
                               f(*[a - d if n == i else a for n, a in enumerate(args)])) / (2 * h)
        # h^2 times a third derivative of order 100, roundings of sums near 100
        # over h, and some tens of fp32 roundings of values near 10
        close(leaves[i].grad, num, (1e-8 + 1e-8 + 400 * U) * torch.ones_like(v), f"differences {i}")


def test_norm_same_bits_again(gpu):
    x, _ = values([31], (3000, 1000), torch.bfloat16)
    dy, _ = values([32], (3000, 1000), torch.bfloat16)
    w, _ = values([33], (1000,), torch.float32)
    _, mean, rstd = norm(x, w, None, 1e-5)
    first = grad(dy, x, w, mean, rstd, (1, 1, 1), torch.float32)
    for _ in range(3):
        again = grad(dy, x, w, mean, rstd, (1, 1, 1), torch.float32)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
