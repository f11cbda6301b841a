"""GPU tests of the router and its gradient against its definition in 64 bits:
picks exactly, weights and gradients within counted roundings."""

import math

import numpy as np
import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.trained_util import TYPES, U, Guarded, close, rounding, values

pytestmark = pytest.mark.gpu

SOFTMAX, SIGMOID = fre.SCORE_SOFTMAX, fre.SCORE_SIGMOID
LEAST = 2.0 ** -64

# T, E, K, groups, top_groups, group_best: from one expert to as many as there
# may be, expert counts that no wave divides, groups of one and of odd sizes
CASES = [
    (1, 1, 1, 1, 1, 1), (5, 7, 7, 1, 1, 1), (33, 8, 2, 1, 1, 1), (1, 256, 8, 8, 4, 2),
    (130, 256, 8, 8, 4, 2), (37, 72, 6, 1, 1, 1), (37, 72, 6, 8, 3, 2), (64, 60, 8, 4, 2, 1),
    (9, 64, 64, 1, 1, 1), (17, 288, 8, 1, 1, 1), (17, 288, 8, 9, 3, 2), (6, 100, 16, 100, 40, 2),
    (3, 1024, 64, 1024, 100, 1), (5, 1000, 9, 40, 7, 2), (7, 513, 8, 3, 2, 2), (3, 128, 8, 4, 1, 2),
    (4, 65, 3, 5, 2, 1), (11, 16, 4, 2, 1, 2), (2, 130, 64, 2, 1, 1), (0, 16, 4, 1, 1, 1),
    (300, 32, 4, 1, 1, 1), (4097, 16, 2, 4, 2, 2), (259, 160, 6, 8, 3, 1),
]


def reference(l, bias, score, K, groups, top_groups, best, renorm, scale):
    """Picks, weights and scores of float64 logits, row by row."""
    T, E = l.shape
    idx = np.full((T, K), -1, np.int32)
    w = np.zeros((T, K))
    scores = np.zeros((T, E))
    size = E // groups
    for t in range(T):
        row = np.where(np.isnan(l[t]), -np.inf, np.minimum(l[t], np.finfo(np.float32).max))
        ok = row > -np.inf
        s = np.zeros(E)
        if ok.any():
            if score == SOFTMAX:
                s[ok] = np.exp(row[ok] - row[ok].max())
                s /= s.sum()
            else:
                with np.errstate(over="ignore"):
                    s[ok] = 1 / (1 + np.exp(-row[ok]))
        scores[t] = s
        key = s if bias is None else s + np.where(np.isnan(bias), -np.inf, bias)
        key = np.where(ok, key, -np.inf)
        if groups > 1:
            total = [np.sort(key[g * size:(g + 1) * size])[::-1][:best].sum() for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-total[g], g))[:top_groups]
            for g in range(groups):
                if g not in kept:
                    key[g * size:(g + 1) * size] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:K]
        idx[t, :len(order)] = order
        w[t, :len(order)] = s[order]
        if renorm:
            w[t] /= max(w[t].sum(), LEAST)
        w[t] *= scale
    return idx, w, scores


def score_tol(l, ref):
    """fp32 roundings of a score: the difference to the largest logit (half a
    step of it, so U times its size relative to the exponential), the
    exponential and its argument's reduction (8 U), the division (U), and for
    the softmax a sum of up to 16 values per lane and six steps of the wave's;
    the weights add a sum of K scores, a division and a product."""
    spread = np.where(np.isfinite(l), np.abs(l - np.where(np.isfinite(l), l, -1e30).max(1, keepdims=True)), 0)
    return U * (spread.max(1, keepdims=True) + np.abs(np.where(np.isfinite(l), l, 0)).max(1, keepdims=True) + 48) * ref


def call(l, K, **kw):
    T, E = l.shape
    g = Guarded()
    idx, w = g.new(T, K, dtype=torch.int32), g.new(T, K)
    scores, local = g.new(T, E), g.new(T, K, dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fre.moe_route_tokens(l, idx, w, st, scores=scores, local_idx=local, **kw)
    g.check()
    return idx, w, scores, local, int(st)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c)) for c in CASES])
def test_route(gpu, case, score, dt):
    T, E, K, groups, top, best = case
    l, l64 = values([1, T, E, K], (T, E), TYPES[dt], 2.0)
    b, b64 = values([2, E], (E,), torch.float32, 0.1)
    for bias, renorm, scale in ((None, True, 1.0), (b, True, 2.5), (b, False, 1.5)):
        first, n = E // 3, max(1, E // 2)
        idx, w, scores, local, st = call(l, K, bias=bias, score=score, groups=groups, top_groups=top,
                                         group_best=best, renorm=renorm, scale=scale, first_expert=first,
                                         local_experts=n)
        ri, rw, rs = reference(l64.numpy(), None if bias is None else b64.numpy(), score, K, groups, top, best,
                               renorm, scale)
        assert st == 0
        got = idx.cpu().numpy()
        assert np.array_equal(got, ri), (got[(got != ri).any(1)], ri[(got != ri).any(1)])
        here = (ri >= first) & (ri < first + n)
        assert np.array_equal(local.cpu().numpy(), np.where(here, ri - first, -1))
        if T:
            close(scores, rs, score_tol(l64.numpy(), rs) + 2.0 ** -149, "scores")
            close(w, rw, score_tol(l64.numpy(), rw) * 2 + 2.0 ** -140, "weights")


@pytest.mark.parametrize("E,groups,top", [(8, 1, 1), (64, 8, 3), (256, 8, 4), (300, 1, 1)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("zero_bias", [False, True])
def test_ties_go_to_the_lowest_index(gpu, E, groups, top, score, zero_bias):
    """Logits of few values: most of a row ties, in experts and in groups."""
    g = np.random.default_rng([E, groups])
    l64 = g.integers(-2, 2, (40, E)).astype(np.float64)
    l64[3] = 0.5
    bias = np.zeros(E) if zero_bias else None
    K = min(8, E)
    idx, _, _, _, _ = call(torch.from_numpy(l64).to(torch.bfloat16).cuda(), K, score=score, groups=groups,
                           top_groups=top, group_best=2,
                           bias=None if bias is None else torch.zeros(E, device="cuda"))
    want, _, _ = reference(l64, bias, score, K, groups, top, 2, True, 1.0)
    assert np.array_equal(idx.cpu().numpy(), want)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
def test_keys_closer_than_fp32(gpu, score):
    """Logits and biases one fp32 step apart: the higher 64-bit key is picked."""
    g = np.random.default_rng(11)
    T, E, K = 64, 96, 6
    l32 = np.repeat(g.standard_normal((T, 1)).astype(np.float32), E, 1)
    step = g.integers(-3, 4, (T, E))
    l32 = l32 + step.astype(np.float32) * np.abs(np.spacing(l32))
    b32 = (np.float32(0.125) + g.integers(0, 3, E).astype(np.float32) * np.spacing(np.float32(0.125)))
    b32 = b32.astype(np.float32)
    idx, _, _, _, _ = call(torch.from_numpy(l32).cuda(), K, bias=torch.from_numpy(b32).cuda(), score=score)
    want, _, _ = reference(l32.astype(np.float64), b32.astype(np.float64), score, K, 1, 1, 1, True, 1.0)
    got = idx.cpu().numpy()
    # (a tie in 64 bits may go either way in the two computations; every pick's key is as high)
    l64 = l32.astype(np.float64)
    s = np.exp(l64 - l64.max(1, keepdims=True))
    s = s / s.sum(1, keepdims=True) if score == SOFTMAX else 1 / (1 + np.exp(-l64))
    key = s + b32.astype(np.float64)
    a, b = np.take_along_axis(key, got, 1), np.take_along_axis(key, want, 1)
    assert (np.abs(a - b) <= 4e-16).all()


@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("dt", list(TYPES))
def test_masks_infinities_and_nan(gpu, dt, score, groups, top):
    """Masked logits, rows with none left, NaN and infinities, a bias that
    switches an expert off."""
    T, E, K = 16, 24, 8
    _, l64 = values([3], (T, E), TYPES[dt])
    l64[0] = -math.inf
    l64[1, 5:] = -math.inf
    l64[2, :] = -math.inf
    l64[2, 7] = torch.finfo(TYPES[dt]).min
    l64[3, ::2] = -math.inf
    l64[4, 3] = math.inf
    l64[5, 3:6] = math.inf
    l64[6] = torch.finfo(TYPES[dt]).min
    l64[7, 0] = torch.finfo(TYPES[dt]).min
    l64[8, ::3] = 60.0
    l64[9] = -300.0
    bias = np.random.default_rng(5).standard_normal(E).astype(np.float32) * 0.1
    bias[9] = -math.inf
    for nan in (False, True):
        if nan:
            l64[10, 2], l64[11, :] = math.nan, math.nan
        l = l64.to(TYPES[dt])
        for b in (None, bias):
            idx, w, _, _, st = call(l.cuda(), K, score=score, groups=groups, top_groups=top, group_best=2,
                                    bias=None if b is None else torch.from_numpy(b).cuda())
            ri, rw, _ = reference(l.double().numpy(), b, score, K, groups, top, 2, True, 1.0)
            assert np.array_equal(idx.cpu().numpy(), ri)
            assert st == (fre.ERR_NAN if nan else 0)
            # the scores below 2^-126 that row 9 sums are divided by 2^-64: 0 in fp32
            close(w, rw, 1e-4 * np.abs(rw) + 1e-37, "weights")
    assert (idx[0] == -1).all() and (w[0] == 0).all()
    b = torch.zeros(E, device="cuda")
    b[4] = math.nan
    idx, _, _, _, st = call(l64[12:].to(TYPES[dt]).cuda(), K, score=score, bias=b)
    assert st == fre.ERR_NAN and not (idx == 4).any()


def scores_of(l, score):
    if score == SIGMOID:
        return torch.sigmoid(l)
    return torch.softmax(l, 1)


def loss(l, idx, dw, ds, score, renorm, scale):
    """What the gradient call differentiates, in 64 bits."""
    s = scores_of(l, score)
    live = idx >= 0
    w = torch.where(live, s.gather(1, idx.clamp(min=0).long()), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=LEAST)
    r = (scale * w * torch.where(live, dw, 0.0)).sum()
    return r if ds is None else r + (s * ds).sum()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("case", [c for c in CASES if c[1] > 1], ids=["x".join(map(str, c)) for c in CASES if c[1] > 1])
def test_route_grad(gpu, case, score, dt):
    T, E, K = case[:3]
    l, l64 = values([4, T, E], (T, E), TYPES[dt], 2.0)
    dw, dw64 = values([5, T, K], (T, K), torch.float32)
    ds, ds64 = values([6, T, E], (T, E), torch.float32, 0.3)
    g = np.random.default_rng(T)
    idx = np.stack([g.permutation(E)[:K] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, K), np.int32)
    if T > 1:
        idx[1, K // 2:] = -1
    if T > 2:
        idx[2] = -1
    live = torch.from_numpy(idx >= 0)
    dw[~live.cuda()] = math.nan      # never read
    for renorm, scale, with_scores in ((True, 2.5, True), (True, 1.0, False), (False, 1.5, False)):
        gd = Guarded()
        out = gd.new(T, E, dtype=TYPES[dt])
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        fre.moe_route_tokens_grad(l, torch.from_numpy(idx).cuda(), dw, out, st, score, renorm, scale,
                                  ds if with_scores else None)
        gd.check()
        assert int(st) == 0
        if not T:
            continue
        x = l64.clone().requires_grad_()
        loss(x, torch.from_numpy(idx), dw64, ds64 if with_scores else None, score, renorm, scale).backward()
        # roundings: those of a score (score_tol's count, S of them) in s, in
        # the K terms and two sums of g, and in the dot product over E
        s = scores_of(l64, score)
        w = torch.where(live, s.gather(1, torch.from_numpy(idx).clamp(min=0).long()), 0.0)
        d = torch.where(live, dw64, 0.0) * scale
        total = w.sum(1, keepdim=True).clamp(min=LEAST)
        mag = (d.abs() + (d.abs() * w).sum(1, keepdim=True) / total) / total if renorm else d.abs()
        gm = (ds64.abs() if with_scores else torch.zeros(T, E, dtype=torch.float64)).scatter_add(
            1, torch.from_numpy(idx).clamp(min=0).long(), torch.where(live, mag, 0.0))
        S = (l64 - l64.max(1, keepdim=True).values).abs().max(1, keepdim=True).values + l64.abs().max() + 64
        tol = U * 4 * S * s * (gm + ((s * gm).sum(1, keepdim=True) if score == SOFTMAX else 0))
        close(out, x.grad, tol + rounding(x.grad, TYPES[dt]), "dlogits")


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_against_differences(gpu, score, renorm):
    """The gradient against central differences of the 64-bit loss."""
    T, E, K = 4, 12, 3
    l, l64 = values([7], (T, E), torch.float32)
    dw, dw64 = values([8], (T, K), torch.float32)
    ds, ds64 = values([9], (T, E), torch.float32)
    idx = torch.tensor([[0, 5, 11], [3, 2, 1], [7, -1, -1], [-1, -1, -1]], dtype=torch.int32)
    out = torch.empty_like(l)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fre.moe_route_tokens_grad(l, idx.cuda(), dw, out, st, score, renorm, 1.5, ds)
    h = 1e-5
    num = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        for e in range(E):
            d = torch.zeros(T, E, dtype=torch.float64)
            d[t, e] = h
            num[t, e] = (loss(l64 + d, idx, dw64, ds64, score, renorm, 1.5) -
                         loss(l64 - d, idx, dw64, ds64, score, renorm, 1.5)) / (2 * h)
    # h^2 times a third derivative of order 10, roundings 2^-53 / h, fp32's in the call
    close(out, num, 1e-8 + 1e-10 + 400 * U * torch.ones(T, E), "differences")


def test_route_grad_of_masked_and_bad_picks(gpu):
    T, E, K = 6, 16, 4
    l, l64 = values([10], (T, E), torch.float32)
    l[0], l[1, ::2], l[2, 3] = -math.inf, -math.inf, math.nan
    dw, dw64 = values([11], (T, K), torch.float32)
    ds, ds64 = values([12], (T, E), torch.float32)
    idx = torch.tensor([[-1] * 4, [1, 3, 5, 7], [0, 1, 2, 4], [0, 16, 2, -2], [5, 5, 1, 2], [0, 1, 2, 3]],
                       dtype=torch.int32)
    for score in (SOFTMAX, SIGMOID):
        out = torch.full((T, E), math.nan, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        fre.moe_route_tokens_grad(l, idx.cuda(), dw, out, st, score, True, 1.0, ds)
        assert int(st) == fre.ERR_BAD_EXPERT
        o = out.cpu()
        assert (o[0] == 0).all() and (o[1, ::2] == 0).all() and o[2, 3] == 0
        ok = idx.clone()
        ok[3, 1] = ok[3, 3] = -1
        x = torch.where(l.cpu().isnan(), -math.inf, l.cpu()).double()
        x[0] = 0.0
        x = x.requires_grad_()
        zero = torch.where(x.detach() == -math.inf, 0.0, ds64)
        zero[0] = 0.0
        loss(x, ok, dw64, zero, score, True, 1.0).backward()
        want = torch.where(x.detach() == -math.inf, 0.0, x.grad)
        close(o, want, 2000 * U * torch.ones(T, E), "masked")     # sums of tens of terms of size up to 10


def test_tiny_sums(gpu):
    """Picked sigmoid scores whose sum is under 2^-64 are divided by that."""
    l = torch.full((2, 8), -50.0, device="cuda")
    l[1] = -80.0
    idx, w, _, _, _ = call(l, 2, score=SIGMOID)
    want = np.array([math.exp(-50.0) / LEAST, math.exp(-80.0) / LEAST])
    close(w, np.repeat(want[:, None], 2, 1), 200 * U * np.repeat(want[:, None], 2, 1), "weights")
    out, st = torch.empty_like(l), torch.zeros(1, dtype=torch.int32, device="cuda")
    fre.moe_route_tokens_grad(l, idx, torch.ones(2, 2, device="cuda"), out, st, SIGMOID, True, 1.0)
    ref = np.zeros((2, 8))
    ref[:, :2] = want[:, None]
    close(out, ref, 400 * U * ref + 1e-40, "gradient")
