"""GPU tests of the router where fp32 keys are 0: softmaxes of far logits and
sigmoids of large negative ones, whose order and groups are still decided as in
64 bits."""

import math

import numpy as np
import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.test_gpu_route import SIGMOID, SOFTMAX, call, reference
from tests.trained_util import TYPES, close

pytestmark = pytest.mark.gpu


def check(l64, dt, score, K, groups, top, best, renorm=True):
    l = torch.from_numpy(l64).to(TYPES[dt])
    idx, w, scores, _, st = call(l.cuda(), K, score=score, groups=groups, top_groups=top, group_best=best,
                                 renorm=renorm)
    ri, rw, rs = reference(l.double().numpy(), None, score, K, groups, top, best, renorm, 1.0)
    got = idx.cpu().numpy()
    assert st == 0 and np.array_equal(got, ri), (got[(got != ri).any(1)], ri[(got != ri).any(1)])
    # scores of the size of 1 by a hundred roundings and the spread of the
    # logits (up to 400) each; those below 2^-126 are 0 in fp32, and their
    # weights are divided by 2^-64 at least
    close(scores, rs, 500 * 2.0 ** -24 * rs + 2.0 ** -126, "scores")
    close(w, rw, 1000 * 2.0 ** -24 * rw + (2.0 ** -62 if renorm else 2.0 ** -126), "weights")


def test_one_group_of_four(gpu):
    """All but the first group's scores are 0 in fp32: it is still the only one
    that is kept, and its masked experts are not replaced by others."""
    l = np.zeros((3, 16))
    l[0, :4] = [150, 149, -200, -300]
    l[1, 8:12] = [-200, 140, 141, -250]
    l[2, 4:8] = [150, -math.inf, 120, -math.inf]
    check(l, "f32", SOFTMAX, 4, 4, 1, 1)
    check(l, "f32", SOFTMAX, 4, 4, 2, 2)
    idx = call(torch.from_numpy(l).float().cuda(), 4, score=SOFTMAX, groups=4, top_groups=1, group_best=1)[0].tolist()
    assert idx == [[0, 1, 2, 3], [10, 9, 8, 11], [4, 6, -1, -1]]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,groups,top,best,K", [
    (16, 1, 1, 1, 4), (16, 4, 2, 1, 4), (16, 4, 1, 2, 4), (64, 8, 3, 2, 8), (256, 8, 4, 2, 8), (256, 1, 1, 1, 16),
    (72, 8, 2, 1, 6), (288, 9, 3, 2, 8), (300, 1, 1, 1, 9), (512, 16, 4, 2, 64), (1000, 40, 7, 2, 9)])
def test_far_logits(gpu, E, groups, top, best, K, renorm, dt):
    """Logits 100 to 400 below 0 in a random order, as far from each other as E
    and the type's steps leave them: far below the largest one (softmax), or
    sigmoids that are 0 in fp32."""
    g = np.random.default_rng([E, groups, K])
    T = 24
    far = -100 - 300 * np.arange(E) / E
    l = np.stack([g.permutation(far) for _ in range(T)])
    l = torch.from_numpy(l).to(TYPES[dt]).double().numpy()
    l[1, ::3] = -math.inf
    l[2, : E // 2] = -math.inf
    check(l, dt, SIGMOID, K, groups, top, best, renorm)
    # one, then a few, that are not far
    l[:, 5] = 3.0
    l[T // 2:, 1::9] = 2.0
    check(l, dt, SOFTMAX, K, groups, top, best, renorm)
    check(l, dt, SIGMOID, K, groups, top, best, renorm)
