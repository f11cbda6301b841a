"""CPU checks around the calls of a trained block: copies of its module, numbers
that a C int cannot hold."""

import copy
import io

import pytest
import torch

import fp8_routed_expert_amd as fre
from fp8_routed_expert_amd import ops


def module():
    return fre.RoutedExperts(E=2, H=8, I=8, K=1, device="cpu")


def test_copies_after_a_pass():
    """What the last call left belongs to its graph: a copy, or a saved module,
    starts without it, and the original keeps it."""
    m = module()
    m.scores = m.router.exp()
    m.table, m.route_status = fre.SortedTokens(), torch.zeros(1, dtype=torch.int32)
    kept = m.scores, m.table, m.route_status
    file = io.BytesIO()
    torch.save(m, file)
    file.seek(0)
    for other in (copy.deepcopy(m), torch.load(file, weights_only=False)):
        assert other.scores is None and other.table is None and other.route_status is None
        assert other.router is not m.router and torch.equal(other.router, m.router)
        assert set(other.state_dict()) == set(m.state_dict()) and other.route == m.route
    assert (m.scores, m.table, m.route_status) == kept


def test_numbers_past_31_bits(monkeypatch):
    """score and group_best are C ints: 2^32 would count as 0."""
    monkeypatch.setattr(ops, "_arg", lambda t, *a: 4096)

    def call(name, stream, dev, *args):
        raise AssertionError(f"{name} called")
    monkeypatch.setattr(ops, "_call", call)
    l, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for kw in (dict(score=2 ** 32), dict(group_best=2 ** 32 + 1), dict(score=-2 ** 32), dict(group_best=1 - 2 ** 32)):
        with pytest.raises(ValueError, match="2147483647"):
            fre.moe_route_tokens(l, i, l, i, **kw)
    for score in (2 ** 32, -2 ** 32):
        with pytest.raises(ValueError, match="2147483647"):
            fre.moe_route_tokens_grad(l, i, l, l, i, score=score)
    # (what the library refuses, it refuses)
    for kw in (dict(score=2), dict(score=-1), dict(group_best=0), dict(group_best=-1)):
        with pytest.raises(AssertionError, match="moe_route_tokens called"):
            fre.moe_route_tokens(l, i, l, i, **kw)
