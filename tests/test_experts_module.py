"""CPU checks of the RoutedExperts module around its calls: copies."""

import copy
import io

import torch

import fp8_routed_expert_amd as fre


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
