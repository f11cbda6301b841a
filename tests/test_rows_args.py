"""CPU checks of the calls that sort tokens by expert and bring them back:
their refusals, in the library (no launch: the pointers are never followed)
and in the binding."""

import ctypes

import pytest
import torch

import fp8_routed_expert_amd as fre
from fp8_routed_expert_amd import _lib

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
N = None


def test_sort_tokens_refusals():
    f = _lib.load().moe_sort_tokens
    ok = dict(idx=P, T=16, K=2, E=4, layout=0, align=128, rows=640, counts=P, offsets=P, slot=P,
              src=P, exp=P, ws=P, wsb=1 << 20, status=P)
    call = lambda **kw: f(*{**ok, **kw}.values(), N)  # noqa: E731
    for bad in (dict(T=-1), dict(K=0), dict(K=65), dict(E=0), dict(E=1025), dict(layout=2),
                dict(align=0), dict(rows=-1), dict(counts=N), dict(offsets=N), dict(status=N),
                dict(ws=N), dict(wsb=8), dict(idx=N), dict(slot=N), dict(src=N), dict(exp=N)):
        assert call(**bad) == 1, bad
    assert call(layout=1, E=1024, rows=1 << 21, wsb=1 << 24) == 2      # rows past 2^31
    assert call(T=1 << 30, K=2, wsb=1 << 62) == 2                      # picks past 2^31
    assert call(ws=ODD) == 2


def test_permute_rows_refusals():
    f = _lib.load().moe_permute_rows
    ok = dict(x=P, dtype=1, T=16, K=2, H=33, slot=P, R=64, a=P, src=N, status=P)
    call = lambda **kw: f(*{**ok, **kw}.values(), N)  # noqa: E731
    for bad in (dict(dtype=4), dict(dtype=-1), dict(T=-1), dict(K=0), dict(K=65), dict(H=0),
                dict(R=-1), dict(x=N), dict(slot=N), dict(a=N), dict(status=N)):
        assert call(**bad) == 1, bad
    assert call(x=ODD) == 2 and call(a=ODD) == 2                       # half an element off
    assert call(H=1 << 30) == 2                                        # a row past 2^31 bytes
    assert call(T=1 << 30) == 2
    assert call(T=0, R=0, x=N, slot=N, a=N) == 0


@pytest.mark.parametrize("name", ["moe_permute_rows_grad", "moe_combine_rows"])
def test_gather_sum_refusals(name):
    f = getattr(_lib.load(), name)
    weighted = name == "moe_combine_rows"
    ok = dict(y=P, dtype=0, R=64, slot=P, T=16, K=2, H=33, out=P, status=P)

    def call(w=P, **kw):
        a = {**ok, **kw}
        args = [a["y"], a["dtype"], a["R"], a["slot"]] + ([w] if weighted else [])
        return f(*args, a["T"], a["K"], a["H"], a["out"], a["status"], N)
    for bad in (dict(dtype=3), dict(dtype=-1), dict(R=-1), dict(T=-1), dict(K=0), dict(K=65),
                dict(H=0), dict(y=N), dict(slot=N), dict(out=N), dict(status=N)):
        assert call(**bad) == 1, bad
    if weighted:
        assert call(w=N) == 1
    assert call(y=ODD) == 2 and call(out=ODD) == 2
    assert call(T=0, y=N, slot=N, out=N) == 0


def test_combine_rows_grad_refusals():
    f = _lib.load().moe_combine_rows_grad
    ok = dict(dout=P, y=P, dtype=2, R=64, slot=P, w=P, T=16, K=2, H=33, dy=P, dw=P, src=N,
              status=P)
    call = lambda **kw: f(*{**ok, **kw}.values(), N)  # noqa: E731
    for bad in (dict(dtype=3), dict(R=-1), dict(T=-1), dict(K=0), dict(K=65), dict(H=0),
                dict(dout=N), dict(slot=N), dict(w=N), dict(y=N), dict(dy=N, dw=N),
                dict(status=N)):
        assert call(**bad) == 1, bad
    assert call(dout=ODD) == 2 and call(y=ODD) == 2 and call(dy=ODD) == 2
    assert call(T=0, dout=N, slot=N) == 0


def test_binding_refusals():
    """Wrong types and shapes are named before any call; host tensors too."""
    x = torch.zeros(4, 8)
    slot = torch.zeros(4, 2, dtype=torch.int32)
    a, st = torch.zeros(16, 8), torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        fre.moe_permute_rows(x, slot, a, st)
    with pytest.raises(TypeError):
        fre.moe_permute_rows(x.double(), slot, a, st)
    with pytest.raises(TypeError):
        fre.moe_permute_rows_grad(a.to(torch.int8), slot, x, st)
    with pytest.raises(ValueError, match="two dimensions"):
        fre.moe_permute_rows(x[0], slot, a, st)
    with pytest.raises(ValueError):
        fre.moe_combine_rows(a, slot, w, x, st)
    with pytest.raises(ValueError):
        fre.moe_combine_rows_grad(x, a, slot, w, None, None, st)
