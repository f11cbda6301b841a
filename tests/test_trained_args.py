"""CPU checks of the router, the layer norm, the experts' products in 32 and 16
bits and the gated activation: their refusals, in the library (no launch: the
pointers are never followed) and in the binding."""

import ctypes
import weakref

import pytest
import torch

import fp8_routed_expert_amd as fre
from fp8_routed_expert_amd import _lib, experts

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
HALF = ctypes.c_void_p(4098)
N = None


def caller(name, ok):
    f = getattr(_lib.load(), name)
    return lambda **kw: f(*{**ok, **kw}.values(), N)


def test_route_refusals():
    call = caller("moe_route_tokens", dict(
        l=P, dtype=1, T=4, E=64, bias=P, score=1, groups=8, top=4, best=2, K=8, renorm=1, scale=1.0, first=0, local=0,
        idx=P, here=N, w=P, scores=N, status=P))
    for bad in (dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(E=0), dict(E=1025), dict(score=2), dict(score=-1),
                dict(groups=0), dict(groups=7), dict(top=0), dict(top=9), dict(best=0), dict(best=3), dict(K=0),
                dict(K=65), dict(E=8, K=9), dict(l=N), dict(idx=N), dict(w=N), dict(status=N), dict(here=P),
                dict(here=P, first=-1, local=4), dict(here=P, first=60, local=5), dict(here=P, first=64, local=1)):
        assert call(**bad) == 1, bad
    assert call(l=ODD) == 2 and call(bias=HALF) == 2 and call(idx=HALF) == 2 and call(w=ODD) == 2
    assert call(dtype=0, l=HALF) == 2 and call(scores=HALF) == 2 and call(here=HALF, local=4) == 2
    assert call(T=0, l=N, idx=N, w=N, status=N, bias=N) == 0


def test_route_grad_refusals():
    call = caller("moe_route_tokens_grad", dict(l=P, dtype=0, T=4, E=64, idx=P, K=8, score=0, renorm=1, scale=1.0,
                                                dw=P, ds=N, dl=P, status=P))
    for bad in (dict(dtype=3), dict(T=-1), dict(E=0), dict(E=1025), dict(score=2), dict(K=0), dict(K=65), dict(K=65),
                dict(l=N), dict(idx=N), dict(dw=N), dict(dl=N), dict(status=N)):
        assert call(**bad) == 1, bad
    assert call(l=HALF) == 2 and call(dl=HALF) == 2 and call(dw=HALF) == 2 and call(ds=HALF) == 2
    assert call(T=0, l=N, idx=N, dw=N, dl=N) == 0


def test_norm_refusals():
    call = caller("moe_layer_norm", dict(x=P, dtype=1, T=4, H=33, w=P, b=P, wt=0, eps=1e-5, y=P, mean=P, rstd=P))
    for bad in (dict(dtype=3), dict(dtype=-1), dict(wt=2), dict(wt=3), dict(dtype=0, wt=1), dict(T=-1), dict(H=0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(x=N), dict(y=N)):
        assert call(**bad) == 1, bad
    assert call(x=ODD) == 2 and call(y=ODD) == 2 and call(w=HALF) == 2 and call(b=HALF) == 2
    assert call(mean=HALF) == 2 and call(rstd=HALF) == 2 and call(H=1 << 30) == 2
    assert call(T=0, x=N, y=N) == 0
    lib = _lib.load()
    assert lib.moe_layer_norm_workspace_bytes(-1, 8) == 0 and lib.moe_layer_norm_workspace_bytes(8, 0) == 0
    need = lib.moe_layer_norm_workspace_bytes(4, 33)
    grad = caller("moe_layer_norm_grad", dict(dy=P, x=P, dtype=1, T=4, H=33, w=P, wt=0, mean=P, rstd=P, dx=P, dw=P,
                                              db=P, ws=P, wsb=need))
    for bad in (dict(dtype=3), dict(wt=2), dict(T=-1), dict(H=0), dict(dy=N), dict(x=N), dict(mean=N), dict(rstd=N),
                dict(dx=N, dw=N, db=N), dict(ws=N), dict(wsb=need - 1),
                dict(H=40000, dw=N, db=N, wsb=8)):                     # (a long row's sums need it for dx as well)
        assert grad(**bad) == 1, bad
    assert grad(dy=ODD) == 2 and grad(dx=ODD) == 2 and grad(dw=HALF) == 2 and grad(ws=HALF) == 2
    assert grad(mean=HALF) == 2 and grad(H=1 << 30) == 2
    assert grad(T=0, dw=N, db=N) == 0


@pytest.mark.parametrize("name", ["moe_grouped_gemm_float", "moe_grouped_gemm_float_grad_rows"])
def test_product_refusals(name):
    call = caller(name, dict(a=P, w=P, dtype=1, off=P, cnt=P, E=4, rows=64, N=40, K=72, c=P, zero=0, status=P))
    for bad in (dict(dtype=3), dict(dtype=-1), dict(E=0), dict(E=1025), dict(rows=-1), dict(N=0), dict(K=0),
                dict(a=N), dict(w=N), dict(off=N), dict(cnt=N), dict(c=N)):
        assert call(**bad) == 1, bad
    assert call(N=44) == 2 and call(K=76) == 2 and call(N=(1 << 20) + 8) == 2 and call(K=(1 << 20) + 8) == 2
    assert call(a=HALF) == 2 and call(w=HALF) == 2 and call(c=HALF) == 2
    assert call(rows=0, a=N, c=N) == 0


def test_weights_gradient_refusals():
    lib = _lib.load()
    call = caller("moe_grouped_gemm_float_grad_weights", dict(
        dc=P, a=P, dtype=1, off=P, cnt=P, E=4, rows=64, N=40, K=72, dw=P, wt=0, ws=P, wsb=1 << 30, status=P))
    for bad in (dict(dtype=3), dict(wt=2), dict(wt=3), dict(dtype=0, wt=1), dict(E=0), dict(E=1025), dict(rows=-1),
                dict(N=0), dict(K=0), dict(dc=N), dict(a=N), dict(off=N), dict(cnt=N), dict(dw=N)):
        assert call(**bad) == 1, bad
    assert call(N=44) == 2 and call(K=76) == 2 and call(dc=HALF) == 2 and call(a=HALF) == 2 and call(dw=HALF) == 2
    assert call(ws=HALF) == 2
    for bad in ((0, 64, 64, 64), (4, -1, 64, 64), (4, 64, 0, 64), (4, 64, 64, 0)):
        assert lib.moe_grouped_gemm_float_workspace_bytes(*bad) == 0


def test_act_refusals():
    for name, ok in (("moe_gated_act", dict(h=P)), ("moe_gated_act_grad", dict(dq=P, h=P))):
        call = caller(name, dict(**ok, dtype=1, off=P, cnt=P, E=4, rows=64, I=40, out=P, zero=0, status=P))
        for bad in (dict(dtype=3), dict(E=0), dict(E=1025), dict(rows=-1), dict(I=0), dict(off=N), dict(cnt=N),
                    dict(out=N), *(dict([(k, N)]) for k in ok)):
            assert call(**bad) == 1, bad
        assert call(I=44) == 2 and call(out=HALF) == 2 and call(h=HALF) == 2 and call(I=1 << 29) == 2
        assert call(rows=0, out=N, h=N) == 0


def test_binding_refusals():
    """Wrong types, shapes and devices are named before any call."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    l, st = torch.zeros(4, 16), i(1)
    with pytest.raises(ValueError, match="device tensor"):
        fre.moe_route_tokens(l, i(4, 2), torch.zeros(4, 2), st)
    with pytest.raises(TypeError):
        fre.moe_route_tokens(l.double(), i(4, 2), torch.zeros(4, 2), st)
    with pytest.raises(ValueError, match="two dimensions"):
        fre.moe_route_tokens(l[0], i(4, 2), torch.zeros(4, 2), st)
    with pytest.raises(TypeError, match="different types"):
        fre.moe_layer_norm(l, torch.zeros(16), torch.zeros(16, dtype=torch.bfloat16), 1e-5, l)
    with pytest.raises(TypeError, match="must be x's or float32"):
        fre.moe_layer_norm(l.bfloat16(), torch.zeros(16, dtype=torch.float16), None, 1e-5, l.bfloat16())
    with pytest.raises(ValueError, match="none of"):
        fre.moe_layer_norm_grad(l, l, None, st, st, None, None, None, st)
    with pytest.raises(ValueError, match="three dimensions"):
        fre.moe_grouped_gemm_float(l, l, st, st, l, st)
    with pytest.raises(TypeError):
        fre.moe_grouped_gemm_float(l.to(torch.int8), torch.zeros(2, 16, 16), i(3), i(2), l, st)
    with pytest.raises(ValueError, match="device tensor"):
        fre.moe_gated_act(l, i(3), i(2), torch.zeros(4, 8), st)
    t = fre.SortedTokens()
    t.E, t.rows_total = 2, 8
    with pytest.raises(ValueError, match="the table's buffer has 8"):
        fre.gated_act(l, t)
    with pytest.raises(ValueError, match="the table has 2"):
        fre.grouped_linear(torch.zeros(8, 16), torch.zeros(3, 16, 16), t)


def test_rows_past_31_bits():
    """A buffer whose rows, rounded up to a tile, leave 31 bits is refused."""
    rows = 0x7fff0001
    for name in ("moe_grouped_gemm_float", "moe_grouped_gemm_float_grad_rows"):
        assert caller(name, dict(a=P, w=P, dtype=1, off=P, cnt=P, E=4, rows=rows, N=8, K=8, c=P, zero=0, status=P))() == 2
    assert caller("moe_grouped_gemm_float_grad_weights", dict(
        dc=P, a=P, dtype=1, off=P, cnt=P, E=4, rows=rows, N=8, K=8, dw=P, wt=0, ws=P, wsb=1 << 40, status=P))() == 2
    for name, ok in (("moe_gated_act", dict(h=P)), ("moe_gated_act_grad", dict(dq=P, h=P))):
        assert caller(name, dict(**ok, dtype=1, off=P, cnt=P, E=4, rows=rows, I=8, out=P, zero=0, status=P))() == 2


def test_module_frees_its_last_pass_first(monkeypatch):
    """The scores that a module holds carry the last pass's graph: it is gone
    before the next one is built."""
    m = fre.RoutedExperts(E=2, H=8, I=8, K=1, device="cpu")
    m.scores = m.router.exp()
    last = weakref.ref(m.scores)

    class Stop(Exception):
        pass

    def layer_norm(*_):
        assert last() is None
        raise Stop

    monkeypatch.setattr(experts, "layer_norm", layer_norm)
    with pytest.raises(Stop):
        m(torch.zeros(1, 8))
