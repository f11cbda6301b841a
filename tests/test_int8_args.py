"""CPU checks of the 8-bit integer calls' refusals, in the library (no launch:
the pointers are never followed) and in the binding."""

import ctypes

import pytest
import torch

import fp8_routed_expert_amd as fre
from fp8_routed_expert_amd import _lib

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)      # 8-byte aligned only
N = None


def calls(name, **ok):
    f = getattr(_lib.load(), name)
    return lambda **kw: f(*{**ok, **kw}.values(), N)


def test_quantize_refusals():
    call = calls("moe_quantize_int8", x=P, dtype=1, rows=4, cols=48, q=P, s=P)
    for bad in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(cols=0), dict(x=N), dict(q=N),
                dict(s=N)):
        assert call(**bad) == 1, bad
    for bad in (dict(cols=40), dict(x=ODD), dict(q=ODD)):
        assert call(**bad) == 2, bad
    assert call(rows=0, x=N, q=N, s=N) == 0


def test_gemm_refusals():
    call = calls("moe_gemm_int8", a=P, sa=P, w=P, sw=P, M=4, N=32, K=48, c=P, ct=1)
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(ct=3), dict(a=N), dict(sa=N), dict(w=N),
                dict(sw=N), dict(c=N)):
        assert call(**bad) == 1, bad
    for bad in (dict(N=40), dict(K=40), dict(K=131072), dict(a=ODD), dict(w=ODD), dict(c=ODD)):
        assert call(**bad) == 2, bad
    assert call(M=0x1ffffc01) == 2 and call(M=0x1ffffc00, a=N) == 1   # row scales past 31 bits
    assert call(M=0, a=N, sa=N, c=N) == 0


def test_grouped_refusals():
    call = calls("moe_grouped_gemm_int8", a=P, sa=P, w=P, sw=P, offs=P, counts=P, E=4, R=64, N=32,
                 K=48, c=P, ct=2, status=P)
    for bad in (dict(E=0), dict(E=1025), dict(R=-1), dict(N=0), dict(K=-16), dict(ct=4),
                dict(a=N), dict(sa=N), dict(w=N), dict(sw=N), dict(offs=N), dict(counts=N),
                dict(c=N)):
        assert call(**bad) == 1, bad
    for bad in (dict(N=40), dict(K=40), dict(K=131072), dict(a=ODD)):
        assert call(**bad) == 2, bad
    assert call(R=0, a=N, sa=N, c=N) == 0
    call = calls("moe_grouped_gemm_int8_gather", x=P, sx=P, T=9, src=P, w=P, sw=P, offs=P,
                 counts=P, E=4, R=64, N=32, K=4096, c=P, ct=2, status=P)
    for bad in (dict(T=-1), dict(src=N), dict(x=N), dict(sx=N), dict(offs=N), dict(c=N)):
        assert call(**bad) == 1, bad
    assert call(T=0x7ffff000 // 4096 + 1) == 2        # x past one descriptor
    assert call(R=0, src=N) == 0


def test_act_refusals():
    call = calls("moe_act_requant_int8", h=P, dtype=2, offs=P, counts=P, E=4, R=64, I=48, q=P,
                 s=P, status=P)
    for bad in (dict(dtype=3), dict(E=0), dict(E=1025), dict(R=-1), dict(I=0), dict(offs=N),
                dict(counts=N), dict(h=N), dict(q=N), dict(s=N)):
        assert call(**bad) == 1, bad
    for bad in (dict(I=40), dict(h=ODD), dict(q=ODD)):
        assert call(**bad) == 2, bad
    assert call(R=0, h=N, q=N, s=N) == 0


def test_linear_refusals():
    lib = _lib.load()
    ws = lib.moe_linear_int8_workspace_bytes
    assert ws(3, 48) == 144 + 12 and ws(0, 48) == 0 and ws(-1, 48) == 0 and ws(3, 0) == 0
    assert ws(1 << 20, 131056) == (1 << 20) * 131060   # past 32 bits
    call = calls("moe_linear_int8", x=P, dtype=1, w=P, sw=P, M=3, N=32, K=48, c=P, ct=1, ws=P,
                 wsb=156)
    for bad in (dict(dtype=3), dict(ct=3), dict(M=-1), dict(N=0), dict(K=0), dict(x=N), dict(w=N),
                dict(sw=N), dict(c=N), dict(ws=N), dict(wsb=155)):
        assert call(**bad) == 1, bad
    for bad in (dict(N=40), dict(K=40), dict(K=131072, wsb=1 << 30), dict(x=ODD), dict(w=ODD),
                dict(c=ODD), dict(ws=ODD)):
        assert call(**bad) == 2, bad
    assert call(M=0, x=N, c=N, ws=N, wsb=0) == 0


def test_binding_refusals():
    a, w = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(16, 32, dtype=torch.int8)
    s4, s16, c = torch.zeros(4), torch.zeros(16), torch.zeros(4, 16)
    with pytest.raises(ValueError, match="device tensor"):
        fre.moe_gemm_int8(a, s4, w, s16, c)
    with pytest.raises(TypeError):
        fre.moe_gemm_int8(a.view(torch.uint8), s4, w, s16, c)
    with pytest.raises(ValueError, match="two dimensions"):
        fre.moe_gemm_int8(a[0], s4, w, s16, c)
    with pytest.raises(ValueError, match="three dimensions"):
        fre.moe_grouped_gemm_int8(a, s4, w, s16, s4, s4, c, s4)
    with pytest.raises(ValueError, match="fuse_act"):
        fre.MoELayer(2, 32, 16, 4, 1, 0, 256, scale_fmt="int8", fuse_act=True, device="cpu")
    layer = fre.MoELayer(2, 32, 16, 4, 1, 0, 256, scale_fmt="int8", device="cpu")
    assert layer.h is not None and layer.q2.dtype == torch.int8 and layer.a is None
