"""Guard bytes around every argument of the row calls and the 8-bit integer
calls: nothing outside an output is written, and no input is."""

import numpy as np
import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.test_gpu_canary import Guarded
from tests.test_gpu_rows import brute_sort, routing

pytestmark = pytest.mark.gpu


def run(g, ins, f, *args, **kw):
    copies = [t.clone() for t in ins]
    f(*args, **kw)
    g.check(f.__name__)
    for t, c in zip(ins, copies):
        assert torch.equal(t.view(torch.uint8), c.view(torch.uint8)), f.__name__


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("T,K,E,H,layout,rows", [(1, 1, 1, 3, 0, 128), (77, 3, 5, 509, 0, 900),
                                                 (40, 4, 6, 1024, 1, 9), (33, 8, 9, 4104, 0, 1400)])
def test_rows(gpu, T, K, E, H, layout, rows, dt):
    g = Guarded()
    idx, w = routing(T, K, E)
    R = E * rows if layout else rows
    i32 = torch.int32
    idxd, wd = g.like(torch.from_numpy(idx).cuda()), g.like(torch.from_numpy(np.nan_to_num(w)).cuda())
    x, y, dout = (g.like(torch.randn(n, H, device="cuda").to(dt)) for n in (T, R, T))
    tab = [g.new((E,), i32), g.new((E + 1,), i32), g.new((T, K), i32), g.new((R,), i32), g.new((R,), i32)]
    ws, st = g.new((fre.moe_layout_workspace_bytes(T, K, E),), torch.uint8), g.new((1,), i32)
    a, dy = g.new((R, H), dt), g.new((R, H), dt)
    out, dx, dw = g.new((T, H), dt), g.new((T, H), dt), g.new((T, K), torch.float32)
    run(g, [idxd], fre.moe_sort_tokens, idxd, E, layout, 128, rows, *tab, ws, st)
    slot, src = tab[2], tab[3]
    assert np.array_equal(slot.cpu().numpy(), brute_sort(idx, E, layout, 128, rows)[0][2])
    run(g, [x, slot, src], fre.moe_permute_rows, x, slot, a, st, row_src=src)
    run(g, [y, slot], fre.moe_permute_rows_grad, y, slot, dx, st)
    run(g, [y, slot, wd], fre.moe_combine_rows, y, slot, wd, out, st)
    run(g, [dout, y, slot, wd, src], fre.moe_combine_rows_grad, dout, y, slot, wd, dy, dw, st,
        row_src=src)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (3, 272, 208), (30, 6160, 80), (100, 1040, 400),
                                   (300, 4112, 144), (1000, 4096, 400), (8200, 4112, 144)])
def test_int8_dense(gpu, M, N, K, dt):
    g = Guarded()
    i8, f32 = torch.int8, torch.float32
    x = g.like(torch.randn(M, K, device="cuda").to(dt))
    w = g.like(torch.randint(-127, 128, (N, K), dtype=i8, device="cuda"))
    sw = g.like(torch.rand(N, device="cuda"))
    q, s = g.new((M, K), i8), g.new((M,), f32)
    c, c2 = g.new((M, N), dt), g.new((M, N), dt)
    ws = g.new((fre.moe_linear_int8_workspace_bytes(M, K),), torch.uint8)
    run(g, [x], fre.moe_quantize_int8, x, q, s)
    run(g, [q, s, w, sw], fre.moe_gemm_int8, q, s, w, sw, c)
    run(g, [x, w, sw], fre.moe_linear_int8, x, w, sw, c2, ws)
    assert torch.equal(c, c2)


@pytest.mark.parametrize("E,T,H,I,layout,rows", [(5, 90, 400, 208, 1, 64), (3, 700, 256, 2048, 0, 3000),
                                                 (2, 9000, 144, 2064, 0, 13000)])
def test_int8_experts(gpu, E, T, H, I, layout, rows):
    K, g = 2, Guarded()
    i8, i32, f32, bf = torch.int8, torch.int32, torch.float32, torch.bfloat16
    R = E * rows if layout else rows
    idx = torch.from_numpy(routing(T, K, E)[0]).cuda()
    tab = [g.new((E,), i32), g.new((E + 1,), i32), g.new((T, K), i32), g.new((R,), i32), g.new((R,), i32)]
    ws, st = g.new((fre.moe_layout_workspace_bytes(T, K, E),), torch.uint8), g.new((1,), i32)
    codes = lambda *s: g.like(torch.randint(-127, 128, s, dtype=i8, device="cuda"))  # noqa: E731
    scale = lambda *s: g.like(torch.rand(*s, device="cuda") / 100)  # noqa: E731
    x, sx, w13, s13, w2, s2 = codes(T, H), scale(T), codes(E, 2 * I, H), scale(E, 2 * I), codes(E, H, I), scale(E, H)
    h, q, qs, y = g.new((R, 2 * I), bf), g.new((R, I), i8), g.new((R,), f32), g.new((R, H), bf)
    fre.moe_sort_tokens(idx, E, layout, 128, rows, *tab, ws, st)
    counts, offsets, _, src, _ = tab
    run(g, [x, sx, src, w13, s13, offsets, counts], fre.moe_grouped_gemm_int8_gather, x, sx, src, w13,
        s13, offsets, counts, h, st)
    run(g, [h, offsets, counts], fre.moe_act_requant_int8, h, offsets, counts, q, qs, st)
    run(g, [q, qs, w2, s2, offsets, counts], fre.moe_grouped_gemm_int8, q, qs, w2, s2, offsets, counts,
        y, st)
