"""GPU tests of the row and int8 calls on buffers of more than 2^32 bytes: the
rows, channels and outputs past that offset are the ones compared.  Tolerances
are those of the same calls' other tests."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.test_gpu_int8 import i32
from tests.test_gpu_int8_whole import check_all
from tests.test_gpu_rows import near

pytestmark = pytest.mark.gpu

PAST = 2 ** 32


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H", [7168, 7161], ids=["aligned", "odd"])
def test_rows(gpu, H):
    """Permute, combine and both gradients with 4.3 GB of routed rows."""
    T, K = 37600, 8
    R = T * K
    assert R * H * 2 > PAST
    torch.manual_seed(H)
    slot = torch.randperm(R, device="cuda").view(T, K).int()
    slot[5] = -1
    sel = torch.cat([(slot >= R - 40).any(1).nonzero()[:, 0], torch.tensor([0, 5, T - 1], device="cuda")])
    st, w = i32(1), torch.rand(T, K, device="cuda")
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)
    a = torch.zeros(R, H, device="cuda", dtype=torch.bfloat16)
    fre.moe_permute_rows(x, slot, a, st)
    for t in sel.tolist():
        if t != 5:
            assert torch.equal(a[slot[t].long()], x[t].expand(K, H))
    y = torch.randn(R, H, device="cuda", dtype=torch.bfloat16)
    ok = slot[sel] >= 0
    rows = y[slot[sel].clamp(min=0).long()].double() * ok[..., None]
    w64, g64 = w[sel].double()[..., None], x[sel].double()
    out = torch.empty_like(x)
    fre.moe_combine_rows(y, slot, w, out, st)
    near(out[sel], (w64 * rows).sum(1).cpu(), (w64 * rows).abs().sum(1).cpu(), K, torch.bfloat16, "combine")
    fre.moe_permute_rows_grad(y, slot, out, st)
    near(out[sel], rows.sum(1).cpu(), rows.abs().sum(1).cpu(), K, torch.bfloat16, "permute grad")
    dw = torch.empty_like(w)
    fre.moe_combine_rows_grad(x, y, slot, w, a, dw, st)
    ref = g64[:, None] * w64
    near(a[slot[sel].clamp(min=0).long()][ok], ref[ok].cpu(), ref[ok].abs().cpu(), 1, torch.bfloat16, "dy")
    dots = g64[:, None] * rows
    near(dw[sel], dots.sum(-1).cpu(), dots.abs().sum(-1).cpu(), 16 + 6 + 2 + -(-H // 2048) + 8, torch.float32, "dw")
    assert int(st) == 0


def test_permute_clears_rows(gpu):
    """Rows without a token are cleared past 2^32 bytes as well."""
    R, H = 620000, 7168
    src = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([[3, R - 2]], dtype=torch.int32, device="cuda")
    src[slot[0].long()] = 0
    x = torch.randint(1, 255, (1, H), dtype=torch.uint8, device="cuda")
    a, st = torch.full((R, H), 9, dtype=torch.uint8, device="cuda"), i32(1)
    assert a.numel() > PAST
    fre.moe_permute_rows(x, slot, a, st, row_src=src)
    assert torch.equal(a[slot[0].long()], x.expand(2, H))
    a[slot[0].long()] = 0
    for b in range(0, R, 1 << 17):
        assert not a[b:b + (1 << 17)].any()


def some_codes(*shape):
    return torch.randint(-128, 128, shape, dtype=torch.int8, device="cuda")


def some_scales(*shape):
    return torch.rand(shape, device="cuda") / 64 + 0.005


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_product_with_a_large_output(gpu, t):
    M, N, K = 300001, 8208, 144
    torch.manual_seed(1)
    a, sa, w, sw = some_codes(M, K), some_scales(M), some_codes(N, K), some_scales(N)
    c = torch.full((M, N), float("nan"), dtype=t, device="cuda")
    assert c.numel() * c.element_size() > PAST
    fre.moe_gemm_int8(a, sa, w, sw, c)
    for b in (0, 261000, M - 2001):
        check_all(c[b:b + 2001], a[b:b + 2001], sa[b:b + 2001], w, sw, f"large output {t} from {b}")
    assert not any(c[b:b + 50000].isnan().any() for b in range(0, M, 50000))


@pytest.mark.parametrize("N", [16, 1040])
def test_product_of_many_rows(gpu, N):
    """The tokens' codes alone past 2^32 bytes."""
    M, K = 610000, 7168
    torch.manual_seed(2)
    a, sa, w, sw = some_codes(M, K), some_scales(M), some_codes(N, K), some_scales(N)
    assert a.numel() > PAST
    c = torch.full((M, N), float("nan"), dtype=torch.float16, device="cuda")
    fre.moe_gemm_int8(a, sa, w, sw, c)
    for b in (0, M - 9000):
        check_all(c[b:b + 9000], a[b:b + 9000], sa[b:b + 9000], w, sw, f"many rows {N} from {b}")
    assert not c.isnan().any()


@pytest.mark.parametrize("rows", [3, 40, 300], ids=["few", "some", "many"])
def test_experts_with_large_weights(gpu, rows):
    E, N, K = 40, 14352, 7680
    assert E * N * K > PAST
    torch.manual_seed(3)
    w, sw = some_codes(E, N, K), some_scales(E, N)
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    counts[0], counts[E - 2], counts[E - 1] = 2, rows, rows - 1
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0, dtype=torch.int32)])
    R = int(offsets[-1])
    a, sa, st = some_codes(R, K), some_scales(R), i32(1)
    c = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    fre.moe_grouped_gemm_int8(a, sa, w, sw, offsets, counts, c, st)
    for e in (0, E - 2, E - 1):
        b, n = int(offsets[e]), int(counts[e])
        check_all(c[b:b + n], a[b:b + n], sa[b:b + n], w[e], sw[e], f"large weights {rows} expert {e}")
    assert int(st) == 0


@pytest.mark.parametrize("cols", [7168, 2048])
def test_quantisers(gpu, cols):
    R = PAST // (2 * cols) + 1000
    torch.manual_seed(4)
    x = torch.randn(R, cols, device="cuda", dtype=torch.bfloat16)
    q, s = torch.zeros(R, cols, dtype=torch.int8, device="cuda"), torch.zeros(R, device="cuda")
    fre.moe_quantize_int8(x, q, s)
    part = slice(R - 3000, R)
    want = (x[part].cpu().float().abs().amax(1) / 127).cuda()
    assert torch.equal(s[part], want)
    assert torch.equal(q[part].double(), torch.round(x[part].double() / want.double()[:, None]))
    # the activation of the same buffer: rows of 2 x cols / 2
    q, s, st = torch.zeros(R, cols // 2, dtype=torch.int8, device="cuda"), torch.zeros(R, device="cuda"), i32(1)
    fre.moe_act_requant_int8(x, torch.tensor([0, R], dtype=torch.int32, device="cuda"),
                             torch.tensor([R], dtype=torch.int32, device="cuda"), q, s, st)
    gate, up = x[part].double().split(cols // 2, dim=1)
    v = gate / (1 + torch.exp(-gate)) * up
    rel = (gate.abs().amax() + 6) * 2.0 ** -23
    assert ((s[part] - v.abs().amax(1) / 127).abs() <= 2 * rel * s[part]).all()
    sd = s[part].double()[:, None]
    assert ((q[part].double() * sd - v).abs() <= sd * (0.5 + 128 * rel) * (1 + 1e-12)).all()
    assert int(st) == 0
