"""GPU test of the norm: a row's mean, rstd and output have the same bits in
every batch, so that the router behind it picks the same experts."""

import pytest
import torch

import fp8_routed_expert_amd as fre
from tests.trained_util import TYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,H", [("bf16", 7168), ("f16", 8192), ("bf16", 4104), ("bf16", 4099), ("f32", 4000),
                                  ("f32", 2050), ("bf16", 512), ("bf16", 2048), ("bf16", 4096), ("f16", 12288),
                                  ("f32", 7), ("f32", 20000)])
def test_same_bits_in_every_batch(gpu, dt, H):
    g = torch.Generator(device="cuda").manual_seed(H)
    x = (torch.randn(2100, H, generator=g, device="cuda") * 2 + 0.7).to(TYPES[dt])
    w, b = torch.randn(2, H, generator=g, device="cuda").to(TYPES[dt])

    def norm(rows):
        y = torch.empty_like(rows)
        mean, rstd = torch.empty(2, rows.shape[0], device="cuda")
        fre.moe_layer_norm(rows, w, b, 1e-5, y, mean, rstd)
        return y, mean, rstd

    whole = norm(x)
    for T in (1, 2, 77, 511, 512, 513, 1030, 2100):
        for got, want in zip(norm(x[:T].clone()), whole):
            assert torch.equal(got, want[:T]), (T, int((got != want[:T]).sum()))
