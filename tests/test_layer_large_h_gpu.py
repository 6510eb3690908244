"""The MoE layer for a few tokens in bf16 with h between bf16's and FP32's largest values."""
import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref
from test_layer_ops_gpu import B16, F32, I32
from test_small_layer_gpu import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


@pytest.mark.parametrize("T,I", [(5, 64), (20, 64), (50, 72), (70, 136), (10, 704)])
def test_h_that_bf16_cannot_hold_and_fp32_can(T, I):
    """Column 0 alone: g = 2^64 - d 2^53 and u = -g or g, both FP32 numbers, silu(g) = g, h = g u of magnitude
    2^128 (1 - d 2^-11)^2.  bf16 rounds magnitudes from 2^128 (1 - 2^-9) on to infinity, FP32 from
    2^128 (1 - 2^-25) on."""
    H, E = 72, 2
    d = torch.tensor([0.5, 1.0, 1.5, 3.0, 0.0], dtype=ref.D)[torch.arange(T) % 5]
    x, w13, w2 = torch.zeros((T, H)), torch.zeros((E, 2 * I, H)), torch.zeros((E, H, I))
    x[:, 0], x[:, 1] = 2.0 ** 32, d.float() * 2.0 ** 26
    w13[:, 0, 0], w13[:, 0, 1] = 2.0 ** 32, -2.0 ** 27
    w13[0, I], w13[1, I] = w13[0, 0], -w13[1, 0]
    w2[:, :, 0] = 2.0 ** -120 * (1 + torch.arange(H) % 4)
    ids = (torch.arange(T) // 5 % 2)[:, None]
    g = 2.0 ** 64 - d * 2.0 ** 53
    h = g * g * torch.tensor([1.0, -1.0], dtype=ref.D)[ids[:, 0]]
    want = h[:, None] * w2[0, :, 0].double()[None]
    want[d == 0] *= float("inf")
    layer = Layer(T, H, I, E, 1)
    layer.run(dict(x=x.to(B16).cuda(), expert_ids=ids.to(I32).cuda(), topk_weights=torch.ones((T, 1), dtype=F32, device="cuda"),
                   w13=w13.to(B16).cuda(), w2=w2.to(B16).cuda()))
    torch.cuda.synchronize()
    assert layer.plan.get_status() == 0
    # h's product and its two parts, the second product's terms, the output
    tol = (2.0 ** -16 + 16 * ref.U + 2.0 ** -8) * want.abs()
    ref.assert_within(layer.out.check(), want, tol.nan_to_num(0, 0, 0), "out")
