"""The operators around the finalize in the forms that only larger calls take:
several tokens a CTA or warp in the norm's gradient, two chunks a thread in the
norm, nine slots or more in the finalize's gradient, long rows of scales and
calls that fill the GPU in the dispatch.  Sizes are for 152 SMs; each list
says which form it reaches.  Against the plain 64-bit forms of layer_ref.py."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import moe_finalize_residual_rmsnorm_gb300 as mfr
from test_layer_ops_gpu import (B16, F32, FP8, QUANTS, Guarded, Maps, check_norm, norm_inputs, randn, run_norm,
                                run_norm_grad)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


# A CTA (of the wide rows' ring) or a warp (of the narrow rows' CTAs of eight) takes
# a second token from this many tokens up, and a ring's stages come round
# again with a CTA's second token.
STEADY = [
    (8001, 8), (8001, 256),                        # a warp a token, one chunk a lane: 3648 tokens a turn
    (6001, 264), (6001, 512),                      # two chunks a lane: 2432
    (3001, 520), (2001, 1032), (2001, 2048),       # 128 threads and four tiles: 608
    (1501, 2056), (1501, 4096),                    # 256 threads: 304
    (901, 4104), (901, 8192),                      # 512 threads: 152
    (401, 8200), (401, 16384),                     # 512 threads and eight tiles: 152
]


@pytest.mark.parametrize("T,H", STEADY)
@pytest.mark.parametrize("kind", ["plain", "inplace", "no_residual_gradient"])
def test_norm_gradient_of_several_tokens_a_cta(T, H, kind):
    d_out, r, gamma = norm_inputs(T, H, 40)
    d_res = None if kind == "no_residual_gradient" else randn((T, H), 6, F32)
    eps = 1e-5
    d_in, d_x, d_gamma = run_norm_grad(d_out, d_res, r, gamma, eps, d_x=kind != "inplace", inplace=kind == "inplace")
    want, size, dg, dg_size = ref.residual_norm_grad(ref.f64(d_out), None if d_res is None else ref.f64(d_res), ref.f64(r),
                                                     ref.f64(gamma), eps)
    ref.assert_within(ref.f64(d_in), want, ref.GRAD_REL * size + ref.TINY, "d_residual_in")
    if d_x is not None:
        assert torch.equal(d_x, d_in.to(B16))              # the FP32 result rounded once
    # over the tokens: a CTA or warp adds at most ceil(T / 152) of them, then at most 8 warps
    # and ceil(608 / 32) + 5 partial sums
    chain = T / 152 + 1 + 8 + 24
    ref.assert_within(ref.f64(d_gamma), dg, (chain + 4) * ref.U * dg_size + ref.Y_REL * dg_size + ref.TINY, "d_gamma")


# two chunks a thread (4097 to 8192 columns, too many tokens for a cluster each),
# three and four of them, one chunk a thread, a cluster of four with whole rows
@pytest.mark.parametrize("T,H", [(45, 8192), (77, 4104), (40, 6000), (39, 12288), (39, 16384), (200, 2048), (38, 16384)])
@pytest.mark.parametrize("quant,tiled", QUANTS)
def test_norm_of_wide_rows(T, H, quant, tiled):
    x, res, gamma = norm_inputs(T, H, 50)
    for bf16, inplace, eps in ((True, False, 1e-6), (False, True, 1e-5)):
        check_norm(x, res, gamma, eps, quant, tiled, run_norm(x, res, gamma, eps, quant, tiled, bf16, inplace))


# nine slots or more with a CTA a token: few tokens, more, wide rows in several
# turns, plenty of tokens (more than 12 an SM) of narrow and of wider rows; and three or
# four slots with a cluster a token
@pytest.mark.parametrize("T,H,k", [(40, 1032, 9), (300, 4096, 16), (200, 8200, 12), (2000, 136, 13), (1900, 1032, 16),
                                   (1900, 264, 10), (5, 8192, 4), (30, 5000, 3)])
@pytest.mark.parametrize("align,share", [(1, 0.0), (4, 0.25)])
@pytest.mark.parametrize("dtype", [B16, F32])
def test_finalize_gradient_by_slots(T, H, k, align, share, dtype):
    m = Maps(T, k, max(16, k), align, share)
    g, E = randn((T, H), 1, dtype), randn((m.R, H), 2, B16)
    w = randn((T, k), 3, F32)
    plan = mfr.FinalizeGradPlan(T, H, k, m.R, grad_dtype=dtype, sentinel_skip=True)
    dE, dw = Guarded((m.R, H), B16), Guarded((T, k), F32)
    plan.run(g, E, m.d_row, m.d_slot, w, dE.t, dw.t)
    torch.cuda.synchronize()
    got, dw = dE.check(), dw.check()
    # row by row on the GPU: in 64 bits, where d_w is a sum, and in FP32 rounded once, where a row is a product
    slot = torch.from_numpy(m.slot_of).cuda()
    here = slot >= 0
    s = slot[here]
    gf = g.float()
    assert torch.equal(got[here], (w.view(-1)[s][:, None] * gf[s // k]).to(B16))
    assert not got[slot == -1].any()
    assert (got[slot == -2].view(torch.uint8) == 0x5A).all()
    d_w, size = torch.zeros(T * k, dtype=torch.float64, device="cuda"), torch.zeros(T * k, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 25) // H)
    rows = torch.nonzero(here)[:, 0]
    for a in range(0, len(rows), step):
        r = rows[a:a + step]
        term = E[r].double() * g[slot[r] // k].double()
        d_w[slot[r]], size[slot[r]] = term.sum(1), term.abs().sum(1)
    ref.assert_within(ref.f64(dw), d_w.view(T, k).cpu().numpy(), ref.CHAIN * ref.U * size.view(T, k).cpu().numpy() + ref.TINY,
                      "d_topk_weights")
    assert plan.get_status() == 0


# 700 x 8208 bytes are 359100 pieces of 16 bytes, more than 2048 an SM: segments of
# 2 KB, the last of one piece; 40 x 208 bytes take segments of 512 bytes.  Rows of
# scales of more than 32 words, and of more than 32 bytes where they are no whole words.
@pytest.mark.parametrize("T,H,k", [(700, 8208, 4), (350, 16384, 9), (40, 208, 5), (3, 8192, 8)])
@pytest.mark.parametrize("sf_bytes", [4, 260, 512, 67])
@pytest.mark.parametrize("align,share", [(1, 0.0), (4, 0.25), (32, 0.0)])
def test_dispatch_with_scales(T, H, k, sf_bytes, align, share):
    m = Maps(T, k, 16, align, share)
    x = torch.randint(0, 256, (T, H), dtype=torch.uint8, device="cuda").view(FP8)
    sf = torch.randint(1, 256, (T, sf_bytes), dtype=torch.uint8, device="cuda")
    plan = mfr.DispatchPlan(T, H, k, m.R, dtype=FP8, sf_bytes=sf_bytes, sentinel_skip=True)
    out, sf_out = Guarded((m.R, H), FP8), Guarded((m.R, sf_bytes), torch.uint8)
    plan.run(x, m.d_row, m.d_slot, out.t, sf, sf_out.t)
    torch.cuda.synchronize()
    slot = torch.from_numpy(m.slot_of).cuda()
    for got, src in ((out.check().view(torch.uint8), x.view(torch.uint8)), (sf_out.check(), sf)):
        assert torch.equal(got[slot >= 0], src[slot[slot >= 0] // k])
        assert not got[slot == -1].any()
        assert (got[slot == -2] == 0x5A).all()             # rows behind the last block are left as they were
    assert plan.get_status() == 0


@pytest.mark.parametrize("T,H,k", [(700, 4104, 4), (2500, 4096, 2)])
@pytest.mark.parametrize("align,share", [(1, 0.0), (16, 0.25)])
def test_dispatch_of_16_bit_rows_that_fill_the_gpu(T, H, k, align, share):
    m = Maps(T, k, 16, align, share)
    x = randn((T, H), T, B16)
    out = Guarded((m.R, H), B16)
    plan = mfr.DispatchPlan(T, H, k, m.R, sentinel_skip=True)
    plan.run(x, m.d_row, m.d_slot, out.t)
    torch.cuda.synchronize()
    slot, got = torch.from_numpy(m.slot_of).cuda(), out.check()
    assert torch.equal(got[slot >= 0], x[slot[slot >= 0] // k]) and not got[slot == -1].any()
    assert (got[slot == -2].view(torch.uint8) == 0x5A).all()
    assert plan.get_status() == 0
