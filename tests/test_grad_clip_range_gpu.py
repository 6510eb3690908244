"""Norms of large values whose squares are FP32 numbers and whose sums are none."""
import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
import test_grad_clip_gpu as clip
from test_layer_ops_gpu import B16, F32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


def large(n, dtype, value, seed, offset=0):
    """n values of magnitudes up to `value`, most of them close to it."""
    buf = torch.zeros(n + offset, dtype=dtype, device="cuda")
    buf[offset:] = (randn((n,), seed, F32).clamp(-1, 1) * value).to(dtype)
    return buf[offset:]


# numbers of elements, type, largest magnitude, first element: a vector, several pieces, pieces of 64 KB
TENSORS = [[(8, B16, 1e19, 0)], [(2, F32, 1.8e19, 1)], [(100003, F32, 3e18, 3), (7, B16, 1.0, 0)], [(200000, B16, 1.8e18, 0)],
           [(40001, B16, 1.8e19, 5), (300, F32, 1.0, 0)], [(24_000_000, B16, 1.6e18, 0), (5, F32, 1.5e19, 2)],
           [(3000, F32, 1.8e19, 0)] * 70]


@pytest.mark.parametrize("made", TENSORS, ids=lambda m: f"{len(m)}x{m[0][0]}")
def test_norms_whose_squares_are_fp32_numbers_clip(made):
    grads = [large(n, dt, v, i, off) for i, (n, dt, v, off) in enumerate(made)]
    before = [t.clone() for t in grads]
    plan, ws, norm = clip.plan_for(grads)
    outs = [torch.zeros_like(t) for t in grads]
    plan.run(grads, 2.0, norm, ws, outs, eps=clip.EPS)
    torch.cuda.synchronize()
    assert torch.isfinite(norm).item()
    clip.check(norm, outs, before, 2.0)
    plan.run(grads, 2.0, norm, ws, eps=clip.EPS)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, outs)) and plan.get_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e19])
def test_among_them_one_that_is_none_scales_nothing(bad):
    grads = [large(50000, B16, 1e19, 1), large(33, F32, 1e19, 2)]
    grads[0][777] = bad
    before = [t.clone() for t in grads]
    plan, ws, norm = clip.plan_for(grads)
    plan.run(grads, 0.5, norm, ws)
    torch.cuda.synchronize()
    assert not torch.isfinite(norm).item() and torch.isnan(norm).item() == (bad != bad)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(grads, before))
