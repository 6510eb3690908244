"""Head norms with the rotation where a lane has no head and eps is zero, and heads
that lie between each other in memory."""
import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref
import test_qk_norm_gpu as qk
from test_layer_ops_gpu import B16, F32, Guarded, randn

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


# heads that do not fill a warp: 32 / ceil(D / 16) of them do
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [B16, F16])
@pytest.mark.parametrize("T,hq,hk,D,rotary", [(5, 2, 1, 128, 128), (9, 5, 3, 80, 32), (1, 1, 1, 8, 0), (40, 33, 7, 16, 16),
                                              (3, 9, 5, 256, 64), (700, 6, 1, 96, 96), (4, 3, 2, 504, 32)])
def test_gradient_with_an_eps_of_zero(monkeypatch, T, hq, hk, D, rotary, dtype, interleaved):
    monkeypatch.setattr(qk, "EPS", 0.0)
    c = qk.Case(T, hq, hk, D, rotary, interleaved, dtype)
    plan = c.plan()
    q, k = Guarded((T, hq, D), dtype), Guarded((T, hk, D), dtype)
    c.run(plan, q.t, k.t)
    outs = Guarded((T, hq, D), dtype), Guarded((T, hk, D), dtype), Guarded((D,), F32), Guarded((D,), F32)
    ws = Guarded((plan.workspace_bytes(),), torch.uint8, fill=0xFF)
    c.run_grad(plan, *[o.t for o in outs], ws.t)
    torch.cuda.synchronize()
    assert plan.get_status() == 0
    ws.check()
    c.check(q.check(), k.check())
    c.check_grad(*[o.check() for o in outs])
