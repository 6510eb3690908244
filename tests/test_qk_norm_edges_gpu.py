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


# where a projection's queries, keys and values of one head lie next to each other, within a
# token or (across) a head's tokens within the head
@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_queries_and_keys_that_lie_between_each_other(T, across):
    h, D = 5, 64
    c = qk.Case(T, h, h, D, D)

    def packed(seed):
        p = randn((h, T, 3, D) if across else (T, h, 3, D), seed, B16)
        return p, p.transpose(0, 1) if across else p
    whole, view = packed(20)
    c.q, c.k = view[:, :, 0], view[:, :, 1]
    before, want = whole.clone(), c.want()
    plan = c.plan()
    c.run(plan, c.q, c.k)                                            # in place
    torch.cuda.synchronize()
    for got, (w, tol) in zip((c.q, c.k), want):
        ref.assert_within(got, w, tol, "in place")
    assert torch.equal(whole[:, :, 2], before[:, :, 2])              # the values are not touched
    whole.copy_(before)
    apart, out = packed(30)
    c.run(plan, out[:, :, 1], out[:, :, 2])
    torch.cuda.synchronize()
    c.check(out[:, :, 1], out[:, :, 2])
    # the gradient onto what came in
    d_whole, d = packed(40)
    d_before = d_whole.clone()
    c.d_q_out, c.d_k_out = d[:, :, 0], d[:, :, 1]
    g = [torch.zeros(D, device="cuda") for _ in range(2)]
    c.run_grad(plan, c.d_q_out, c.d_k_out, *g, torch.zeros(plan.workspace_bytes(), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    got = c.d_q_out.clone(), c.d_k_out.clone()
    assert torch.equal(d_whole[:, :, 2], d_before[:, :, 2])
    d_whole.copy_(d_before)
    c.check_grad(*got, *g)
    assert plan.get_status() == 0


def test_heads_that_share_some_bytes_are_still_refused():
    T, h, D = 6, 5, 64
    c = qk.Case(T, h, h, D, D)
    flat = torch.zeros((T * h + 1) * 3 * D, dtype=B16, device="cuda")
    plan = c.plan()

    def heads(at, token=h * 3 * D, head=3 * D):
        return flat.as_strided((T, h, D), (token, head, 1), at)
    for q_out, k_out in ((heads(0), heads(D - 8)), (heads(0), heads(2 * D + 8)), (heads(8), heads(0)),
                         (heads(0), heads(3 * D)), (heads(0), heads(D, token=(h - 1) * 3 * D + D)),
                         (heads(0), heads(D, head=2 * D))):
        with pytest.raises(mfr.MFRError, match="overlaps"):
            plan.run(c.q, c.k, c.gq, c.gk, qk.EPS, c.table, c.pos, q_out, k_out)
    with pytest.raises(mfr.MFRError, match="overlaps"):              # q_out in k's place
        plan.run(heads(0), heads(D), c.gq, c.gk, qk.EPS, c.table, c.pos, heads(D), heads(2 * D))
    plan.run(heads(0), heads(D), c.gq, c.gk, qk.EPS, c.table, c.pos, heads(0), heads(2 * D))
    torch.cuda.synchronize()
