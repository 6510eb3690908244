"""The failure path of the norm gradient's ring, without a fault: with a limit so
short that its waits run out, a run ends, reports it, and the plan's next run with
the usual limit is as if nothing had been."""
import ctypes

import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
from test_layer_ops_gpu import B16, F32, Guarded, norm_inputs, randn

pytestmark = pytest.mark.gpu

USUAL = 4_000_000_000


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


class Run:
    def __init__(self, T, H, **kw):
        self.plan = mfr.ResidualNormGradPlan(T, H, **kw)
        self.d_out, self.r, self.gamma = norm_inputs(T, H, 60)
        self.d_res = randn((T, H), 6, F32)
        self.d_in, self.d_x, self.d_g = Guarded((T, H), F32), Guarded((T, H), B16), Guarded((H,), F32)
        self.ws = Guarded((self.plan.workspace_bytes(),), torch.uint8)

    def __call__(self):
        for b in (self.d_in, self.d_x, self.d_g, self.ws):
            b.t.view(torch.uint8).fill_(0x11)
        self.plan.run(self.d_out, self.d_res, self.r, self.gamma, 1e-6, self.d_in.t, self.d_g.t, self.ws.t, self.d_x.t)
        torch.cuda.synchronize()
        self.ws.check()
        return [b.check().clone() for b in (self.d_in, self.d_x, self.d_g)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


# each form of the ring, with one token a CTA (its producer never waits) and with many
@pytest.mark.parametrize("T,H", [(1, 520), (2001, 1032), (2, 4096), (1501, 4096), (100, 4104), (901, 8192), (3, 16384), (401, 9000)])
def test_a_ring_that_gives_up_ends_and_reports_it(T, H):
    run = Run(T, H)
    want = run()
    assert run.plan.get_status() == 0
    for limit in (0, 1, 200, 0):
        run.plan.set_wait_limit(limit)
        got = run()
        st = run.plan.get_status()
        if limit == 0:
            assert st == mfr.STATUS_TIMEOUT
        else:                               # the waits may or may not run out
            assert st == mfr.STATUS_TIMEOUT or (st == 0 and same(got, want))
    run.plan.set_wait_limit(USUAL)
    assert same(run(), want)
    assert run.plan.get_status() == 0


def test_debug_checks_report_a_ring_that_gave_up():
    run = Run(300, 1032, debug_checks=True)
    want = run()
    run.plan.set_wait_limit(0)
    with pytest.raises(mfr.MFRError, match="timed out"):
        run()
    run.plan.set_wait_limit(USUAL)
    assert same(run(), want)


def test_narrow_rows_have_no_wait():
    run = Run(5000, 512)
    want = run()
    run.plan.set_wait_limit(0)
    assert same(run(), want) and run.plan.get_status() == 0


def test_limits_that_are_refused():
    plan = mfr.ResidualNormGradPlan(4, 1024)
    for limit in (-1, USUAL + 1):
        with pytest.raises(mfr.MFRError) as e:
            plan.set_wait_limit(limit)
        assert e.value.name == "MFR_ERR_INVALID_ARG"
    lib, other = mfr.load_library(), mfr.ResidualNormPlan(4, 1024)
    fn = lib.moe_residual_rmsnorm_grad_set_wait_limit
    assert fn(other._h, ctypes.c_int64(1)) == 1 and fn(None, ctypes.c_int64(1)) == 1
