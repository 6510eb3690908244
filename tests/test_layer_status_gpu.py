"""The status word of the plans: no bit is lost between streams and threads."""
import threading

import pytest
import torch

import layer_ref as ref
import moe_finalize_residual_rmsnorm_gb300 as mfr

pytestmark = pytest.mark.gpu

I32, F32, B16 = torch.int32, torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


def new(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


class Route:
    """A small route whose ids are all in range, or one of them is not."""

    def __init__(self, plan, bad):
        T, k, E = plan.T, plan.k, plan.E
        ids = ref.draw_ids(T, k, E, seed=1)
        if bad:
            ids[T // 2, 0] = E
        self.plan, self.ids = plan, torch.from_numpy(ids).cuda()
        self.outs = [new((T, k), I32), new((plan.R,), I32), new((E + 1,), I32), new((E,), I32)]

    def run(self, stream=None):
        self.plan.run(self.ids, *self.outs, None, stream)


class Finalize:
    """The same for the finalize: rows in range, or one of them is not."""

    def __init__(self, plan, bad):
        T, H, k, R = plan.T, plan.H, plan.k, plan.R
        row_of = torch.arange(T * k, dtype=I32).view(T, k)
        if bad:
            row_of[T // 2, 0] = R
        g = torch.Generator().manual_seed(1)
        self.plan, self.row_of = plan, row_of.cuda()
        self.rows, self.w = torch.randn((R, H), generator=g).to(B16).cuda(), torch.rand((T, k), generator=g).cuda()
        self.res, self.res_out, self.out = new((T, H)), new((T, H)), new((T, H), B16)
        self.gamma = torch.ones(H, dtype=B16, device="cuda")

    def run(self, stream=None):
        self.plan.run(self.rows, self.row_of, self.w, self.res, self.res_out, self.gamma, 1e-6, self.out, stream)


CALLS = {"route": (Route, lambda **kw: mfr.RoutePlan(8, 8, 16, **kw)),
         "finalize": (Finalize, lambda **kw: mfr.Plan(8, 256, 4, **kw))}


@pytest.mark.parametrize("kind", CALLS)
def test_a_status_read_on_one_stream_keeps_the_bits_of_another(kind):
    """A call that raises a bit runs on one stream while the word is read and
    cleared on another, at ever different moments: every call's bit is reported by
    one of the reads."""
    make, plan_of = CALLS[kind]
    plan = plan_of()
    call = make(plan, bad=True)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    lost = 0
    for n in range(4000):
        with torch.cuda.stream(b):
            torch.cuda._sleep(n % 50 * 1000)               # up to about 25 us
        call.run(b)
        got = plan.get_status(a) | plan.get_status(a) | plan.get_status(a)
        b.synchronize()
        got |= plan.get_status(b)
        lost += got != mfr.STATUS_BAD_INDEX
    assert lost == 0


@pytest.mark.parametrize("kind", CALLS)
def test_debug_checks_report_each_threads_own_call(kind):
    """Two threads, each with a stream, share a plan with debug_checks: every
    call of the one that passes a bad id fails, no call of the other does."""
    make, plan_of = CALLS[kind]
    plan = plan_of(debug_checks=True)
    calls = [make(plan, bad=False), make(plan, bad=True)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    failures, errors = [0, 0], []
    torch.cuda.synchronize()

    def work(i):
        try:
            for _ in range(500):
                try:
                    calls[i].run(streams[i])
                except mfr.MFRError as e:
                    assert e.name == "MFR_ERR_BAD_INDEX"
                    failures[i] += 1
        except Exception as e:                             # reported by the test, not by the thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert failures == [0, 500]


@pytest.mark.parametrize("cls,fused", [(mfr.Plan, True), (mfr.FinalizePlan, False), (mfr.ExpertNormPlan, False)])
def test_debug_checks_report_a_timeout_in_every_form(cls, fused):
    """A wait that ran out (the self test's) is an error of the checked call that
    reads it, whatever the plan computes; the next call is clean."""
    T, H, k = 4, 256, 4
    plan = cls(T, H, k, debug_checks=True)
    rows, row_of = torch.ones((T * k, H), dtype=B16, device="cuda"), torch.arange(T * k, dtype=I32, device="cuda").view(T, k)
    w, gamma, out = torch.ones((T, k), device="cuda"), torch.ones(H, dtype=B16, device="cuda"), new((T, H), B16)

    def run():
        if fused:
            plan.run(rows, row_of, w, new((T, H)), new((T, H)), gamma, 1e-6, out)
        elif cls is mfr.FinalizePlan:
            plan.run(rows, row_of, w, out)
        else:
            plan.run(rows, row_of, w, gamma, 1e-6, out)
    run()
    plan.wait_selftest(2_000_000, arrive=False)
    with pytest.raises(mfr.MFRError, match="timed out"):
        run()
    run()
    assert plan.get_status() == 0


@pytest.mark.parametrize("kind", CALLS)
@pytest.mark.parametrize("where", ["this thread", "another thread"])
def test_a_plan_may_go_while_a_graph_is_captured(kind, where):
    """Closing a plan that the graph has nothing to do with leaves the capture whole."""
    make, plan_of = CALLS[kind]
    call, gone = make(plan_of(), bad=False), plan_of()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        call.run()
        if where == "this thread":
            gone.close()
        else:
            t = threading.Thread(target=gone.close)
            t.start()
            t.join()
        call.run()
    outs = call.outs if kind == "route" else [call.res_out, call.out]
    assert not any(o.any() for o in outs)
    graph.replay()
    torch.cuda.synchronize()
    assert any(o.any() for o in outs) and call.plan.get_status() == 0


@pytest.mark.parametrize("kind", CALLS)
def test_checks_and_readings_while_a_graph_is_captured(kind):
    """On another stream they work; on the captured one they are refused, before
    anything is enqueued, and the capture goes on."""
    make, plan_of = CALLS[kind]
    call, checked, refused = make(plan_of(), False), make(plan_of(debug_checks=True), False), make(plan_of(debug_checks=True), False)
    wrong = make(plan_of(debug_checks=True), True)

    def outs(c):
        return c.outs if kind == "route" else [c.res_out, c.out]
    graph, side, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        call.run()
        checked.run(other)
        assert checked.plan.get_status(other) == 0
        with pytest.raises(mfr.MFRError) as e:
            wrong.run(other)
        assert e.value.name == "MFR_ERR_BAD_INDEX"
        for refusal in (refused.run, refused.plan.get_status):
            with pytest.raises(mfr.MFRError, match="being captured") as e:
                refusal(side)
            assert e.value.name == "MFR_ERR_INVALID_ARG"
        call.run()
    assert any(o.any() for o in outs(checked))
    graph.replay()
    torch.cuda.synchronize()
    assert any(o.any() for o in outs(call)) and not any(o.any() for o in outs(refused))
    assert call.plan.get_status() == 0


@pytest.mark.parametrize("kind", CALLS)
def test_a_plan_that_could_not_be_made_leaves_no_error_behind(kind):
    """Plans are made before a capture; one that is tried inside fails and ends it.
    Later calls of the library are as if it had not been tried."""
    make, plan_of = CALLS[kind]
    before, other = make(plan_of(), False), mfr.Plan(8, 256, 4)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with pytest.raises((mfr.MFRError, RuntimeError)):
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            plan_of()
    other.wait_selftest(2_000_000, arrive=True)
    before.run()
    assert other.get_status() == 0 and before.plan.get_status() == 0
