"""The gate and its gradient on the GPU against their plain 64-bit forms."""
import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref
from test_layer_ops_gpu import B16, F32, I32, Guarded, randn

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


KINDS = [(0, True), (0, False), (1, True), (1, False)]        # score, renormalize


def run(logits, k, score, renorm, scale=1.0, bias=None, **kw):
    T, E = logits.shape
    plan = mfr.GatePlan(T, E, k, score=score, renormalize=renorm, scale=scale, dtype=logits.dtype, **kw)
    ids, w = Guarded((T, k), I32), Guarded((T, k), F32)
    plan.run(logits, ids.t, w.t, bias)
    torch.cuda.synchronize()
    assert plan.get_status() == 0
    return plan, ids.check(), w.check()


def check(logits, k, score, renorm, scale=1.0, bias=None):
    plan, ids, w = run(logits, k, score, renorm, scale, bias)
    want_ids, want, tol = ref.gate(logits, k, score == 1, renorm, scale, bias)
    assert torch.equal(ids.cpu().long(), want_ids)
    ref.assert_within(w, want, tol, "weights")
    return plan, ids, w


SHAPES = [(1, 1, 1), (1, 4, 1), (3, 5, 5), (2, 16, 16), (7, 31, 3), (9, 32, 8), (5, 33, 8), (8, 128, 8), (13, 130, 6),
          (33, 256, 8), (4, 257, 16), (6, 512, 10), (3, 515, 7), (2, 1023, 16), (5, 1024, 16), (513, 64, 8)]


@pytest.mark.parametrize("score,renorm", KINDS)
@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gate(T, E, k, dtype, score, renorm):
    check(randn((T, E), T + E, dtype, 2.0), k, score, renorm, scale=2.5)


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (40, 64, 8), (300, 256, 8), (20, 1000, 16), (50, 33, 1), (9, 16, 16)])
def test_a_bias_decides_the_choice_alone(T, E, k, dtype):
    check(randn((T, E), 3, dtype), k, 1, True, bias=randn((E,), 4, F32, 0.3))


@pytest.mark.parametrize("score,bias", [(0, False), (1, False), (1, True)])
def test_ties_go_to_the_lowest_index(score, bias):
    T, E, k = 6, 200, 8
    logits = torch.randint(0, 3, (T, E), generator=torch.Generator().manual_seed(1)).float()
    logits[0] = 0.0
    logits[1, ::2], logits[1, 1::2] = 0.0, -0.0
    check(logits.cuda(), k, score, True, bias=torch.zeros(E).cuda() if bias else None)


def test_close_keys_are_told_apart():
    """Biases and logits whose FP32 keys collide, and whose exact keys do not."""
    T, E, k = 64, 128, 8
    logits = randn((T, 1), 5, F32).repeat(1, E) + 2e-7 * randn((T, E), 6, F32)
    check(logits, k, 1, True, bias=(1e-8 * randn((E,), 7, F32)))
    # keys equal up to the bias' last bits, sigmoids saturated
    check(torch.full((3, E), 30.0).cuda() + randn((3, E), 8, F32), k, 1, True, bias=torch.zeros(E).cuda())


@pytest.mark.parametrize("score,renorm", KINDS)
@pytest.mark.parametrize("E,k", [(8, 4), (130, 8)])
def test_masked_experts(E, k, score, renorm):
    logits = randn((8, E), 9, F32)
    logits[0] = -INF                                  # nothing is left
    logits[1] = NAN
    logits[2, 1:] = -INF                              # one is left
    logits[3, : E // 2] = -INF
    logits[4, 2] = NAN
    logits[5] = torch.finfo(F32).min                  # the type's lowest value is no mask
    logits[6] = -200.0
    logits[7, ::3] = torch.finfo(F32).max
    plan, ids, w = check(logits, k, score, renorm)
    assert (ids[:2] == -1).all() and (w[:2] == 0).all() and (ids[2, 1:] == -1).all() and (w[2, 1:] == 0).all()
    if score == 1:
        check(logits, k, 1, renorm, bias=torch.where(torch.arange(E, device="cuda") == 3, -INF, 0.1).float())


@pytest.mark.parametrize("E", [40, 200])
@pytest.mark.parametrize("many", [2, 4, 9, 36])
def test_biases_that_are_not_finite(E, many):
    """Infinite ones come first, the lower index before the higher; an expert with a NaN is not chosen."""
    bias = randn((E,), 11, F32)
    bias[E - many:] = INF
    bias[1] = NAN
    for k in (4, 16):
        _, ids, _ = check(randn((9, E), 12, F32), k, 1, True, bias=bias)
        n = min(k, many)
        assert ids[:, :n].tolist() == [list(range(E - many, E - many + n))] * 9 and not (ids == 1).any()


def test_infinity_counts_as_the_largest_value():
    logits = randn((2, 64), 10, F32)
    logits[0, 5] = INF
    logits[1, 5] = logits[1, 9] = INF
    _, ids, w = run(logits, 4, 0, True)
    assert ids[0, 0] == 5 and ids[1, :2].tolist() == [5, 9]
    assert w[0].tolist() == [1, 0, 0, 0] and w[1].tolist() == [0.5, 0.5, 0, 0]


@pytest.mark.parametrize("score,renorm", KINDS)
@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gradient(T, E, k, dtype, score, renorm):
    logits, g = randn((T, E), T + E + 1, dtype, 2.0), randn((T, k), T, F32)
    if E > 8:
        logits[0, 2] = -INF
    check_grad(logits, ref.gate(logits, k, score == 1, renorm)[0].to(I32).cuda(), g, score, renorm, 1.5)


def check_grad(logits, ids, g, score, renorm, scale=1.0, status=0):
    (T, E), k = logits.shape, ids.shape[1]
    plan = mfr.GatePlan(T, E, k, score=score, renormalize=renorm, scale=scale, dtype=logits.dtype)
    d = Guarded((T, E), logits.dtype)
    plan.run_grad(g, logits, ids, d.t)
    torch.cuda.synchronize()
    assert plan.get_status() == status
    want, size = ref.gate_grad(g, logits, ids, score == 1, renorm, scale)
    l = ref.f64(logits)
    live = torch.where(l > -INF, l, torch.full_like(l, float(l[l > -INF].max()) if (l > -INF).any() else 0.0))
    span = (live.amax(1, keepdim=True) - live).clamp(max=200)
    tol = (2 * E + 4 * k + 60 + 4 * span) * ref.U * size
    ref.assert_within(d.check(), want, tol + ref.HALF_STEP[logits.dtype] * (want.abs() + tol) + ref.TINY, "d_logits")
    return d.t


@pytest.mark.parametrize("score,renorm", KINDS)
def test_gradient_with_masks_empty_slots_and_repeats(score, renorm):
    T, E, k = 6, 50, 4
    logits, g = randn((T, E), 11, F32), randn((T, k), 12, F32)
    logits[0] = -INF
    logits[1, 1:] = -INF
    ids = torch.tensor([[-1, -1, -1, -1], [0, -1, -1, -1], [3, 3, 3, 7], [49, 0, 49, 1], [-1, 5, -1, 6], [1, 2, 3, 4]])
    check_grad(logits, ids.to(I32).cuda(), g, score, renorm)
    ids[2, 1], ids[5, 0] = E, -2                      # out of range
    check_grad(logits, ids.to(I32).cuda(), g, score, renorm, status=mfr.STATUS_BAD_INDEX)


@pytest.mark.parametrize("score,renorm", KINDS)
def test_gradient_against_differences(score, renorm):
    """The kernel's own weights in FP32 at l + h and l - h."""
    T, E, k, h = 4, 24, 4, 2.0 ** -6
    logits, g = randn((T, E), 13, F32), randn((T, k), 14, F32)
    plan, ids, _ = run(logits, k, score, renorm)
    d = torch.zeros_like(logits)
    plan.run_grad(g, logits, ids, d)
    want = torch.zeros_like(d)
    for e in range(E):
        step = torch.zeros_like(logits)
        step[:, e] = h
        sides = []
        for sign in (1, -1):
            moved = ref._scores(ref.f64(logits + sign * step), score == 1)
            w = torch.gather(moved, 1, ids.cpu().long())
            if renorm:
                w = w / w.sum(1, keepdim=True)
            sides.append((w * ref.f64(g)).sum(1))
        want[:, e] = ((sides[0] - sides[1]) / (2 * h)).float()
    # third derivatives of both functions are below 1 (of quotients of four scores below 8): h^2 / 6 of that times the slots
    assert (d - want).abs().max() < h * h / 6 * 8 * k * float(g.abs().max()) + 1e-5


def test_zero_tokens_and_refusals():
    z = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    plan = mfr.GatePlan(0, 8, 2)
    plan.run(z(0, 8), z(0, 2, dtype=I32), z(0, 2))
    plan.run_grad(z(0, 2), z(0, 8), z(0, 2, dtype=I32), z(0, 8))
    assert plan.get_status() == 0
    lib, plan = mfr.load_library(), mfr.GatePlan(4, 8, 2)
    l, i, w = z(4, 8), z(4, 2, dtype=I32), z(4, 2)
    a, b, c = l.data_ptr(), i.data_ptr(), w.data_ptr()
    assert lib.moe_gate_run(plan._h, a, None, b, c, None) == 0
    assert lib.moe_gate_run(plan._h, None, None, b, c, None) == 1 and lib.moe_gate_run(plan._h, a, None, None, c, None) == 1
    assert lib.moe_gate_run(plan._h, a, c, b, c, None) == 1           # a bias needs sigmoid scores
    assert lib.moe_gate_run(plan._h, a + 4, None, b, c, None) == 3 and lib.moe_gate_run(plan._h, a, None, b + 2, c, None) == 3
    assert lib.moe_gate_run(plan._h, a, None, a, c, None) == 1 and lib.moe_gate_run(plan._h, a, None, b, b, None) == 1
    assert lib.moe_gate_grad_run(plan._h, c, a, b, a, None) == 1 and lib.moe_gate_grad_run(plan._h, c, a, b, None, None) == 1
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [5, 700])
def test_gate_route_layer_as_a_step_runs_them(T):
    """Router logits to experts to the layer and to the sorted maps, captured and replayed, no wait between."""
    H, I, E, k = 256, 128, 16, 4
    gate = mfr.GatePlan(T, E, k, score=1, renormalize=True)
    route = mfr.RoutePlan(T, k, E, sentinel_skip=True)
    layer = mfr.MoeLayerPlan(T, H, I, E, k, sentinel_skip=True)
    x, w13, w2 = randn((T, H), 1, B16), randn((E, 2 * I, H), 2, B16, H ** -0.5), randn((E, H, I), 3, B16, I ** -0.5)
    logits = randn((T, E), 4, F32)
    logits[0, 3:] = -INF                              # a token with an empty slot
    new = lambda s, dtype=I32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    ids, w, out = new((T, k)), new((T, k), F32), new((T, H), B16)
    maps = new((T, k)), new((route.R,)), new((E + 1,)), new((E,))
    ws = [new((p.workspace_bytes(),), torch.uint8) for p in (route, layer)]

    def step():
        gate.run(logits, ids, w)
        route.run(ids, *maps, ws[0])
        layer.run(x, ids, w, w13, w2, out, ws[1])
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for n in range(2):
        logits.copy_(torch.where(logits.isinf(), logits, randn((T, E), 20 + n, F32)))
        g.replay()
        torch.cuda.synchronize()
        want_ids, want_w, tol = ref.gate(logits, k, True, True)
        assert torch.equal(ids.cpu().long(), want_ids)
        ref.assert_within(w, want_w, tol, "weights")
        want, tol = ref.moe_layer(x, ids, w, w13, w2)
        ref.assert_within(out, want, tol, "out")
        assert int(maps[3].sum()) == int((ids >= 0).sum())
    assert [p.get_status() for p in (gate, route, layer)] == [0, 0, 0]
