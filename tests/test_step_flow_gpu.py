"""The operators of a MoE layer's step as they are used together: a training step
there and back through the router, and a decode step."""
import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref
from test_layer_ops_gpu import B16, F32, I32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


def new(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def workspace(plan):
    return new((plan.workspace_bytes(),), torch.uint8)


@pytest.mark.parametrize("score,renormalize", [(0, True), (0, False), (1, True), (1, False)])
@pytest.mark.parametrize("T,H,k,E", [(1, 64, 2, 4), (37, 264, 4, 16), (300, 512, 8, 64)])
def test_training_step_through_the_router(T, H, k, E, score, renormalize):
    """Gate, sort, dispatch, experts that multiply by a power of two, the weighted sum; back to the
    rows, the router weights and the logits; then the norm of both gradients and the clipping."""
    gate = mfr.GatePlan(T, E, k, score=score, renormalize=renormalize, scale=1.5)
    route = mfr.RoutePlan(T, k, E, sentinel_skip=True)
    R = route.R
    kw = dict(sentinel_skip=True)
    disp, fin = mfr.DispatchPlan(T, H, k, R, **kw), mfr.FinalizePlan(T, H, k, R, **kw)
    back = mfr.FinalizeGradPlan(T, H, k, R, grad_dtype=F32, **kw)
    clip = mfr.GradClipPlan([T * E, T * H], [F32, B16])
    x, logits, g = randn((T, H), 1, B16), randn((T, E), 2, F32), randn((T, H), 3, F32)
    logits[0, 1:] = float("-inf")                  # a token with one expert
    factor = 2.0 ** (torch.arange(E, device="cuda") % 3 - 1)
    ids, w = new((T, k), I32), new((T, k))
    row_of, slot_of, offsets, counts = new((T, k), I32), new((R,), I32), new((E + 1,), I32), new((E,), I32)
    rows, out, d_E, d_w = new((R, H), B16), new((T, H), B16), new((R, H), B16), new((T, k))
    d_logits, d_x, norm = new((T, E)), new((T, H), B16), new((1,))
    ws_r, ws_c = workspace(route), workspace(clip)

    def step():
        gate.run(logits, ids, w)
        route.run(ids, row_of, slot_of, offsets, counts, ws_r)
        disp.run(x, row_of, slot_of, rows)
        at = torch.arange(R, device="cuda")
        expert = torch.searchsorted(offsets[1:].long(), at, right=True).clamp(max=E - 1)
        scale = factor[expert][:, None].to(B16)
        fin.run(rows * scale, row_of, w, out)
        back.run(g, rows * scale, row_of, slot_of, w, d_E, d_w)
        gate.run_grad(d_w, logits, ids, d_logits)
        disp.run_grad(d_E * scale, row_of, d_x)
        before = d_logits.clone(), d_x.clone()
        clip.run([d_logits, d_x], 1.0, norm, ws_c)
        return before
    before = step()
    torch.cuda.synchronize()
    assert [p.get_status() for p in (gate, route, disp, fin, back, clip)] == [0] * 6
    # in 64 bits, by differentiation with the choice held fixed
    want_ids, want_w, tol_w = ref.gate(logits, k, score == 1, renormalize, 1.5)
    assert torch.equal(ids.cpu().long(), want_ids)
    ref.assert_within(w, want_w, tol_w, "weights")
    f, live = ref.f64(factor)[want_ids.clamp(min=0)], (want_ids >= 0).double()
    dots = (ref.f64(x) * ref.f64(g)).sum(1, keepdim=True)
    size = (ref.f64(x) * ref.f64(g)).abs().sum(1, keepdim=True)
    want_dw = live * f * dots
    tol_dw = (H + 8) * ref.U * live * f * size
    ref.assert_within(d_w, want_dw, tol_dw + ref.TINY, "d_w")
    want, mag = ref.gate_grad(want_dw, logits, want_ids, score == 1, renormalize, 1.5)
    _, off = ref.gate_grad(tol_dw, logits, want_ids, score == 1, renormalize, 1.5)
    tol = (2 * E + 4 * k + 100) * ref.U * mag + off + ref.TINY
    ref.assert_within(before[0], want, tol, "d_logits")
    terms = want_w * live * f
    want_x = (terms.sum(1, keepdim=True) * ref.f64(g))
    # every row's w g is rounded to bf16, the sum over the slots in FP32, then to bf16
    tol_x = (2 ** -8 + (k + 40) * ref.U) * (terms.abs().sum(1, keepdim=True) * ref.f64(g).abs())
    ref.assert_within(before[1], want_x, tol_x + 2 ** -8 * (want_x.abs() + tol_x) + ref.TINY, "d_x")
    total, scaled = ref.clip(before, 1.0, 1e-6)
    ref.assert_within(norm, total.reshape(1), ref.CLIP_REL * total, "norm")
    for got, s in zip((d_logits, d_x), scaled):
        ref.assert_within(got, s, (ref.HALF_STEP[got.dtype] + 2 * ref.CLIP_REL) * s.abs() + ref.TINY, "clipped")


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_step(fp8):
    """Head norms in place in a packed projection, then residual norm, gate, layer, residual norm,
    captured once and replayed with other inputs."""
    T, H, I, E, k, hq, hk, D, most = 5, 512, 256, 16, 4, 4, 1, 64, 100
    qk = mfr.QkNormRopePlan(T, hq, hk, D, max_positions=most)
    first = mfr.ResidualNormPlan(T, H, quant=mfr.QUANT_GROUP128)
    gate = mfr.GatePlan(T, E, k, dtype=B16)
    layer = mfr.MoeLayerPlan(T, H, I, E, k, dtype=torch.float8_e4m3fn if fp8 else B16, sentinel_skip=True)
    second = mfr.ResidualNormPlan(T, H, quant=mfr.QUANT_NONE)
    from test_small_layer_gpu import inputs
    weights = inputs(T, H, I, E, k, fp8)
    gq, gk = (1 + 0.2 * randn((D,), 1, F32)).to(B16), (1 + 0.2 * randn((D,), 2, F32)).to(B16)
    g1, g2, router = (1 + 0.2 * randn((H,), 3, F32)).to(B16), (1 + 0.2 * randn((H,), 4, F32)).to(B16), randn((H, E), 5, B16, H ** -0.5)
    table = torch.cat([torch.cos(torch.arange(most * 32).view(most, 32) * 0.1), torch.sin(torch.arange(most * 32).view(most, 32) * 0.1)], 1).float().cuda()
    qkv, pos = new((T, hq + 2 * hk, D), B16), new((T,), I32)
    q, kk = qkv[:, :hq], qkv[:, hq:hq + hk]
    x, res, r1, r2 = new((T, H), B16), new((T, H)), new((T, H)), new((T, H))
    y, codes, sf, out, z = new((T, H), B16), new((T, H), torch.float8_e4m3fn), new((T, H // 128)), new((T, H), B16), new((T, H), B16)
    logits, ids, w, ws = new((T, E), B16), new((T, k), I32), new((T, k)), workspace(layer)

    def step():
        qk.run(q, kk, gq, gk, 1e-6, table, pos, q, kk)
        first.run(x, res, r1, g1, 1e-6, y, codes, sf)
        torch.mm(y, router, out=logits)
        gate.run(logits, ids, w)
        if fp8:
            layer.run(codes, ids, w, weights["w13"], weights["w2"], out, ws, sf, weights["w13_sf"], weights["w2_sf"])
        else:
            layer.run(y, ids, w, weights["w13"], weights["w2"], out, ws)
        second.run(out, r1, r2, g2, 1e-6, z)
    step()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in (10, 20):
        qkv.copy_(randn(qkv.shape, seed, B16))
        pos.copy_(torch.randint(0, most, (T,), generator=torch.Generator().manual_seed(seed)))
        x.copy_(randn((T, H), seed + 1, B16))
        res.copy_(randn((T, H), seed + 2, F32))
        before = qkv.clone()
        graph.replay()
        torch.cuda.synchronize()
        for got, src, gamma in ((q, before[:, :hq], gq), (kk, before[:, hq:hq + hk], gk)):
            want, tol = ref.qk_norm(src, gamma, 1e-6, table, pos, D, False)
            ref.assert_within(got, want, tol + 2 ** -8 * (want.abs() + tol) + ref.TINY, "heads")
        assert torch.equal(qkv[:, hq + hk:], before[:, hq + hk:])
        want_ids, want_w, tol = ref.gate(logits, k, False, True)
        assert torch.equal(ids.cpu().long(), want_ids)
        ref.assert_within(w, want_w, tol, "weights")
        scales = (sf, weights["w13_sf"], weights["w2_sf"]) if fp8 else ()
        want, tol = ref.moe_layer(codes if fp8 else y, ids, w, weights["w13"], weights["w2"], *scales)
        ref.assert_within(out, want, tol, "layer")
        assert torch.equal(r2, r1 + out.float())
    assert [p.get_status() for p in (qk, first, gate, layer, second)] == [0] * 5
