"""The norm of many gradient tensors and clipping on the GPU against the plain
64-bit form."""
import ctypes

import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref
from test_layer_ops_gpu import B16, F32, randn

pytestmark = pytest.mark.gpu
F16 = torch.float16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    mfr.build()
    mfr.load_library()


def tensors(sizes, types, seed=0, scale=1.0, offsets=None):
    """Tensors inside guarded buffers, off elements behind a 16-byte boundary."""
    out = []
    for i, n in enumerate(sizes):
        dt, off = types[i % len(types)], 0 if offsets is None else offsets[i % len(offsets)]
        buf = torch.full((n + off + 16,), 77.0, dtype=dt, device="cuda")
        t = buf[off:off + n]
        t.copy_(randn((n,), seed + i, F32, scale).to(dt))
        out.append((buf, off, t))
    return out


def guards_whole(made):
    return all((b[:o] == 77).all() and (b[o + t.numel():] == 77).all() for b, o, t in made)


def plan_for(grads, **kw):
    plan = mfr.GradClipPlan([t.numel() for t in grads], [t.dtype for t in grads], **kw)
    return plan, torch.full((plan.workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")


def check(norm, outs, before, max_norm, eps=EPS):
    want, scaled = ref.clip(before, max_norm, eps)
    ref.assert_within(norm, want.reshape(1), ref.CLIP_REL * want + ref.TINY, "norm")
    for i, (o, w) in enumerate(zip(outs, scaled)):
        slack = 2.0 ** -25 if o.dtype is F16 else ref.TINY
        ref.assert_within(o, w, (ref.HALF_STEP[o.dtype] + 2 * ref.CLIP_REL) * w.abs() + slack, f"tensor {i}")


SIZES = [[1], [0], [7, 0, 1], [16384], [16383, 5, 100000], [1 << 21, 3], [131072 + 1, 65536 - 1, 8, 9, 10], list(range(1, 60)),
         [4096] * 600, [33] * 1100]


@pytest.mark.parametrize("types", [[F32], [B16], [F16], [B16, F32, F16]])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("limit", [0.25, 3.0])
def test_clip_in_place_and_apart(sizes, types, limit):
    made = tensors(sizes, types)
    grads = [t for _, _, t in made]
    before = [t.clone() for t in grads]
    max_norm = limit * max(1e-3, float(ref.clip(before, 1.0, 0.0)[0]))
    plan, ws, norm = plan_for(grads)
    apart = tensors(sizes, types, seed=5000)
    plan.run(grads, max_norm, norm, ws, [t for _, _, t in apart], eps=EPS)
    torch.cuda.synchronize()
    check(norm, [t for _, _, t in apart], before, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, before)) and guards_whole(apart)
    first = norm.clone()
    plan.run(grads, max_norm, norm, ws, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(norm, first) and guards_whole(made) and plan.get_status() == 0
    assert all(torch.equal(a, t) for a, (_, _, t) in zip(grads, apart))
    if limit > 1:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))


@pytest.mark.parametrize("types", [[F32], [B16, F32, F16]])
@pytest.mark.parametrize("offsets,out_offsets", [([1, 2, 3], [1, 2, 3]), ([0, 1, 5], [3, 1, 0]), ([7], [0])])
def test_tensors_that_start_anywhere(types, offsets, out_offsets):
    sizes = [1, 2, 3, 5, 9, 17, 1000, 65537, 300000]
    made, apart = tensors(sizes, types, offsets=offsets), tensors(sizes, types, seed=900, offsets=out_offsets)
    grads, outs = [t for _, _, t in made], [t for _, _, t in apart]
    plan, ws, norm = plan_for(grads)
    plan.run(grads, 1.0, norm, ws, outs, eps=EPS)
    torch.cuda.synchronize()
    check(norm, outs, grads, 1.0)
    assert guards_whole(made) and guards_whole(apart)


def test_no_tensors():
    plan, ws, norm = plan_for([])
    norm.fill_(5)
    plan.run([], 1.0, norm, ws)
    torch.cuda.synchronize()
    assert norm.item() == 0 and plan.get_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e19])
@pytest.mark.parametrize("at", [0, 4, 16383])
def test_a_norm_that_is_not_finite_scales_nothing(bad, at):
    grads = [randn((16384,), 1, F32), randn((50,), 2, B16)]
    grads[0][at] = bad
    before = [t.clone() for t in grads]
    plan, ws, norm = plan_for(grads)
    plan.run(grads, 0.5, norm, ws)
    torch.cuda.synchronize()
    assert not torch.isfinite(norm).item() and torch.isnan(norm).item() == (bad != bad)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(grads, before))
    outs = [torch.zeros_like(t) for t in grads]
    plan.run(grads, 0.5, norm, ws, outs)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, before))


def test_zeros_and_a_largest_norm_of_zero():
    grads = [torch.zeros(100, device="cuda"), torch.zeros(3, dtype=B16, device="cuda")]
    plan, ws, norm = plan_for(grads)
    plan.run(grads, 1.0, norm, ws, eps=0.0)
    torch.cuda.synchronize()
    assert norm.item() == 0 and all((t == 0).all() for t in grads)
    grads[0].fill_(1.0)
    plan.run(grads, 0.0, norm, ws)
    torch.cuda.synchronize()
    assert norm.item() == 10 and all((t == 0).all() for t in grads)


@pytest.mark.parametrize("pdl", [True, False])
def test_captured_replayed_and_on_another_stream(pdl):
    sizes = [70000, 11, 5000]
    grads = [randn((n,), n, B16) for n in sizes]
    outs = [torch.zeros_like(t) for t in grads]
    plan, ws, norm = plan_for(grads, enable_pdl=pdl)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        plan.run(grads, 2.0, norm, ws, outs)
        plan.run(outs, 1.0, norm, ws, outs)           # and once more, in place
    for seed in (0, 10):
        for t in grads:
            t.copy_(randn(t.shape, seed + t.numel(), B16))
        g.replay()
        torch.cuda.synchronize()
        check(norm, [], [(ref.f64(t) * (2.0 / (ref.clip(grads, 1, 0)[0] + EPS))).to(B16) for t in grads], 1.0)
    with torch.cuda.stream(s):
        plan.run(grads, 2.0, norm, ws, outs)
    s.synchronize()
    check(norm, outs, grads, 2.0)


def test_gradients_of_a_step_are_clipped_as_they_lie():
    """The tensors that the gradient plans write, with no wait between."""
    T, H = 300, 1024
    norm_grad = mfr.ResidualNormGradPlan(T, H)
    d_in, d_x, d_g = torch.zeros((T, H), device="cuda"), torch.zeros((T, H), dtype=B16, device="cuda"), torch.zeros(H, device="cuda")
    ws_n = torch.zeros(norm_grad.workspace_bytes(), dtype=torch.uint8, device="cuda")
    args = randn((T, H), 1, B16), randn((T, H), 2, F32), randn((T, H), 3, F32), (1 + 0.1 * randn((H,), 4, F32)).to(B16), 1e-6
    grads = [d_in, d_x, d_g]
    plan, ws, norm = plan_for(grads)
    norm_grad.run(*args, d_in, d_g, ws_n, d_x)
    torch.cuda.synchronize()
    before = [t.clone() for t in grads]
    norm_grad.run(*args, d_in, d_g, ws_n, d_x)
    plan.run(grads, 1.0, norm, ws)
    torch.cuda.synchronize()
    check(norm, grads, before, 1.0)


def test_refusals():
    lib = mfr.load_library()
    grads = [torch.zeros(64, device="cuda"), torch.zeros(64, dtype=B16, device="cuda")]
    plan, ws, norm = plan_for(grads)
    P = ctypes.c_void_p * 2
    a, b = grads[0].data_ptr(), grads[1].data_ptr()

    def call(src=(a, b), dst=(a, b), limit=1.0, eps=0.0, n=norm.data_ptr(), w=ws.data_ptr(), size=ws.numel()):
        return lib.moe_grad_clip_run(plan._h, None if src is None else P(*src), None if dst is None else P(*dst), limit, eps,
                                     n, w, size, torch.cuda.current_stream().cuda_stream)
    assert call() == 0
    assert call(src=None) == 1 and call(dst=None) == 1 and call(src=(a, None)) == 1 and call(dst=(None, b)) == 1
    assert call(n=None) == 1 and call(w=None) == 1 and call(size=ws.numel() - 1) == 1
    assert call(limit=-1.0) == 1 and call(limit=float("nan")) == 1 and call(limit=float("inf")) == 1 and call(eps=-1.0) == 1
    assert call(src=(a + 2, b)) == 3 and call(dst=(a, b + 1)) == 3 and call(n=norm.data_ptr() + 2) == 3
    assert call(dst=(a + 4, b)) == 1 and call(n=a) == 1 and call(n=ws.data_ptr()) == 1
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="expected 2 tensors"):
        plan.run(grads[:1], 1.0, norm, ws)
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        plan.run([grads[0], grads[0]], 1.0, norm, ws)
    with pytest.raises(ValueError, match=r"out\[0\]"):
        plan.run(grads, 1.0, norm, ws, [grads[0].cpu(), grads[1]])


@pytest.mark.parametrize("n", [3, 100])
def test_tensors_that_meet_are_refused(n):
    """The same tensor twice, or an output on another one's input, is a race; inputs may meet."""
    flat = torch.ones(n * 64 + 64, device="cuda")
    grads = [flat[i * 64:(i + 1) * 64] for i in range(n)]
    plan, ws, norm = plan_for(grads)
    plan.run(grads, 1.0, norm, ws)                                       # neighbours
    plan.run(grads[::-1], 1.0, norm, ws)
    others = [torch.zeros(64, device="cuda") for _ in range(n)]
    plan.run([grads[0]] * n, 1.0, norm, ws, others)                      # an input n times
    for src, dst in ((grads[:-1] + [grads[0]], None), (grads[:-1] + [flat[32:96]], None),
                     (grads, others[:-1] + [others[0]]), (grads, [others[0], grads[0]] + others[2:])):
        with pytest.raises(mfr.MFRError, match="overlaps"):
            plan.run(src, 1.0, norm, ws, dst)
    torch.cuda.synchronize()
