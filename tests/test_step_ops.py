"""The operators of a MoE layer's step, without a GPU: the header is plain C,
every symbol is exported and bound, plans and calls refuse what they cannot do
before any device is touched, and the references agree with differences."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import moe_finalize_residual_rmsnorm_gb300 as mfr
import step_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_step_ops.h")
INVALID, SHAPE, BAD_DEVICE = 1, 2, 4
I32, F32, B16, F16, FP8 = torch.int32, torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    mfr.build()
    return mfr.load_library()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"\b(moe_\w+)\s*\(", text))


def test_every_declared_symbol_is_exported_and_bound(lib):
    names = declared()
    assert {"moe_gate_run", "moe_gate_grad_run", "moe_small_layer_run", "moe_qk_norm_rope_run", "moe_qk_norm_rope_grad_run",
            "moe_grad_clip_run"} <= names
    assert not [n for n in names if not hasattr(lib, n)]
    assert names <= set(mfr.SIGNATURES)


def test_header_is_c99(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "moe_step_ops.h"\nint main(void) { moe_op_t op = 0; moe_op_destroy(op); return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", f"-I{os.path.dirname(HEADER)}", str(src)],
                   check=True)


N = float("nan")
TWO = (ctypes.c_int64 * 2)(5, 7), (ctypes.c_int * 2)(0, 1)
PLANS = {
    "moe_gate_plan": ((4, 64, 8, 0, 1, 1.0, 0), [
        ((-1, 64, 8, 0, 1, 1.0, 0), INVALID), ((4, 64, 8, 2, 1, 1.0, 0), INVALID), ((4, 64, 8, -1, 1, 1.0, 0), INVALID),
        ((4, 64, 8, 0, 2, 1.0, 0), INVALID), ((4, 64, 8, 0, 1, 1.0, 3), INVALID), ((4, 64, 8, 0, 1, 0.0, 0), INVALID),
        ((4, 64, 8, 0, 1, N, 0), INVALID), ((4, 64, 0, 0, 1, 1.0, 0), SHAPE), ((4, 64, 17, 0, 1, 1.0, 0), SHAPE),
        ((4, 7, 8, 0, 1, 1.0, 0), SHAPE), ((4, 1025, 8, 0, 1, 1.0, 0), SHAPE), (((1 << 26) + 1, 64, 8, 0, 1, 1.0, 0), SHAPE)]),
    "moe_qk_norm_rope_plan": ((4, 8, 2, 64, 64, 0, 0, 100), [
        ((-1, 8, 2, 64, 64, 0, 0, 100), INVALID), ((4, 8, 2, 64, 64, 2, 0, 100), INVALID), ((4, 8, 2, 64, 64, 0, 2, 100), INVALID),
        ((4, 0, 2, 64, 64, 0, 0, 100), SHAPE), ((4, 8, 0, 64, 64, 0, 0, 100), SHAPE), ((4, 1025, 2, 64, 64, 0, 0, 100), SHAPE),
        ((4, 8, 2, 60, 16, 0, 0, 100), SHAPE), ((4, 8, 2, 520, 64, 0, 0, 100), SHAPE), ((4, 8, 2, 0, 0, 0, 0, 100), SHAPE),
        ((4, 8, 2, 64, 72, 0, 0, 100), SHAPE), ((4, 8, 2, 64, 80, 0, 0, 100), SHAPE), ((4, 8, 2, 64, 24, 0, 0, 100), SHAPE),
        ((4, 8, 2, 64, -16, 0, 0, 100), SHAPE), ((4, 8, 2, 64, 64, 0, 0, 0), SHAPE)]),
    "moe_grad_clip_plan": ((2, *TWO), [
        ((-1, *TWO), INVALID), ((2, None, TWO[1]), INVALID), ((2, TWO[0], None), INVALID), ((65537, *TWO), SHAPE),
        ((2, (ctypes.c_int64 * 2)(5, -1), TWO[1]), INVALID), ((2, (ctypes.c_int64 * 2)(1 << 40, 5), TWO[1]), SHAPE),
        ((2, TWO[0], (ctypes.c_int * 2)(0, 3)), INVALID), ((2, TWO[0], (ctypes.c_int * 2)(-1, 0)), INVALID)]),
    "moe_small_layer_plan": ((4, 64, 64, 8, 2, 0), [
        ((-1, 64, 64, 8, 2, 0), INVALID), ((4, 64, 64, 8, 2, 2), INVALID), ((4, 64, 64, 8, 2, -1), INVALID),
        ((4, 60, 64, 8, 2, 0), SHAPE), ((4, 0, 64, 8, 2, 0), SHAPE), ((4, 16392, 64, 8, 2, 0), SHAPE),
        ((4, 64, 60, 8, 2, 0), SHAPE), ((4, 64, 0, 8, 2, 0), SHAPE), ((4, 64, 16392, 8, 2, 0), SHAPE),
        ((4, 64, 64, 0, 2, 0), SHAPE), ((4, 64, 64, 1025, 2, 0), SHAPE), ((4, 64, 64, 8, 0, 0), SHAPE),
        ((4, 64, 64, 8, 17, 0), SHAPE), ((4097, 64, 64, 8, 1, 0), SHAPE), ((257, 64, 64, 8, 16, 0), SHAPE),
        ((4, 72, 128, 8, 2, 1), SHAPE), ((4, 64, 64, 8, 2, 1), SHAPE), ((1 << 62, 64, 64, 8, 2, 0), SHAPE)]),
}


@pytest.mark.parametrize("fn,args,code", [(fn, a, c) for fn, (_, bad) in PLANS.items() for a, c in bad])
def test_plans_refuse_what_they_cannot_do(lib, fn, args, code):
    h = ctypes.c_void_p(123)
    assert getattr(lib, fn)(ctypes.byref(h), *args, None) == code
    assert not h.value
    assert lib.moe_finalize_rmsnorm_last_error().decode()
    assert getattr(lib, fn)(None, *args, None) == INVALID


@pytest.mark.parametrize("fn", list(PLANS))
def test_plans_refuse_options_that_are_not_theirs(lib, fn):
    h = ctypes.c_void_p()
    args = PLANS[fn][0]
    for options in (mfr.Options(1, mfr.VARIANT_ROWS, 0, 0, 0), mfr.Options(1, 0, 3, 0, 0), mfr.Options(1, 0, 4, 0, 0)):
        assert getattr(lib, fn)(ctypes.byref(h), *args, ctypes.byref(options)) == INVALID
    if not torch.cuda.is_available():
        assert getattr(lib, fn)(ctypes.byref(h), *args, None) == BAD_DEVICE


def test_null_plans_are_refused(lib):
    for name in declared():
        if name.endswith("_run"):
            args = mfr.SIGNATURES[name][1]
            assert getattr(lib, name)(*[0 if a in (ctypes.c_int64, ctypes.c_float) else None for a in args]) == INVALID


def test_binding_refuses_other_types():
    with pytest.raises(ValueError, match="dtype"):
        mfr.MoeLayerPlan(4, 64, 64, 8, 2, dtype=torch.float16)
    with pytest.raises(ValueError, match="dtype"):
        mfr.GatePlan(4, 64, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="dtype"):
        mfr.QkNormRopePlan(4, 8, 2, 64, dtype=torch.float32, max_positions=10)
    with pytest.raises(ValueError, match="dtypes"):
        mfr.GradClipPlan([4, 5], [torch.float32, torch.float64])
    with pytest.raises(ValueError, match="dtypes"):
        mfr.GradClipPlan([4, 5], [torch.float32])


# ---- the binding's checks of tensors: nothing below reaches the library --------------

class _NoCall:
    def __getattr__(self, name):
        def call(*_):
            raise AssertionError(f"the binding reached {name}")
        return call


def _plan(cls, **fields):
    p = cls.__new__(cls)
    p._lib, p._h, p.device = _NoCall(), None, torch.device("cpu")
    for n, v in fields.items():
        setattr(p, n, v)
    return p


def _z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


def _layer(dtype):
    T, H, I, E, k = 4, 256, 128, 8, 2
    a = dict(x=_z(T, H, dtype=dtype), expert_ids=_z(T, k, dtype=I32), topk_weights=_z(T, k), w13=_z(E, 2 * I, H, dtype=dtype),
             w2=_z(E, H, I, dtype=dtype), out=_z(T, H, dtype=B16), workspace=_z(64, dtype=torch.uint8))
    if dtype is FP8:
        a.update(x_sf=_z(T, 2), w13_sf=_z(E, 2, 2), w2_sf=_z(E, 2, 1))
    return _plan(mfr.MoeLayerPlan, T=T, H=H, I=I, E=E, k=k, dtype=dtype, _need=64), a, "run"


def _gate(grad):
    T, E, k = 4, 64, 8
    plan = _plan(mfr.GatePlan, T=T, E=E, k=k, score=mfr.SCORE_SIGMOID, dtype=B16)
    if grad:
        return plan, dict(d_topk_weights=_z(T, k), logits=_z(T, E, dtype=B16), expert_ids=_z(T, k, dtype=I32),
                          d_logits=_z(T, E, dtype=B16)), "run_grad"
    return plan, dict(logits=_z(T, E, dtype=B16), expert_ids=_z(T, k, dtype=I32), topk_weights=_z(T, k), bias=_z(E)), "run"


def _qk(grad):
    T, hq, hk, D, most = 4, 6, 2, 64, 10
    plan = _plan(mfr.QkNormRopePlan, T=T, heads_q=hq, heads_k=hk, D=D, dtype=F16, rotary_dim=32, max_positions=most, _need=64)

    def q():
        return _z(T, hq, D, dtype=F16)

    def k():
        return _z(T, hk, D, dtype=F16)
    shared = dict(gamma_q=_z(D, dtype=F16), gamma_k=_z(D, dtype=F16), eps=1e-6, cos_sin=_z(most, 32), positions=_z(T, dtype=I32))
    if grad:
        return plan, dict(d_q_out=q(), d_k_out=k(), q=q(), k=k(), **shared, d_q=q(), d_k=k(), d_gamma_q=_z(D), d_gamma_k=_z(D),
                          workspace=_z(64, dtype=torch.uint8)), "run_grad"
    return plan, dict(q=q(), k=k(), **shared, q_out=q(), k_out=k()), "run"


CALLS = {"gate": lambda: _gate(False), "gate_grad": lambda: _gate(True), "qk": lambda: _qk(False), "qk_grad": lambda: _qk(True),
         "layer_bf16": lambda: _layer(B16), "layer_e4m3": lambda: _layer(FP8)}


@pytest.mark.parametrize("op", list(CALLS))
def test_binding_refuses_each_wrong_tensor(op):
    plan, args, fn = CALLS[op]()
    for name, t in args.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = [t[:-1], t.to(torch.float64), 5]
        if name == "workspace":
            wrong = [t[:-1], None, 5]
        elif t.dim() > 1 and name not in ("q", "k", "d_q_out", "d_k_out", "q_out", "k_out", "d_q", "d_k"):
            wrong += [t.new_zeros((*t.shape[:-1], 2 * t.shape[-1]))[..., ::2], t.reshape(-1)]
        for bad in wrong:
            with pytest.raises(ValueError, match=name if name != "workspace" else "workspace|bytes"):
                getattr(plan, fn)(**{**args, name: bad})
    plan.device = torch.device("meta")       # every tensor is on another device than the plan's
    with pytest.raises(ValueError, match="device|workspace"):
        getattr(plan, fn)(**args, stream=0)
    plan.device = torch.device("cpu")
    with pytest.raises(AssertionError, match="reached"):
        getattr(plan, fn)(**args, stream=0)


def test_a_layer_for_bf16_takes_no_scales():
    plan, args, _ = _layer(B16)
    with pytest.raises(ValueError, match="bf16"):
        plan.run(**args, w2_sf=_z(8, 2, 1))


def test_clip_refuses_each_wrong_tensor():
    plan = _plan(mfr.GradClipPlan, numels=[5, 8], dtypes=[F32, B16], _need=8, _pointers=ctypes.c_void_p * 2)
    good = [_z(5), _z(8, dtype=B16)]
    args = dict(max_norm=1.0, norm=_z(1), workspace=_z(8, dtype=torch.uint8))
    for name in ("grads", "out"):
        for i, wrong in ((0, _z(4)), (0, _z(5, dtype=B16)), (1, 5), (1, None), (1, _z(16, dtype=B16)[::2])):
            bad = list(good)
            bad[i] = wrong
            with pytest.raises(ValueError, match=rf"{name}\[{i}\]"):
                plan.run(**{"grads": good, **args, name: bad})
        with pytest.raises(ValueError, match=name):
            plan.run(**{"grads": good, **args, name: good[:1]})
    for name, wrong in (("norm", _z(2)), ("norm", _z(1, dtype=B16)), ("workspace", _z(7, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="norm|workspace"):
            plan.run(good, **{**args, name: wrong})
    with pytest.raises(AssertionError, match="reached"):
        plan.run(good, **args, stream=0)
    plan.device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="device"):
        plan.run(good, **args, stream=0)


def test_a_bias_needs_sigmoid_scores():
    plan, args, _ = _gate(False)
    plan.score = mfr.SCORE_SOFTMAX
    with pytest.raises(ValueError, match="bias"):
        plan.run(**args)


# ---- the references ----------------------------------------------------------------------

def test_reference_gradients_against_differentiation():
    g = torch.Generator().manual_seed(0)
    logits = torch.randn((3, 9), generator=g, dtype=torch.float64)
    d_w = torch.randn((3, 4), generator=g, dtype=torch.float64)
    for sigmoid in (False, True):
        for renorm in (False, True):
            ids, w, _ = ref.gate(logits, 4, sigmoid, renorm, 1.5)
            l = logits.clone().requires_grad_(True)
            p = torch.sigmoid(l) if sigmoid else torch.softmax(l, 1)
            q = torch.gather(p, 1, ids)
            q = 1.5 * (q / q.sum(1, keepdim=True) if renorm else q)
            assert torch.allclose(q.detach(), w, atol=1e-14)
            (q * d_w).sum().backward()
            assert torch.allclose(ref.gate_grad(d_w, logits, ids, sigmoid, renorm, 1.5)[0], l.grad, atol=1e-14)
    table = torch.randn((7, 16), generator=g)
    pos = torch.tensor([0, 6, 3])
    for interleaved in (False, True):
        x = torch.randn((3, 2, 24), generator=g, dtype=torch.float64, requires_grad=True)
        gamma = torch.randn(24, generator=g, dtype=torch.float64, requires_grad=True)
        d = torch.randn((3, 2, 24), generator=g, dtype=torch.float64)
        n = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + float(torch.tensor(1e-3))) * gamma
        r = n[..., :16].unflatten(-1, (8, 2)) if interleaved else n[..., :16].unflatten(-1, (2, 8)).transpose(-1, -2)
        c, s = (table[pos].double()[:, None, :8], table[pos].double()[:, None, 8:])
        z = torch.stack([r[..., 0] * c - r[..., 1] * s, r[..., 0] * s + r[..., 1] * c], -1)
        z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
        out = torch.cat([z, n[..., 16:]], -1)
        assert torch.allclose(out, ref.qk_norm(x, gamma, 1e-3, table, pos, 16, interleaved)[0], atol=1e-12)
        (out * d).sum().backward()
        d_x, _, d_g, _ = ref.qk_norm_grad(d, x, gamma, 1e-3, table, pos, 16, interleaved)
        assert torch.allclose(d_x, x.grad, atol=1e-12) and torch.allclose(d_g, gamma.grad, atol=1e-12)


def test_reference_layer_is_the_formula():
    g = torch.Generator().manual_seed(0)
    T, H, I, E, k = 3, 16, 8, 4, 2
    x, w13, w2 = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((T, H), (E, 2 * I, H), (E, H, I)))
    ids, w = torch.tensor([[0, 3], [-1, 2], [1, 1]]), torch.rand((T, k), generator=g, dtype=torch.float64)
    out, _ = ref.moe_layer(x, ids, w, w13, w2)
    for t in range(T):
        want = torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                both = w13[e] @ x[t]
                want += w[t, j] * (w2[e] @ (torch.nn.functional.silu(both[:I]) * both[I:]))
        assert torch.allclose(out[t], want, atol=1e-12)
