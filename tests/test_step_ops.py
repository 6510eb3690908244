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
    assert "moe_small_layer_run" in names
    assert not [n for n in names if not hasattr(lib, n)]
    assert names <= set(mfr.SIGNATURES)


def test_header_is_c99(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "moe_step_ops.h"\nint main(void) { moe_op_t op = 0; moe_op_destroy(op); return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", f"-I{os.path.dirname(HEADER)}", str(src)],
                   check=True)


PLANS = {
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


CALLS = {"layer_bf16": lambda: _layer(B16), "layer_e4m3": lambda: _layer(FP8)}


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
