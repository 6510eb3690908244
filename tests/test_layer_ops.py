"""The operators around the finalize, without a GPU: the header is plain C,
every symbol is exported and bound, and plans and calls refuse what they
cannot do before any device is touched."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import layer_ref as ref
import moe_finalize_residual_rmsnorm_gb300 as mfr
import workloads as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_layer_ops.h")


@pytest.fixture(scope="module")
def lib():
    mfr.build()
    return mfr.load_library()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"\b(moe_\w+)\s*\(", text))


def test_every_declared_symbol_is_exported_and_bound(lib):
    names = declared()
    assert {"moe_route_run", "moe_dispatch_run", "moe_dispatch_grad_run", "moe_finalize_grad_run",
            "moe_residual_rmsnorm_run", "moe_residual_rmsnorm_grad_run", "moe_op_destroy"} <= names
    assert not [n for n in names if not hasattr(lib, n)]
    assert names <= set(mfr.SIGNATURES)


def test_header_is_c99(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "moe_layer_ops.h"\nint main(void) { moe_op_t op = 0; moe_op_destroy(op); return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", f"-I{os.path.dirname(HEADER)}", str(src)],
                   check=True)


INVALID, SHAPE, BAD_DEVICE = 1, 2, 4


@pytest.mark.parametrize("fn,args,code", [
    ("moe_route_plan", (-1, 8, 16, 1), INVALID),
    ("moe_route_plan", (1 << 62, 8, 16, 1), SHAPE),
    ("moe_route_plan", (4, 0, 16, 1), SHAPE),
    ("moe_route_plan", (4, 17, 16, 1), SHAPE),
    ("moe_route_plan", (4, 8, 0, 1), SHAPE),
    ("moe_route_plan", (4, 8, 1025, 1), SHAPE),
    ("moe_route_plan", (4, 8, 16, 0), SHAPE),
    ("moe_route_plan", (4, 8, 16, 4097), SHAPE),
    ("moe_route_plan", ((1 << 26) + 1, 1, 8, 1), SHAPE),
    ("moe_dispatch_plan", (4, 4096, 8, -1, 2, 0), INVALID),
    ("moe_dispatch_plan", (4, 4096, 8, 1 << 31, 2, 0), SHAPE),
    ("moe_dispatch_plan", (4, 4096, 8, 32, 3, 0), INVALID),
    ("moe_dispatch_plan", (4, 4096, 8, 32, 2, -4), INVALID),
    ("moe_dispatch_plan", (4, 4096, 8, 32, 2, 65537), INVALID),
    ("moe_dispatch_plan", (4, 4100, 8, 32, 2, 0), SHAPE),
    ("moe_dispatch_plan", (4, 4104, 8, 32, 1, 0), SHAPE),
    ("moe_dispatch_plan", (4, 16400, 8, 32, 2, 0), SHAPE),
    ("moe_dispatch_plan", (4, 4096, 17, 32, 2, 0), SHAPE),
    ("moe_finalize_grad_plan", (4, 4100, 8, 32, 0), SHAPE),
    ("moe_finalize_grad_plan", (4, 4096, 8, 32, 2), INVALID),
    ("moe_finalize_grad_plan", (-4, 4096, 8, 32, 0), INVALID),
    ("moe_residual_rmsnorm_plan", (4, 4096, 4, 0), INVALID),
    ("moe_residual_rmsnorm_plan", (4, 4096, -1, 0), INVALID),
    ("moe_residual_rmsnorm_plan", (4, 4096, 2, 1), INVALID),      # tiled scales only with MX32
    ("moe_residual_rmsnorm_plan", (4, 4096, 3, 2), INVALID),
    ("moe_residual_rmsnorm_plan", (4, 4100, 2, 0), SHAPE),
    ("moe_residual_rmsnorm_plan", (4, 16392, 2, 0), SHAPE),
    ("moe_residual_rmsnorm_grad_plan", (4, 0), SHAPE),
    ("moe_residual_rmsnorm_grad_plan", (1 << 40, 4096), SHAPE),
])
def test_plans_refuse_what_they_cannot_do(lib, fn, args, code):
    h = ctypes.c_void_p(123)
    assert getattr(lib, fn)(ctypes.byref(h), *args, None) == code
    assert not h.value
    assert lib.moe_finalize_rmsnorm_last_error().decode()
    assert getattr(lib, fn)(None, *args, None) == INVALID


@pytest.mark.parametrize("fn,args", [("moe_route_plan", (4, 8, 16, 1)), ("moe_dispatch_plan", (4, 64, 8, 32, 2, 0)),
                                     ("moe_finalize_grad_plan", (4, 64, 8, 32, 0)),
                                     ("moe_residual_rmsnorm_plan", (4, 64, 2, 0)),
                                     ("moe_residual_rmsnorm_grad_plan", (4, 64))])
def test_plans_refuse_options_that_are_not_theirs(lib, fn, args):
    h = ctypes.c_void_p()
    assert getattr(lib, fn)(ctypes.byref(h), *args, ctypes.byref(mfr.Options(1, mfr.VARIANT_ROWS, 0, 0, 0))) == INVALID
    assert getattr(lib, fn)(ctypes.byref(h), *args, ctypes.byref(mfr.Options(1, 0, 3, 0, 0))) == INVALID
    if fn != "moe_route_plan":
        assert getattr(lib, fn)(ctypes.byref(h), *args, ctypes.byref(mfr.Options(1, 0, 4, 0, 0))) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU answer")
def test_plans_without_a_gpu_report_a_bad_device(lib):
    for make in (lambda: mfr.RoutePlan(4, 8, 16), lambda: mfr.DispatchPlan(4, 64, 8), lambda: mfr.FinalizeGradPlan(4, 64, 8),
                 lambda: mfr.ResidualNormPlan(4, 64), lambda: mfr.ResidualNormGradPlan(4, 64)):
        with pytest.raises(mfr.MFRError) as e:
            make()
        assert e.value.code == BAD_DEVICE


def test_null_plans_are_refused(lib):
    st = ctypes.c_int(0)
    assert lib.moe_op_get_status(None, None, ctypes.byref(st)) == INVALID
    assert lib.moe_op_workspace_bytes(None) == -1
    assert lib.moe_route_rows(None) == -1
    assert lib.moe_residual_rmsnorm_sf_bytes(None) == -1
    for name, (res, args) in mfr.SIGNATURES.items():
        if name.startswith(("moe_route", "moe_dispatch", "moe_finalize_grad", "moe_residual")) and name.endswith("_run"):
            assert getattr(lib, name)(*[0 if a in (ctypes.c_int64, ctypes.c_float) else None for a in args]) == INVALID
    lib.moe_op_destroy(None)


def test_finalize_grad_refuses_other_gradient_types():
    with pytest.raises(ValueError, match="grad_dtype"):
        mfr.FinalizeGradPlan(4, 64, 8, grad_dtype=torch.float16)


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


T, H, K, R, E = 4, 64, 8, 40, 16


def _calls():
    i32, f32, b16 = torch.int32, torch.float32, torch.bfloat16
    z = torch.zeros
    q = dict(out_q=z((T, H), dtype=torch.float8_e4m3fn), out_sf=z((T, 1), dtype=f32))
    return {
        "route": (_plan(mfr.RoutePlan, T=T, k=K, E=E, align=1, R=R, _need=0),
                  dict(expert_ids=z((T, K), dtype=i32), permuted_row_of=z((T, K), dtype=i32), slot_of_row=z((R,), dtype=i32),
                       expert_offsets=z((E + 1,), dtype=i32), expert_counts=z((E,), dtype=i32)), "run"),
        "dispatch": (_plan(mfr.DispatchPlan, T=T, H=H, k=K, R=R, dtype=b16, sf_bytes=8),
                     dict(x=z((T, H), dtype=b16), permuted_row_of=z((T, K), dtype=i32), slot_of_row=z((R,), dtype=i32),
                          rows_out=z((R, H), dtype=b16), sf=z((T, 2)), sf_out=z((R, 2))), "run"),
        "dispatch_grad": (_plan(mfr.DispatchPlan, T=T, H=H, k=K, R=R, dtype=b16, sf_bytes=0),
                          dict(d_rows=z((R, H), dtype=b16), permuted_row_of=z((T, K), dtype=i32), d_x=z((T, H), dtype=b16)),
                          "run_grad"),
        "finalize_grad": (_plan(mfr.FinalizeGradPlan, T=T, H=H, k=K, R=R, grad_dtype=f32),
                          dict(d_out=z((T, H)), expert_out=z((R, H), dtype=b16), permuted_row_of=z((T, K), dtype=i32),
                               slot_of_row=z((R,), dtype=i32), topk_weights=z((T, K)), d_expert_out=z((R, H), dtype=b16),
                               d_topk_weights=z((T, K))), "run"),
        "residual_norm": (_plan(mfr.ResidualNormPlan, T=T, H=H, quant=mfr.QUANT_GROUP128, sf_layout=0),
                          dict(x=z((T, H), dtype=b16), residual_in=z((T, H)), residual_out=z((T, H)),
                               gamma=z((H,), dtype=b16), eps=1e-6, **q), "run"),
        "residual_norm_grad": (_plan(mfr.ResidualNormGradPlan, T=T, H=H, _need=64),
                               dict(d_out=z((T, H), dtype=b16), d_residual_out=z((T, H)), residual=z((T, H)),
                                    gamma=z((H,), dtype=b16), eps=1e-6, d_residual_in=z((T, H)), d_gamma=z((H,)),
                                    workspace=z((64,), dtype=torch.uint8), d_x=z((T, H), dtype=b16)), "run"),
    }


@pytest.mark.parametrize("op", list(_calls()))
def test_binding_refuses_each_wrong_tensor(op):
    plan, args, fn = _calls()[op]
    for name, t in args.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = [t[:-1], t.to(torch.float64), t.cpu().numpy() if t.dtype not in (torch.bfloat16, torch.float8_e4m3fn) else 5]
        if t.dim() == 2 and name not in ("sf", "sf_out", "out_sf"):
            wrong += [torch.zeros((t.shape[1], t.shape[0]), dtype=t.dtype).t(), t.new_zeros((t.shape[0], 2 * t.shape[1]))[:, ::2]]
        if name in ("workspace",):
            wrong = [t[:-1], None, 5]
        for bad in wrong:
            with pytest.raises(ValueError, match=name if name not in ("workspace",) else "workspace|bytes"):
                getattr(plan, fn)(**{**args, name: bad})
        plan.device = torch.device("meta")       # every tensor is on another device than the plan's
        with pytest.raises(ValueError, match="device|workspace"):
            getattr(plan, fn)(**args, stream=0)
        plan.device = torch.device("cpu")
    with pytest.raises(AssertionError, match="reached"):
        getattr(plan, fn)(**args, stream=0)


def test_binding_refuses_outputs_that_the_plan_does_not_have():
    p, a, _ = _calls()["residual_norm"]
    p.quant = mfr.QUANT_NONE
    with pytest.raises(ValueError, match="8-bit"):
        p.run(**a)
    a["out_q"] = a["out_sf"] = None
    with pytest.raises(ValueError, match="out is required"):
        p.run(**a)
    p, a, _ = _calls()["dispatch"]
    with pytest.raises(ValueError, match="sf_out"):
        p.run(**{**a, "sf_out": a["sf_out"].to(torch.int32)})
    p.sf_bytes = 0
    with pytest.raises(ValueError, match="without scales"):
        p.run(**a)
    p, a, _ = _calls()["dispatch_grad"]
    p.dtype = torch.float16
    with pytest.raises(ValueError, match="bfloat16"):
        p.run_grad(**a)


# ---- the references --------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 3, 7), (40, 8, 16)])
def test_reference_route_is_the_grouped_layout(T, k, E):
    ids = ref.draw_ids(T, k, E, seed=T)
    row_of, slot_of, offsets, counts = ref.route(ids, E, 1)
    assert np.array_equal(row_of, W.grouped_index_map(ids))
    assert np.array_equal(row_of.reshape(-1)[slot_of], np.arange(T * k))
    assert offsets[-1] == T * k == counts.sum()


def test_reference_gradients_against_differences():
    """The references' gradients against central differences in 64 bits."""
    rng = np.random.default_rng(3)
    T, H, k = 3, 16, 2
    row_of, slot_of, *_ = ref.route(ref.draw_ids(T, k, 4, seed=1), 4, 1)
    E, w, g = rng.normal(size=(T * k, H)), rng.random((T, k)), rng.normal(size=(T, H))

    def loss(E, w):
        return sum(g[t] @ sum(w[t, j] * E[row_of[t, j]] for j in range(k)) for t in range(T))
    d_rows, d_w, _ = ref.finalize_grad(g, E, row_of, slot_of, w)
    h = 1e-6
    for _ in range(5):
        dE, dw = rng.normal(size=E.shape), rng.normal(size=w.shape)
        diff = (loss(E + h * dE, w + h * dw) - loss(E - h * dE, w - h * dw)) / (2 * h)
        assert abs(diff - (d_rows * dE).sum() - (d_w * dw).sum()) < 1e-7 * (1 + abs(diff))
    r, gamma, g_r = rng.normal(size=(T, H)), rng.normal(size=H), rng.normal(size=(T, H))
    eps = float(np.float32(1e-3))

    def loss_norm(r, gamma):
        return (g * (r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * gamma)).sum() + (g_r * r).sum()
    d_r, _, d_gamma, _ = ref.residual_norm_grad(g, g_r, r, gamma, eps)
    for _ in range(5):
        dr, dg = rng.normal(size=r.shape), rng.normal(size=H)
        diff = (loss_norm(r + h * dr, gamma + h * dg) - loss_norm(r - h * dr, gamma - h * dg)) / (2 * h)
        assert abs(diff - (d_r * dr).sum() - (d_gamma * dg).sum()) < 1e-7 * (1 + abs(diff))
