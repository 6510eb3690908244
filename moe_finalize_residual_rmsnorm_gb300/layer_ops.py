"""Binding of the operators around the finalize (include/moe_layer_ops.h):
expert sorting, row dispatch, the finalize's gradient, residual RMSNorm with
an 8-bit output, and their gradients.

Argument marshalling only, like the rest of the package: each plan checks the
tensors of a call against its shapes (the C ABI receives bare pointers) and
enqueues the kernels on the caller's stream.  Nothing is allocated on a run.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import Options, SF_ROW_MAJOR, SF_TILED_128x4, _check, load_library

__all__ = ["RoutePlan", "DispatchPlan", "FinalizeGradPlan", "ResidualNormPlan", "ResidualNormGradPlan",
           "QUANT_NONE", "QUANT_TOKEN", "QUANT_GROUP128", "QUANT_MX32", "ROW_PADDING", "ROW_UNUSED"]

QUANT_NONE, QUANT_TOKEN, QUANT_GROUP128, QUANT_MX32 = 0, 1, 2, 3
ROW_PADDING, ROW_UNUSED = -1, -2


# the handle of torch's current stream of a device: without the Stream object
# that torch.cuda.current_stream makes (2 us of an 8 us call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _tensor(name: str, t, dtype, shape, device) -> int:
    """The address of a contiguous tensor of this type, shape and device; ValueError otherwise."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on the plan's device {device}, not on {t.device}")
    return t.data_ptr()             # a torch.Tensor subclass, such as a Parameter


def _workspace(t, need: int, device):
    """(address, bytes) of a workspace tensor of any type; (None, 0) where none is needed and none given."""
    if t is None:
        if need:
            raise ValueError(f"this plan needs a workspace of {need} bytes")
        return None, 0
    if not isinstance(t, torch.Tensor) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    size = t.numel() * t.element_size()
    if size < need:
        raise ValueError(f"workspace has {size} bytes, the plan needs {need}")
    return t.data_ptr(), size


class _OpPlan:
    """What the plans share: the C handle, the device, the stream, the status word."""

    _h: Optional[int] = None

    def _make(self, where: str, *args, enable_pdl: bool, debug_checks: bool, sentinel_skip: bool = False,
              cluster_size: int = 0) -> None:
        self._lib = load_library()
        self.device = torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else None
        opt = Options(int(bool(enable_pdl)), 0, int(cluster_size), int(bool(debug_checks)), int(bool(sentinel_skip)))
        h = ctypes.c_void_p()
        _check(getattr(self._lib, where)(ctypes.byref(h), *args, ctypes.byref(opt)), where)
        self._h = h.value

    def _stream(self, stream) -> int:
        if stream is None:
            return _current_stream(self.device.index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def workspace_bytes(self) -> int:
        """Bytes of workspace that run() takes (0: none)."""
        return int(self._lib.moe_op_workspace_bytes(self._h))

    def get_status(self, stream=None) -> int:
        """Waits for the stream, returns the STATUS_* bits and clears them."""
        st = ctypes.c_int(0)
        _check(self._lib.moe_op_get_status(self._h, self._stream(stream), ctypes.byref(st)), "moe_op_get_status")
        return st.value

    def close(self) -> None:
        if self._h:
            self._lib.moe_op_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class RoutePlan(_OpPlan):
    """The (token, slot) pairs of T tokens and k slots sorted by expert, for E
    experts whose blocks of rows are padded to multiples of `align`
    (C: moe_route_plan / moe_route_run).  R is the number of rows that always
    holds every block."""

    def __init__(self, T: int, k: int, E: int, *, align: int = 1, enable_pdl: bool = True, cluster_size: int = 0,
                 debug_checks: bool = False, sentinel_skip: bool = False):
        self.T, self.k, self.E, self.align = int(T), int(k), int(E), int(align)
        self._make("moe_route_plan", self.T, self.k, self.E, self.align, enable_pdl=enable_pdl,
                   debug_checks=debug_checks, sentinel_skip=sentinel_skip, cluster_size=cluster_size)
        self.R = int(self._lib.moe_route_rows(self._h))
        self._need = self.workspace_bytes()

    def run(self, expert_ids, permuted_row_of, slot_of_row, expert_offsets, expert_counts, workspace=None,
            stream=None) -> None:
        """expert_ids int32 [T, k] -> permuted_row_of int32 [T, k], slot_of_row
        int32 [R], expert_offsets int32 [E + 1], expert_counts int32 [E]."""
        i32, dev, pairs = torch.int32, self.device, (self.T, self.k)
        ws, ws_bytes = _workspace(workspace, self._need, dev)
        _check(self._lib.moe_route_run(
            self._h, _tensor("expert_ids", expert_ids, i32, pairs, dev),
            _tensor("permuted_row_of", permuted_row_of, i32, pairs, dev),
            _tensor("slot_of_row", slot_of_row, i32, (self.R,), dev),
            _tensor("expert_offsets", expert_offsets, i32, (self.E + 1,), dev),
            _tensor("expert_counts", expert_counts, i32, (self.E,), dev), ws, ws_bytes, self._stream(stream)),
            "moe_route_run")


class DispatchPlan(_OpPlan):
    """The rows of T tokens copied into expert order, R rows, k of them a token
    (C: moe_dispatch_plan / moe_dispatch_run), and the gradient of that copy
    (C: moe_dispatch_grad_run).  `dtype`: of the rows (1, 2 or 4 bytes an
    element); `sf_bytes`: bytes of each row's scales (0: none)."""

    def __init__(self, T: int, H: int, k: int, R: Optional[int] = None, *, dtype=torch.bfloat16, sf_bytes: int = 0,
                 enable_pdl: bool = True, debug_checks: bool = False, sentinel_skip: bool = False):
        self.T, self.H, self.k = int(T), int(H), int(k)
        self.R = self.T * self.k if R is None else int(R)
        self.dtype, self.sf_bytes = dtype, int(sf_bytes)
        self._make("moe_dispatch_plan", self.T, self.H, self.k, self.R, dtype.itemsize, self.sf_bytes,
                   enable_pdl=enable_pdl, debug_checks=debug_checks, sentinel_skip=sentinel_skip)

    def _scales(self, name: str, t, rows: int):
        if self.sf_bytes == 0:
            if t is not None:
                raise ValueError(f"{name}: this plan was made without scales (sf_bytes = 0)")
            return None
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[0] != rows or \
                t.shape[1] * t.element_size() != self.sf_bytes:
            raise ValueError(f"{name}: expected [{rows}, n] with {self.sf_bytes} bytes a row")
        return _tensor(name, t, t.dtype, t.shape, self.device)

    def run(self, x, permuted_row_of, slot_of_row, rows_out, sf=None, sf_out=None, stream=None) -> None:
        """x [T, H] -> rows_out [R, H], and sf [T, n] -> sf_out [R, n]."""
        i32, dev = torch.int32, self.device
        if sf is not None and sf_out is not None and sf.dtype is not sf_out.dtype:
            raise ValueError(f"sf_out: expected {sf.dtype}, got {sf_out.dtype}")
        _check(self._lib.moe_dispatch_run(
            self._h, _tensor("x", x, self.dtype, (self.T, self.H), dev), self._scales("sf", sf, self.T),
            _tensor("permuted_row_of", permuted_row_of, i32, (self.T, self.k), dev),
            _tensor("slot_of_row", slot_of_row, i32, (self.R,), dev),
            _tensor("rows_out", rows_out, self.dtype, (self.R, self.H), dev), self._scales("sf_out", sf_out, self.R),
            self._stream(stream)), "moe_dispatch_run")

    def run_grad(self, d_rows, permuted_row_of, d_x, stream=None) -> None:
        """d_rows [R, H] -> d_x [T, H], the FP32 sum of each token's rows; plans of torch.bfloat16 without scales."""
        if self.dtype is not torch.bfloat16 or self.sf_bytes:
            raise ValueError("the gradient needs a plan of torch.bfloat16 rows without scales")
        dev = self.device
        _check(self._lib.moe_dispatch_grad_run(
            self._h, _tensor("d_rows", d_rows, self.dtype, (self.R, self.H), dev),
            _tensor("permuted_row_of", permuted_row_of, torch.int32, (self.T, self.k), dev),
            _tensor("d_x", d_x, self.dtype, (self.T, self.H), dev), self._stream(stream)), "moe_dispatch_grad_run")


class FinalizeGradPlan(_OpPlan):
    """Gradient of the finalize's weighted sum (C: moe_finalize_grad_plan /
    _run).  `grad_dtype`: of d_out, torch.bfloat16 or torch.float32."""

    def __init__(self, T: int, H: int, k: int, R: Optional[int] = None, *, grad_dtype=torch.bfloat16,
                 enable_pdl: bool = True, debug_checks: bool = False, sentinel_skip: bool = False):
        if grad_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"grad_dtype must be torch.bfloat16 or torch.float32, got {grad_dtype}")
        self.T, self.H, self.k = int(T), int(H), int(k)
        self.R = self.T * self.k if R is None else int(R)
        self.grad_dtype = grad_dtype
        self._make("moe_finalize_grad_plan", self.T, self.H, self.k, self.R, int(grad_dtype is torch.float32),
                   enable_pdl=enable_pdl, debug_checks=debug_checks, sentinel_skip=sentinel_skip)

    def run(self, d_out, expert_out, permuted_row_of, slot_of_row, topk_weights, d_expert_out, d_topk_weights,
            stream=None) -> None:
        """d_out [T, H], expert_out bf16 [R, H] -> d_expert_out bf16 [R, H], d_topk_weights FP32 [T, k]."""
        i32, f32, b16, dev = torch.int32, torch.float32, torch.bfloat16, self.device
        pairs, rows = (self.T, self.k), (self.R, self.H)
        _check(self._lib.moe_finalize_grad_run(
            self._h, _tensor("d_out", d_out, self.grad_dtype, (self.T, self.H), dev),
            _tensor("expert_out", expert_out, b16, rows, dev),
            _tensor("permuted_row_of", permuted_row_of, i32, pairs, dev),
            _tensor("slot_of_row", slot_of_row, i32, (self.R,), dev),
            _tensor("topk_weights", topk_weights, f32, pairs, dev),
            _tensor("d_expert_out", d_expert_out, b16, rows, dev),
            _tensor("d_topk_weights", d_topk_weights, f32, pairs, dev), self._stream(stream)),
            "moe_finalize_grad_run")


class ResidualNormPlan(_OpPlan):
    """Residual addition + RMSNorm, written as E4M3 with scales and / or bf16
    (C: moe_residual_rmsnorm_plan / _run).  `quant`: QUANT_TOKEN (a FP32 scale
    a token), QUANT_GROUP128 (one per 128 columns), QUANT_MX32 (an E8M0 scale
    per 32 columns, row-major or with sf_layout=SF_TILED_128x4 in the tiles
    that block-scaled GEMMs read) or QUANT_NONE (bf16 alone)."""

    def __init__(self, T: int, H: int, *, quant: int = QUANT_GROUP128, sf_layout: int = SF_ROW_MAJOR,
                 enable_pdl: bool = True, debug_checks: bool = False):
        self.T, self.H, self.quant, self.sf_layout = int(T), int(H), int(quant), int(sf_layout)
        self._make("moe_residual_rmsnorm_plan", self.T, self.H, self.quant, self.sf_layout, enable_pdl=enable_pdl,
                   debug_checks=debug_checks)

    def sf_shape(self) -> tuple:
        """Shape of out_sf: FP32 [T, 1], FP32 [T, ceil(H/128)], uint8 [T, ceil(H/32)], or the bytes of the tiled layout."""
        T, S = self.T, -(-self.H // 32)
        if self.quant == QUANT_MX32 and self.sf_layout == SF_TILED_128x4:
            return (-(-T // 128) * 128 * (-(-S // 4) * 4),)
        return {QUANT_NONE: (0,), QUANT_TOKEN: (T, 1), QUANT_GROUP128: (T, -(-self.H // 128)), QUANT_MX32: (T, S)}[self.quant]

    def run(self, x, residual_in, residual_out, gamma, eps: float, out=None, out_q=None, out_sf=None,
            stream=None) -> None:
        """residual_out = residual_in + x (may be residual_in); its RMSNorm to
        out (bf16 [T, H], optional) and to out_q (E4M3 [T, H]) with out_sf."""
        f32, b16, dev, shape = torch.float32, torch.bfloat16, self.device, (self.T, self.H)
        q = sf = None
        if self.quant != QUANT_NONE:
            q = _tensor("out_q", out_q, torch.float8_e4m3fn, shape, dev)
            sf = _tensor("out_sf", out_sf, torch.uint8 if self.quant == QUANT_MX32 else f32, self.sf_shape(), dev)
        elif out_q is not None or out_sf is not None:
            raise ValueError("out_q, out_sf: this plan was made without an 8-bit output")
        elif out is None:
            raise ValueError("out is required without an 8-bit output")
        _check(self._lib.moe_residual_rmsnorm_run(
            self._h, _tensor("x", x, b16, shape, dev), _tensor("residual_in", residual_in, f32, shape, dev),
            _tensor("residual_out", residual_out, f32, shape, dev), _tensor("gamma", gamma, b16, (self.H,), dev), eps,
            None if out is None else _tensor("out", out, b16, shape, dev), q, sf, self._stream(stream)),
            "moe_residual_rmsnorm_run")


class ResidualNormGradPlan(_OpPlan):
    """Gradient of residual addition + RMSNorm (C: moe_residual_rmsnorm_grad_plan / _run)."""

    def __init__(self, T: int, H: int, *, enable_pdl: bool = True, debug_checks: bool = False):
        self.T, self.H = int(T), int(H)
        self._make("moe_residual_rmsnorm_grad_plan", self.T, self.H, enable_pdl=enable_pdl, debug_checks=debug_checks)
        self._need = self.workspace_bytes()

    def set_wait_limit(self, limit_cycles: int) -> None:
        """SM cycles after which an on-chip wait of this plan's runs gives up and
        raises STATUS_TIMEOUT; 0: at once (C: moe_residual_rmsnorm_grad_set_wait_limit)."""
        _check(self._lib.moe_residual_rmsnorm_grad_set_wait_limit(self._h, int(limit_cycles)),
               "moe_residual_rmsnorm_grad_set_wait_limit")

    def run(self, d_out, d_residual_out, residual, gamma, eps: float, d_residual_in, d_gamma, workspace, d_x=None,
            stream=None) -> None:
        """d_out bf16, d_residual_out FP32 (None: zeros), residual FP32 (the
        forward's residual_out), all [T, H] -> d_residual_in FP32 [T, H] (may
        be d_residual_out), d_gamma FP32 [H], d_x bf16 [T, H] (optional)."""
        f32, b16, dev, shape = torch.float32, torch.bfloat16, self.device, (self.T, self.H)
        ws, ws_bytes = _workspace(workspace, self._need, dev)
        _check(self._lib.moe_residual_rmsnorm_grad_run(
            self._h, _tensor("d_out", d_out, b16, shape, dev),
            None if d_residual_out is None else _tensor("d_residual_out", d_residual_out, f32, shape, dev),
            _tensor("residual", residual, f32, shape, dev), _tensor("gamma", gamma, b16, (self.H,), dev), eps,
            _tensor("d_residual_in", d_residual_in, f32, shape, dev),
            None if d_x is None else _tensor("d_x", d_x, b16, shape, dev),
            _tensor("d_gamma", d_gamma, f32, (self.H,), dev), ws, ws_bytes, self._stream(stream)),
            "moe_residual_rmsnorm_grad_run")
