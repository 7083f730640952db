"""Operators around the tensor-parallel GEMM, over the C ABI in
``include/dg_layer.h``: residual add with RMS norm (16- or 8-bit output),
products grouped by expert, microscaled 4-bit tensors and their product.

:mod:`reduce_scatter_gb300.ops` exports the public names.  Arguments are checked
and marshalled, and outputs allocated with torch, by the extension
``_lib/dg_layer_torch.so`` (``csrc/torch_layer.cpp``); every computation runs in
``libdg.so`` on the current stream of the inputs' device.  There is no fallback:
without the built libraries the first call raises ``RuntimeError``.  No call
synchronizes; each may be captured into a CUDA graph after one call outside
capture.  ``add_rms_norm`` (bf16 output) and ``grouped_matmul`` (bf16) take part
in autograd; their gradients can also be called directly.  No call carries on
forward-mode tangents (``ValueError``).

Errors: ``ValueError`` / ``TypeError`` for arguments that the front end refuses,
``dg.DGError`` for what the C ABI refuses.
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import dg

EXT_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "dg_layer_torch.so")

# Every symbol include/dg_layer.h declares.
EXPORTS = ("dg_layer_add_rms_norm", "dg_layer_add_rms_norm_backward", "dg_layer_add_rms_norm_backward_workspace",
           "dg_layer_products_workspace", "dg_layer_grouped_matmul", "dg_layer_grouped_grad_workspace",
           "dg_layer_grouped_weight_grad", "dg_layer_mx4_scale_bytes", "dg_layer_mx4_quantize",
           "dg_layer_mx4_dequantize", "dg_layer_mx4_matmul", "dg_layer_check", "dg_layer_last_error")

_LIB = None
_EXT = None
_lock = threading.Lock()


def lib():
    """The C ABI through ctypes, for callers without torch tensors."""
    global _LIB
    if _LIB is None:
        L = dg.lib()
        i64, i32, vp, f32, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
        sigs = {
            "add_rms_norm": (i32, [vp, i64, vp, i64, i32, vp, i32, vp, i32, vp, i64, vp, vp, vp, i64, i64, f32, vp]),
            "add_rms_norm_backward_workspace": (sz, [i64, i64]),
            "add_rms_norm_backward": (i32, [vp, i64, vp, i64, i32, vp, i32, vp, vp, i64, vp, vp, vp, i64, i64, vp]),
            "products_workspace": (sz, []),
            "grouped_matmul": (i32, [vp, i64, i32, vp, i64, i64, i32, i32, vp, i32, vp, i64, vp, i64, i64, vp, i32,
                                     i64, i64, i64, vp, vp, vp]),
            "grouped_grad_workspace": (sz, [i32, i64, i64]),
            "grouped_weight_grad": (i32, [vp, i64, vp, i64, vp, i32, vp, i32, i64, i64, i64, vp, vp, vp, vp]),
            "mx4_scale_bytes": (sz, [i64, i64]),
            "mx4_quantize": (i32, [vp, i64, i32, vp, vp, i64, i64, vp]),
            "mx4_dequantize": (i32, [vp, vp, vp, i32, i64, i64, vp]),
            "mx4_matmul": (i32, [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, vp, vp]),
            "check": (i32, [vp, vp]),
            "last_error": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, "dg_layer_" + name)
            fn.restype, fn.argtypes = res, args
        _LIB = L
    return _LIB


def _load():
    """The extension; raises if it has not been built."""
    global _EXT
    with _lock:
        if _EXT is None:
            if not os.path.exists(EXT_PATH):
                raise RuntimeError(f"{EXT_PATH} is missing: build it with __graft_entry__.build()")
            dg.lib()
            spec = importlib.util.spec_from_file_location("dg_layer_torch", EXT_PATH)
            ext = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(ext)
            ext.set_error(dg.DGError)
            _EXT = ext
    return _EXT


def check_products(device=None) -> None:
    """Synchronize the current stream of ``device`` and raise ``dg.DGError`` if
    a product launched there since the last check gave up a pipeline wait (its
    output is then undefined)."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    (_EXT or _load()).check(torch.cuda.current_device() if dev.index is None else dev.index)


def clear_workspaces() -> None:
    """Drop the products' cached workspaces (``ops.clear_caches`` calls this)."""
    if _EXT is not None:
        _EXT.clear_workspaces()


# ------------------------------------------------------- residual add + norm


class NormResult(NamedTuple):
    """``y``: the normed rows; ``residual``: the new residual stream (``x``
    itself without a residual); ``scale``: the fp32 scale of each row of an
    8-bit ``y`` (else None); ``rstd``: the rows' reciprocal deviations (with
    ``keep_rstd``, else None)."""

    y: torch.Tensor
    residual: torch.Tensor
    scale: torch.Tensor | None
    rstd: torch.Tensor | None


class _AddRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, _, rstd = (_EXT or _load()).add_rms_norm(x, weight, residual, eps, torch.bfloat16, None, True, False)
        ctx.save_for_backward(h, weight, rstd)
        ctx.has_residual = residual is not None
        ctx.mark_non_differentiable(rstd)
        return (y, h, rstd) if ctx.has_residual else (y, rstd)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, *rest):
        h, weight, rstd = ctx.saved_tensors
        dh = rest[0] if ctx.has_residual else None
        dx, dw = add_rms_norm_backward(dy, h, weight, rstd, d_residual=dh)
        return dx.to(torch.bfloat16), dw, dx if ctx.has_residual else None, None


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor | None = None, eps: float = 1e-5,
                 out_dtype: torch.dtype = torch.bfloat16, scale=None, keep_rstd: bool = False,
                 inplace: bool = False) -> NormResult:
    """``h = x + residual`` (rounded to the residual's type) and
    ``y = h * rsqrt(mean(h * h) + eps) * weight`` over the last dimension.

    ``x`` (..., H) bfloat16; ``residual`` of x's shape, bfloat16 or float32;
    ``weight`` (H,) bfloat16 or float32.  ``out_dtype``: bfloat16, or a float8
    type: then each row has its own scale ``max|y| / largest finite value``
    (the result's ``scale``; ``y * scale[..., None]`` are the values), or, with
    ``scale`` (a number or a one-element float32 tensor), the one given --
    ``fused_all_gather_scaled_matmul`` takes such rows with ``A_scale=scale``,
    ``grouped_matmul`` rows with either.  ``inplace`` writes the sum over
    ``residual`` (and raises its version, as torch's in-place operations do); its
    rows may not overlap, nor share memory with the weight or with x other than
    x's same values.  Differentiable with a bfloat16 output.
    """
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad or
                                    (residual is not None and residual.requires_grad) or
                                    (scale is not None and getattr(scale, "requires_grad", False))):
        if out_dtype != torch.bfloat16 or inplace:
            raise ValueError("an 8-bit output or an in-place residual has no gradient: call under torch.no_grad()")
        if scale is not None:
            raise ValueError("a scale needs a float8 out_dtype")
        out = _AddRMSNorm.apply(x, weight, residual, eps)
        return NormResult(out[0], out[1] if residual is not None else x, None, out[-1] if keep_rstd else None)
    return NormResult(*(_EXT or _load()).add_rms_norm(x, weight, residual, eps, out_dtype, scale, bool(keep_rstd),
                                                      bool(inplace)))


def add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                          d_residual: torch.Tensor | None = None):
    """``(dx, dweight)`` of :func:`add_rms_norm`: ``h`` and ``rstd`` are the
    forward's ``residual`` and ``rstd``, ``d_residual`` (h's type) the gradient
    that reaches ``h`` on its other way.  ``dx``, in h's type, is the gradient
    of both ``x`` and ``residual``."""
    return (_EXT or _load()).add_rms_norm_backward(dy, h, weight, rstd, d_residual)


# ---------------------------------------------------- products grouped by expert


class _GroupedMatmul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, B, ends, out_dtype):
        ctx.save_for_backward(A, B, ends)
        return (_EXT or _load()).grouped_matmul(A, B, ends, None, None, out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dD):
        A, B, ends = ctx.saved_tensors
        dA, dB = grouped_matmul_backward(dD.to(torch.bfloat16), A, B, ends, need=ctx.needs_input_grad[:2])
        return dA, dB, None, None


def grouped_matmul(A: torch.Tensor, B: torch.Tensor, group_ends: torch.Tensor, *, scale_a=None, scale_b=None,
                   out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``D[t] = A[t] @ B[e]`` for the rows ``group_ends[e - 1] <= t < group_ends[e]``.

    ``A`` (T, K): the rows sorted by expert; ``B`` (experts, K, N), of A's type
    family (bfloat16, or both float8); ``group_ends``: int32 on the device, so
    that a router's counts need no trip to the host (ends are clamped to
    [previous end, T]; a group may be empty; rows past the last end give 0).
    B is read in place as the transposed view of contiguous (experts, N, K)
    weights, or, in bfloat16, as contiguous (experts, K, N); any other layout
    is copied.  ``scale_a`` (T,) or one element, ``scale_b`` (experts, N),
    (experts,) or one element: float32 factors of D's rows and of each expert's
    columns.  ``out_dtype``: bfloat16 or float32.  K % 8 == 0 (16 for float8)
    and N % 8 == 0.  Differentiable in bfloat16 without scales (the gradients are
    products of bfloat16 operands, accumulated in fp32).
    """
    if torch.is_grad_enabled() and (A.requires_grad or B.requires_grad or
                                    (scale_a is not None and getattr(scale_a, "requires_grad", False)) or
                                    (scale_b is not None and getattr(scale_b, "requires_grad", False))):
        if scale_a is not None or scale_b is not None or A.dtype != torch.bfloat16:
            raise ValueError("float8 operands and scales have no gradient: call under torch.no_grad()")
        return _GroupedMatmul.apply(A, B, group_ends, out_dtype)
    return (_EXT or _load()).grouped_matmul(A, B, group_ends, scale_a, scale_b, out_dtype)


def grouped_matmul_backward(dD: torch.Tensor, A: torch.Tensor, B: torch.Tensor, group_ends: torch.Tensor, *,
                            need=(True, True)):
    """``(dA, dB)`` of the bfloat16 :func:`grouped_matmul`: ``dA[t] = dD[t] @ B[e].T``
    (0 past the last group) and ``dB[e] = A_e.T @ dD_e`` (0 for an empty group),
    dB in B's layout; ``need``: which of the two to compute (else None)."""
    return (_EXT or _load()).grouped_matmul_backward(dD, A, B, group_ends, bool(need[0]), bool(need[1]))


# --------------------------------------------------------- microscaled 4 bits


class MX4Tensor(NamedTuple):
    """A rows x cols matrix in OCP microscaled 4 bits: ``codes`` (rows,
    cols / 2) uint8, two e2m1 codes to a byte, the even column in the low half;
    ``scales`` uint8, one e8m0 byte (2^(byte - 127), 255 = NaN) for each 32
    columns, in tiles of 128 rows x 4 scales: shape (ceil(rows / 128),
    2 * ceil(cols / 256), 512), row r and scale s of a tile at
    ``(r % 32) * 16 + (r // 32) * 4 + s``, absent ones 0."""

    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int


def quantize_mx4(x: torch.Tensor) -> MX4Tensor:
    """``x`` (..., cols), bfloat16 or float32, its leading dimensions flattened
    into rows, in microscaled 4 bits: for each 32 columns the scale
    2^(floor(log2 max) - 2) and the nearest codes (ties to even, saturating at
    6); a block with a NaN or an infinity becomes NaN.  cols % 32 == 0.  Not
    differentiable: an ``x`` that requires a gradient is refused outside
    ``torch.no_grad()``."""
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("4-bit codes have no gradient: call under torch.no_grad(), or on x.detach()")
    return MX4Tensor(*(_EXT or _load()).quantize_mx4(x))


def dequantize_mx4(q: MX4Tensor, *, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The (rows, cols) values of ``q`` in bfloat16 (exact) or float32."""
    return (_EXT or _load()).dequantize_mx4(q, out_dtype)


def mx4_matmul(a: MX4Tensor, b: MX4Tensor, *, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``a @ b.T`` over the values of two microscaled tensors: ``a`` M x K (the
    activations), ``b`` N x K (a weight as it is stored), N % 8 == 0; fp32
    accumulation, ``out_dtype`` bfloat16 or float32."""
    return (_EXT or _load()).mx4_matmul(a, b, out_dtype)
