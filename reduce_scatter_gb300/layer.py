"""Operators around the tensor-parallel GEMM, over the C ABI in
``include/dg_layer.h``: residual add with RMS norm (16- or 8-bit output),
products grouped by expert, microscaled 4-bit tensors and their product.

:mod:`reduce_scatter_gb300.ops` exports the public names.  This module checks
and marshals arguments and allocates outputs with torch; every computation runs
in ``libdg.so`` on the current stream of the inputs' device.  No call
synchronizes; each may be captured into a CUDA graph after one call outside
capture.  ``add_rms_norm`` (bf16 output) and ``grouped_matmul`` (bf16) take
part in autograd; their gradients can also be called directly.
"""

from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple

import torch

from . import dg

_TYPES = {torch.bfloat16: dg.TYPE_BF16, torch.float32: dg.TYPE_F32}
for _name, _t in (("float8_e4m3fn", dg.TYPE_E4M3), ("float8_e5m2", dg.TYPE_E5M2)):
    if hasattr(torch, _name):
        _TYPES[getattr(torch, _name)] = _t

# Every symbol include/dg_layer.h declares.
EXPORTS = ("dg_layer_add_rms_norm", "dg_layer_add_rms_norm_backward", "dg_layer_add_rms_norm_backward_workspace",
           "dg_layer_products_workspace", "dg_layer_grouped_matmul", "dg_layer_grouped_grad_workspace",
           "dg_layer_grouped_weight_grad", "dg_layer_mx4_scale_bytes", "dg_layer_mx4_quantize",
           "dg_layer_mx4_dequantize", "dg_layer_mx4_matmul", "dg_layer_check", "dg_layer_last_error")

_LIB = None
_lock = threading.Lock()
_state: dict = {}  # device index -> status word and its address
_workspaces: dict = {}  # (device index, stream) -> address of the products' workspace, and its tensor


def lib():
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
            "grouped_weight_grad": (i32, [vp, i64, vp, i64, vp, i32, vp, i32, i64, i64, i64, vp, vp, vp]),
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


def _type(t: torch.dtype, what: str) -> int:
    got = _TYPES.get(t)
    if got is None:
        raise TypeError(f"{what} must be bfloat16, float32 or a float8 type, got {t}")
    return got


# the current stream's handle without building a Stream object (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index):  # noqa: F811
        return torch.cuda.current_stream(index).cuda_stream


def _call(dev: torch.device, fn, *args):
    """``fn(*args, stream)`` on ``dev``, whose current stream is appended; raises on an error."""
    index = dev.index
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:  # the library works on the current device
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != dg.OK:
        raise dg.DGError(rc, _LIB.dg_layer_last_error().decode())


def _same_device(x: torch.Tensor, *tensors) -> torch.device:
    if not x.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    dev = x.device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on the same CUDA device")
    return dev


_COUNTER_BYTES = 2048  # DG_LAYER_COUNTER_BYTES


def _status(dev: torch.device) -> int:
    """Address of the device's status word (created on first use)."""
    st = _state.get(dev.index)
    if st is None:
        with _lock:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("make one call outside of stream capture first")
            word = torch.zeros(32, dtype=torch.int64, device=dev)
            torch.cuda.current_stream(dev).synchronize()  # zero before any stream uses it
            st = _state.setdefault(dev.index, (word, word.data_ptr()))
    return st[1]


def _workspace(dev: torch.device):
    """(address, tensor) of the products' workspace: one for each stream, whose calls run
    one after another; inside a stream capture one of the graph's own, since
    its replays may run beside the stream's later calls."""
    key = (dev.index, _raw_stream(dev.index))
    ws = _workspaces.get(key)
    capturing = torch.cuda.is_current_stream_capturing()
    if ws is None or capturing:
        with torch.cuda.device(dev):
            ws = torch.empty(lib().dg_layer_products_workspace(), dtype=torch.uint8, device=dev)
        ws[:_COUNTER_BYTES].zero_()
        if capturing:
            return ws.data_ptr(), ws
        ws = _workspaces[key] = (ws.data_ptr(), ws)
    return ws


def clear_workspaces() -> None:
    """Drop the products' cached workspaces (``ops.clear_caches`` calls this)."""
    _workspaces.clear()


def check_products(device=None) -> None:
    """Synchronize the current stream of ``device`` and raise ``dg.DGError`` if
    a product launched there since the last check gave up a pipeline wait (its
    output is then undefined)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    _call(dev, lib().dg_layer_check, _status(dev))


def _ptr(t):
    return None if t is None else t.data_ptr()


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


def _as_rows(t: torch.Tensor, hidden: int) -> torch.Tensor:
    """(..., hidden) as a matrix whose rows are contiguous; copies only where the strides leave no other way."""
    if t.dim() != 2:
        t = t.reshape(-1, hidden)
    return t if t.stride(1) == 1 or hidden == 1 else t.contiguous()


def _norm_forward(x, weight, residual, eps, out_dtype, scale, keep_rstd, inplace):
    shape = x.shape
    hidden = shape[-1]
    dev = x.device
    x2 = _as_rows(x, hidden)
    rows = x2.shape[0]
    y = torch.empty(shape, dtype=out_dtype, device=dev)
    row_scale = rstd = h = scale_in = None
    r_ptr, r_ld, r_type, h_ptr, h_ld = None, 0, 0, None, 0
    if residual is not None:
        r2 = _as_rows(residual, hidden)
        if inplace:
            if r2.data_ptr() != residual.data_ptr():
                raise ValueError("an in-place residual must have rows that are contiguous")
            h = residual
        else:
            h = torch.empty(shape, dtype=residual.dtype, device=dev)
        r_ptr, r_ld, r_type = r2.data_ptr(), r2.stride(0), _TYPES[r2.dtype]
        h_ptr, h_ld = (r_ptr, r_ld) if inplace else (h.data_ptr(), hidden)
    if out_dtype != torch.bfloat16:
        if scale is None:
            row_scale = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        elif isinstance(scale, torch.Tensor):
            if scale.numel() != 1 or scale.dtype != torch.float32:
                raise ValueError("a given scale is a number or a one-element float32 tensor")
            _same_device(x, scale)
            scale_in = scale
        else:
            scale_in = torch.full((1,), float(scale), dtype=torch.float32, device=dev)
    if keep_rstd:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    _call(dev, (_LIB or lib()).dg_layer_add_rms_norm, x2.data_ptr(), x2.stride(0), r_ptr, r_ld, r_type,
          weight.data_ptr(), _TYPES[weight.dtype], y.data_ptr(), _TYPES[out_dtype], h_ptr, h_ld, _ptr(row_scale),
          _ptr(scale_in), _ptr(rstd), rows, hidden, eps)
    return y, x if h is None else h, row_scale, rstd


class _AddRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, _, rstd = _norm_forward(x, weight, residual, eps, torch.bfloat16, None, True, False)
        ctx.save_for_backward(h, weight, rstd)
        ctx.has_residual = residual is not None
        ctx.x_dtype = x.dtype
        ctx.mark_non_differentiable(rstd)
        return (y, h, rstd) if ctx.has_residual else (y, rstd)

    @staticmethod
    def backward(ctx, dy, *rest):
        h, weight, rstd = ctx.saved_tensors
        dh = rest[0] if ctx.has_residual else None
        if dy is None:
            dy = torch.zeros(h.shape, dtype=torch.bfloat16, device=h.device)
        dx, dw = add_rms_norm_backward(dy, h, weight, rstd, d_residual=dh)
        return dx.to(ctx.x_dtype), dw, dx if ctx.has_residual else None, None


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
    ``residual``.  Differentiable with a bfloat16 output.
    """
    if x.dim() < 1 or x.dtype != torch.bfloat16:
        raise TypeError("x must be a bfloat16 tensor with a last dimension to normalise")
    hidden = x.shape[-1]
    if weight.dim() != 1 or weight.shape[0] != hidden or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous vector of {hidden} values")
    if weight.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("weight must be bfloat16 or float32")
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        if residual.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("residual must be bfloat16 or float32")
    elif inplace:
        raise ValueError("inplace needs a residual")
    if out_dtype not in _TYPES or out_dtype == torch.float32:
        raise ValueError(f"out_dtype must be bfloat16 or a float8 type, got {out_dtype}")
    if scale is not None and out_dtype == torch.bfloat16:
        raise ValueError("a scale needs a float8 out_dtype")
    _same_device(x, weight, residual)
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad or
                                    (residual is not None and residual.requires_grad)):
        if out_dtype != torch.bfloat16 or inplace:
            raise ValueError("an 8-bit output or an in-place residual has no gradient: call under torch.no_grad()")
        out = _AddRMSNorm.apply(x, weight, residual, float(eps))
        return NormResult(out[0], out[1] if residual is not None else x, None, out[-1] if keep_rstd else None)
    return NormResult(*_norm_forward(x, weight, residual, float(eps), out_dtype, scale, keep_rstd, inplace))


def add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                          d_residual: torch.Tensor | None = None):
    """``(dx, dweight)`` of :func:`add_rms_norm`: ``h`` and ``rstd`` are the
    forward's ``residual`` and ``rstd``, ``d_residual`` (h's type) the gradient
    that reaches ``h`` on its other way.  ``dx``, in h's type, is the gradient
    of both ``x`` and ``residual``."""
    hidden = h.shape[-1]
    if dy.shape != h.shape or rstd.shape != h.shape[:-1] or weight.shape != (hidden,):
        raise ValueError("dy must have h's shape, rstd that of its rows, weight that of one row")
    if d_residual is not None and (d_residual.shape != h.shape or d_residual.dtype != h.dtype):
        raise ValueError("d_residual must have h's shape and type")
    if dy.dtype != torch.bfloat16 or rstd.dtype != torch.float32:
        raise TypeError("dy must be bfloat16 and rstd float32")
    if h.dtype not in (torch.bfloat16, torch.float32) or weight.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("h and weight must be bfloat16 or float32")
    dev = _same_device(h, dy, weight, rstd, d_residual)
    dy2, h2 = _as_rows(dy, hidden), _as_rows(h, hidden)
    d2 = None if d_residual is None else _as_rows(d_residual, hidden)
    weight, rstd = weight.contiguous(), rstd.contiguous()
    rows = h2.shape[0]
    dx = torch.empty(h.shape, dtype=h.dtype, device=dev)
    dw = torch.empty_like(weight)
    L = lib()
    ws = torch.empty(L.dg_layer_add_rms_norm_backward_workspace(rows, hidden), dtype=torch.uint8, device=dev)
    _call(dev, L.dg_layer_add_rms_norm_backward, dy2.data_ptr(), dy2.stride(0), h2.data_ptr(), h2.stride(0),
          _TYPES[h2.dtype], weight.data_ptr(), _TYPES[weight.dtype], rstd.data_ptr(), _ptr(d2),
          0 if d2 is None else d2.stride(0), dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), rows, hidden)
    return dx, dw


# ---------------------------------------------------- products grouped by expert


def _pitch_ok(t: torch.Tensor, dims) -> bool:
    esz = t.element_size()
    return t.data_ptr() % 16 == 0 and all(t.stride(d) * esz % 16 == 0 for d in dims)


def _rows_operand(t: torch.Tensor) -> torch.Tensor:
    """(T, K) with contiguous, 16-byte aligned rows that do not overlap; a copy only where it is not."""
    if t.stride(1) == 1 and t.stride(0) >= t.shape[1] and _pitch_ok(t, (0,)):
        return t
    return t.contiguous() if not t.is_contiguous() else t.clone()


def _experts_operand(B: torch.Tensor, f8: bool):
    """``(tensor, row pitch, expert pitch, n_major)`` of a (E, K, N) B: used in
    place when its K rows (or, in bf16, its N rows) are contiguous and aligned."""
    E, K, N = B.shape
    if E == 1 or B.stride(0) > 0:
        if B.stride(1) == 1 and B.stride(2) >= K and _pitch_ok(B, (0, 2) if E > 1 else (2,)):
            return B, B.stride(2), B.stride(0), 0
        if not f8 and B.stride(2) == 1 and B.stride(1) >= N and _pitch_ok(B, (0, 1) if E > 1 else (1,)):
            return B, B.stride(1), B.stride(0), 1
    C = torch.empty((E, N, K), dtype=B.dtype, device=B.device)
    C.copy_(B.transpose(1, 2))
    return C, K, N * K, 0


def _grouped_check(A, B, ends):
    if A.dim() != 2 or B.dim() != 3 or B.shape[1] != A.shape[1]:
        raise ValueError(f"A must be (T, K) and B (experts, K, N), got {tuple(A.shape)} and {tuple(B.shape)}")
    if ends.dtype != torch.int32 or ends.dim() != 1 or ends.shape[0] != B.shape[0]:
        raise ValueError("group_ends must be an int32 vector with one ascending end for each expert")
    _same_device(A, B, ends)


def _scale_strides(s, shape, what):
    """A fp32 scale broadcast to ``shape``: (tensor, strides in elements, 0 where shared)."""
    if s is None:
        return None, [0] * len(shape)
    if not isinstance(s, torch.Tensor) or s.dtype != torch.float32:
        raise TypeError(f"{what} must be a float32 tensor")
    try:
        v = s.expand(shape) if s.shape != shape else s
    except RuntimeError:
        raise ValueError(f"{what} of shape {tuple(s.shape)} does not broadcast to {tuple(shape)}") from None
    return v, [v.stride(d) if v.shape[d] > 1 else 0 for d in range(len(shape))]


def _grouped_forward(A, B, ends, scale_a, scale_b, out_dtype):
    T, K = A.shape
    E, _, N = B.shape
    dev = A.device
    f8 = A.element_size() == 1
    A = _rows_operand(A) if T else A
    Bt, ld_b, ld_e, n_major = _experts_operand(B, f8)
    ends = ends if ends.is_contiguous() else ends.contiguous()
    sa, (sa_s,) = _scale_strides(scale_a, (T,), "scale_a")
    if scale_b is not None and isinstance(scale_b, torch.Tensor) and scale_b.dim() == 1 and scale_b.shape[0] == E:
        scale_b = scale_b[:, None]  # one for each expert
    sb, (sb_e, sb_n) = _scale_strides(scale_b, (E, N), "scale_b")
    _same_device(A, sa, sb)
    D = torch.empty((T, N), dtype=out_dtype, device=dev)
    ws = _workspace(dev)
    _call(dev, (_LIB or lib()).dg_layer_grouped_matmul, A.data_ptr(), A.stride(0), _TYPES[A.dtype], Bt.data_ptr(), ld_b,
          ld_e, _TYPES[B.dtype], n_major, ends.data_ptr(), E, _ptr(sa), sa_s, _ptr(sb), sb_e, sb_n, D.data_ptr(),
          _TYPES[out_dtype], T, N, K, ws[0], _status(dev))
    return D


class _GroupedMatmul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, B, ends, out_dtype):
        ctx.save_for_backward(A, B, ends)
        return _grouped_forward(A, B, ends, None, None, out_dtype)

    @staticmethod
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
    and N % 8 == 0.  Differentiable in bfloat16 without scales.
    """
    _grouped_check(A, B, group_ends)
    ta, tb = _type(A.dtype, "A"), _type(B.dtype, "B")
    if dg.TYPE_F32 in (ta, tb) or (ta == dg.TYPE_BF16) != (tb == dg.TYPE_BF16):
        raise TypeError(f"A and B must be both bfloat16 or both float8, got {A.dtype} and {B.dtype}")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    if torch.is_grad_enabled() and (A.requires_grad or B.requires_grad):
        if scale_a is not None or scale_b is not None or ta != dg.TYPE_BF16:
            raise ValueError("float8 operands and scales have no gradient: call under torch.no_grad()")
        return _GroupedMatmul.apply(A, B, group_ends, out_dtype)
    return _grouped_forward(A, B, group_ends, scale_a, scale_b, out_dtype)


def _weight_grad(rows, feats, ends, experts):
    """(experts, rows' columns, feats' columns): sum over each group of rows[t, :, None] * feats[t, None, :]."""
    T, N = rows.shape
    K = feats.shape[1]
    dev = rows.device
    if T:
        rows, feats = _rows_operand(rows), _rows_operand(feats)
    ends = ends if ends.is_contiguous() else ends.contiguous()
    out = torch.empty((experts, N, K), dtype=torch.bfloat16, device=dev)
    L = lib()
    ws = torch.empty(L.dg_layer_grouped_grad_workspace(experts, N, K), dtype=torch.uint8, device=dev)
    _call(dev, L.dg_layer_grouped_weight_grad, rows.data_ptr(), rows.stride(0), feats.data_ptr(), feats.stride(0),
          ends.data_ptr(), experts, out.data_ptr(), dg.TYPE_BF16, T, N, K, ws.data_ptr(), _status(dev))
    return out


def grouped_matmul_backward(dD: torch.Tensor, A: torch.Tensor, B: torch.Tensor, group_ends: torch.Tensor, *,
                            need=(True, True)):
    """``(dA, dB)`` of the bfloat16 :func:`grouped_matmul`: ``dA[t] = dD[t] @ B[e].T``
    (0 past the last group) and ``dB[e] = A_e.T @ dD_e`` (0 for an empty group),
    dB in B's layout; ``need``: which of the two to compute (else None)."""
    _grouped_check(A, B, group_ends)
    if dD.shape != (A.shape[0], B.shape[2]):
        raise ValueError(f"dD must be {(A.shape[0], B.shape[2])}, got {tuple(dD.shape)}")
    if not (dD.dtype == A.dtype == B.dtype == torch.bfloat16):
        raise TypeError("dD, A and B must be bfloat16")
    _same_device(A, dD)
    dA = _grouped_forward(dD, B.transpose(1, 2), group_ends, None, None, torch.bfloat16) if need[0] else None
    dB = None
    if need[1]:
        E = B.shape[0]
        if B.stride(2) == 1 and B.stride(1) != 1:  # contiguous along N
            dB = _weight_grad(A, dD, group_ends, E)
        else:
            dB = _weight_grad(dD, A, group_ends, E).transpose(1, 2)
    return dA, dB


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


def _scale_shape(rows, cols):
    return (-(-rows // 128), -(-cols // 256) * 2, 512)


def _mx4_check(q: MX4Tensor, what: str):
    if not isinstance(q, MX4Tensor):
        raise TypeError(f"{what} must be an MX4Tensor")
    rows, cols = q.rows, q.cols
    if q.codes.dtype != torch.uint8 or q.codes.shape != (rows, cols // 2) or not q.codes.is_contiguous():
        raise ValueError(f"{what}.codes must be contiguous uint8 of shape {(rows, cols // 2)}")
    if q.scales.dtype != torch.uint8 or q.scales.shape != _scale_shape(rows, cols) or not q.scales.is_contiguous():
        raise ValueError(f"{what}.scales must be contiguous uint8 of shape {_scale_shape(rows, cols)}")
    _same_device(q.codes, q.scales)


def quantize_mx4(x: torch.Tensor) -> MX4Tensor:
    """``x`` (..., cols), bfloat16 or float32, its leading dimensions flattened
    into rows, in microscaled 4 bits: for each 32 columns the scale
    2^(floor(log2 max) - 2) and the nearest codes (ties to even, saturating at
    6); a block with a NaN or an infinity becomes NaN.  cols % 32 == 0."""
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if x.dim() < 1:
        raise ValueError("x must have a last dimension")
    cols = x.shape[-1]
    dev = _same_device(x)
    x2 = _as_rows(x, cols)
    if not _pitch_ok(x2, (0,)):
        x2 = x2.contiguous() if not x2.is_contiguous() else x2.clone()
    rows = x2.shape[0]
    if cols % 32:
        raise ValueError(f"the last dimension ({cols}) must be a multiple of 32")
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty(_scale_shape(rows, cols), dtype=torch.uint8, device=dev)
    _call(dev, (_LIB or lib()).dg_layer_mx4_quantize, x2.data_ptr(), x2.stride(0), _TYPES[x2.dtype], codes.data_ptr(),
          scales.data_ptr(), rows, cols)
    return MX4Tensor(codes, scales, rows, cols)


def dequantize_mx4(q: MX4Tensor, *, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The (rows, cols) values of ``q`` in bfloat16 (exact) or float32."""
    _mx4_check(q, "q")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    dev = q.codes.device
    y = torch.empty((q.rows, q.cols), dtype=out_dtype, device=dev)
    _call(dev, (_LIB or lib()).dg_layer_mx4_dequantize, q.codes.data_ptr(), q.scales.data_ptr(), y.data_ptr(),
          _TYPES[out_dtype], q.rows, q.cols)
    return y


def mx4_matmul(a: MX4Tensor, b: MX4Tensor, *, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``a @ b.T`` over the values of two microscaled tensors: ``a`` M x K (the
    activations), ``b`` N x K (a weight as it is stored), N % 8 == 0; fp32
    accumulation, ``out_dtype`` bfloat16 or float32."""
    _mx4_check(a, "a")
    _mx4_check(b, "b")
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    dev = _same_device(a.codes, b.codes)
    D = torch.empty((a.rows, b.rows), dtype=out_dtype, device=dev)
    ws = _workspace(dev)
    _call(dev, (_LIB or lib()).dg_layer_mx4_matmul, a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(),
          b.scales.data_ptr(), D.data_ptr(), _TYPES[out_dtype], a.rows, b.rows, a.cols, ws[0], _status(dev))
    return D
