"""Python binding of the operators around the dense products.

Argument checks and marshalling only, as in the package's ``gemm``: every step
runs in the library's CUDA kernels.  Outputs that the caller does not pass are
allocated on the stream that the call runs on.
"""
from __future__ import annotations

import contextlib

import torch

import software_pipelined_tiled_gb300 as _pkg

# sptg_type values of include/sptgemm.h
TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.int8: 2, torch.float8_e4m3fn: 3}
# sptg_dtype of (operand type, output type)
_PAIRS = {(torch.float16, torch.float16): 1, (torch.float16, torch.float32): 0,
          (torch.bfloat16, torch.bfloat16): 3, (torch.bfloat16, torch.float32): 4}
_16BIT = (torch.float16, torch.bfloat16)
_empty = torch.empty


def _pitch(t, rows: int, cols: int, dtype, device, name: str) -> int:
    """Elements between the rows of a rows x cols CUDA tensor with contiguous rows."""
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor on {device}")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} must be {rows} x {cols}, not {tuple(t.shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows (stride(1) == 1)")
    if rows <= 1:
        return cols  # the stride of a single row says nothing
    if s0 < cols:
        raise ValueError(f"the rows of {name} overlap")
    return s0


def _dense(t, shape, dtype, device, name: str):
    if t.dtype != dtype or t.device != device or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")


def _matrix(t, name: str):
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")


def _on(stream):
    """Allocations inside belong to the stream that the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def _call(function, device_index: int, stream, *args):
    handle = (_pkg._current_stream(device_index) if stream is None
              else _pkg._stream_handle(stream))
    if device_index == torch.cuda.current_device():
        rc = function(*args, handle)
    else:
        with torch.cuda.device(device_index):
            rc = function(*args, handle)
    if rc != 0:
        raise _pkg.SptgError(rc, _pkg.last_error() or _pkg.status_string(rc))


def add_rms_norm(x, residual, weight, eps: float = 1e-6, out_dtype=None, h=None, y=None,
                 scales=None, stream=None):
    """Residual addition and root-mean-square norm: returns (h, y, scales).

    ``h = x + residual`` (the new residual stream, in x's type; may be x or
    residual itself), ``v = h * weight / sqrt(mean(h^2) + eps)`` in 32 bits.
    With ``out_dtype`` torch.int8 or torch.float8_e4m3fn, ``y * scales[:, None]``
    stands for v, each row scaled to the type's largest value; by default y is v
    in x's type and scales is None.  x, residual, h and y are 2-D with
    contiguous rows.
    """
    _matrix(x, "x")
    dtype, device = x.dtype, x.device
    if dtype not in _16BIT:
        raise ValueError(f"x must be float16 or bfloat16, not {dtype}")
    if out_dtype is None:
        out_dtype = dtype if y is None else y.dtype
    code = TYPES.get(out_dtype)
    if code is None or (code < 2 and out_dtype != dtype):
        raise ValueError(f"out_dtype must be int8, float8_e4m3fn or {dtype}, not {out_dtype}")
    rows, cols = x.shape
    ldx = _pitch(x, rows, cols, dtype, device, "x")
    ldr = _pitch(residual, rows, cols, dtype, device, "residual")
    _dense(weight, (cols,), dtype, device, "weight")
    with _on(stream):
        if h is None:
            h, ldh = _empty((rows, cols), dtype=dtype, device=device), cols
        else:
            ldh = _pitch(h, rows, cols, dtype, device, "h")
        if y is None:
            y, ldy = _empty((rows, cols), dtype=out_dtype, device=device), cols
        else:
            ldy = _pitch(y, rows, cols, out_dtype, device, "y")
        if code < 2:
            if scales is not None:
                raise ValueError("a 16-bit y has no scales")
        elif scales is None:
            scales = _empty(rows, dtype=torch.float32, device=device)
        else:
            _dense(scales, (rows,), torch.float32, device, "scales")
    _call((_pkg._lib or _pkg.load()).sptg_add_rms_norm, device.index, stream, rows, cols,
          TYPES[dtype], code, x.data_ptr(), ldx, residual.data_ptr(), ldr, weight.data_ptr(), eps,
          h.data_ptr(), ldh, y.data_ptr(), ldy, None if scales is None else scales.data_ptr())
    return h, y, scales


def gemm_w4(x, codes, scales, zeros=None, x_scales=None, out=None, stream=None):
    """Product with 4-bit weights: ``out = x @ W.T``, ``W[n, k] = scales[n, g] * (code - zero)``.

    x: M x K, float16 or bfloat16, or int8 or float8_e4m3fn with ``x_scales``
    (M float32, as add_rms_norm gives them); codes: N x K/2 uint8, the even
    column in the low half of a byte; scales: N x K/group in the output's type,
    for groups of 32, 64 or 128 columns; zeros: N x K/group uint8 (0 to 15), or
    None for 8 everywhere.  x, codes and out are 2-D with contiguous rows.
    Returns out (M x N, of the scales' type).
    """
    _matrix(x, "x")
    _matrix(codes, "codes")
    _matrix(scales, "scales")
    device, dtype = x.device, scales.dtype
    m, k = x.shape
    n = codes.shape[0]
    code = TYPES.get(x.dtype)
    if dtype not in _16BIT or code is None or (code < 2 and x.dtype != dtype):
        raise ValueError("x must be of the scales' 16-bit type, int8 or float8_e4m3fn")
    groups = scales.shape[1]
    group = k // groups if groups else 32
    if k % 2 or (groups and group * groups != k):
        raise ValueError(f"{groups} groups do not divide K = {k}")
    ldx = _pitch(x, m, k, x.dtype, device, "x")
    ldw = _pitch(codes, n, k // 2, torch.uint8, device, "codes")
    _dense(scales, (n, groups), dtype, device, "scales")
    if zeros is not None:
        _dense(zeros, (n, groups), torch.uint8, device, "zeros")
    if (code < 2) != (x_scales is None):
        raise ValueError("x_scales belong to 8-bit x, and to no other")
    if x_scales is not None:
        _dense(x_scales, (m,), torch.float32, device, "x_scales")
    if out is None:
        with _on(stream):
            out = _empty((m, n), dtype=dtype, device=device)
        ldo = n
    else:
        ldo = _pitch(out, m, n, dtype, device, "out")
    _call((_pkg._lib or _pkg.load()).sptg_gemm_w4, device.index, stream, m, n, k, group, code,
          TYPES[dtype], x.data_ptr(), ldx, None if x_scales is None else x_scales.data_ptr(),
          codes.data_ptr(), ldw, scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
          out.data_ptr(), ldo)
    return out


def _experts(W, rows, offsets, name: str):
    if W.dim() != 3 or not W.is_cuda or W.dtype not in _16BIT:
        raise ValueError("W must be an experts x N x K CUDA tensor, float16 or bfloat16")
    _dense(W, tuple(W.shape), W.dtype, W.device, "W")
    _matrix(rows, name)
    _dense(offsets, (W.shape[0] + 1,), torch.int32, W.device, "offsets")
    return W.shape


def _grouped(function, rows, W, offsets, width, cols, out, out_dtype, stream, name):
    e, n, k = W.shape
    t = rows.shape[0]
    dtype, device = W.dtype, W.device
    ld = _pitch(rows, t, width, dtype, device, name)
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    pair = _PAIRS.get((dtype, out_dtype))
    if pair is None:
        raise ValueError(f"the output of {dtype} operands is {dtype} or float32, not {out_dtype}")
    if out is None:
        with _on(stream):
            out = _empty((t, cols), dtype=out_dtype, device=device)
        ldo = cols
    else:
        ldo = _pitch(out, t, cols, out_dtype, device, "out")
    _call(function, device.index, stream, e, t, n, k, pair, offsets.data_ptr(), rows.data_ptr(), ld,
          W.data_ptr(), out.data_ptr(), ldo)
    return out


def grouped_gemm(X, W, offsets, out=None, out_dtype=None, stream=None):
    """Products grouped by expert: ``Y[t] = X[t] @ W[e].T`` for the rows t of expert e.

    X: T x K; W: experts x N x K, contiguous; offsets: experts + 1 int32 on the
    GPU, rows ``offsets[e]`` to ``offsets[e + 1] - 1`` belonging to expert e
    (read there: the call does not wait for them).  Rows of no expert get
    zeros.  out_dtype: the operands' type (default) or float32.  Returns Y, T x N.
    """
    _, n, k = _experts(W, X, offsets, "X")
    return _grouped((_pkg._lib or _pkg.load()).sptg_grouped_gemm, X, W, offsets, k, n, out,
                    out_dtype, stream, "X")


def grouped_gemm_dx(dY, W, offsets, out=None, out_dtype=None, stream=None):
    """Gradient of grouped_gemm by X: ``dX[t] = dY[t] @ W[e]``; dY: T x N. Returns dX, T x K."""
    _, n, k = _experts(W, dY, offsets, "dY")
    return _grouped((_pkg._lib or _pkg.load()).sptg_grouped_gemm_dx, dY, W, offsets, n, k, out,
                    out_dtype, stream, "dY")


def grouped_gemm_dw(dY, X, offsets, out=None, out_dtype=None, stream=None):
    """Gradient of grouped_gemm by W: ``dW[e] = dY[rows of e].T @ X[rows of e]``.

    dY: T x N, X: T x K; returns dW, experts x N x K (zeros for an expert
    without rows), in the operands' type (default) or float32.
    """
    _matrix(X, "X")
    _matrix(dY, "dY")
    dtype, device = X.dtype, X.device
    if dtype not in _16BIT:
        raise ValueError("X and dY must be float16 or bfloat16")
    t, k = X.shape
    n = dY.shape[1]
    e = offsets.shape[0] - 1 if offsets.dim() == 1 else -1
    _dense(offsets, (max(e, 0) + 1,), torch.int32, device, "offsets")
    ldx = _pitch(X, t, k, dtype, device, "X")
    ldy = _pitch(dY, t, n, dtype, device, "dY")
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    pair = _PAIRS.get((dtype, out_dtype))
    if pair is None:
        raise ValueError(f"the output of {dtype} operands is {dtype} or float32, not {out_dtype}")
    if out is None:
        with _on(stream):
            out = _empty((e, n, k), dtype=out_dtype, device=device)
    else:
        _dense(out, (e, n, k), out_dtype, device, "out")
    _call((_pkg._lib or _pkg.load()).sptg_grouped_gemm_dw, device.index, stream, e, t, n, k, pair,
          offsets.data_ptr(), dY.data_ptr(), ldy, X.data_ptr(), ldx, out.data_ptr())
    return out
