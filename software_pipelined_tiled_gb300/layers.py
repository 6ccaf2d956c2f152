"""Python binding of the operators around the dense products.

Argument checks and marshalling only, as in the package's ``gemm``: every step
runs in the library's CUDA kernels.  Outputs that the caller does not pass are
allocated on the stream that the call runs on.

``stream`` (a torch.cuda.Stream or a raw handle; by default PyTorch's current
stream) is where a call runs.  It does not wait for any other: what was written
on another stream has to be waited for first (``stream.wait_stream``), as has the
call itself before its results are used elsewhere.  The tensors passed may be
dropped as soon as the call returns: the allocator learns that the stream uses them.

``grouped_gemm`` takes part in PyTorch's automatic differentiation; the other
calls, like ``gemm``, return tensors without a history.

A decoding step makes these calls for every layer and token, so the checks are
written for little time: each looks at attributes only, and what a message
needs is worked out when a check has failed.
"""
from __future__ import annotations

import ctypes

import torch

import software_pipelined_tiled_gb300 as _pkg

# sptg_type values of include/sptgemm.h
TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.int8: 2, torch.float8_e4m3fn: 3}
# sptg_dtype of (operand type, output type)
_PAIRS = {(torch.float16, torch.float16): 1, (torch.float16, torch.float32): 0,
          (torch.bfloat16, torch.bfloat16): 3, (torch.bfloat16, torch.float32): 4}
_16BIT = (torch.float16, torch.bfloat16)
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_new = torch.empty

_lib = _pkg.load()
_norm, _norm_ex, _w4 = _lib.sptg_add_rms_norm, _lib.sptg_add_rms_norm_ex, _lib.sptg_gemm_w4
_y, _dx, _dw = _lib.sptg_grouped_gemm, _lib.sptg_grouped_gemm_dx, _lib.sptg_grouped_gemm_dw
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _pkg._current_stream)


def _refuse(name: str, t, want: str):
    raise ValueError(f"{name} must be {want}; it is {t.dtype} of shape {tuple(t.shape)} with "
                     f"strides {t.stride()} on {t.device}")


def _pitch(t, rows: int, cols: int, dtype, device: int, name: str) -> int:
    """Elements between the rows of a rows x cols CUDA tensor with contiguous rows."""
    if t.dtype is dtype and t.get_device() == device and t.shape == (rows, cols):
        if t.is_contiguous():
            return cols
        s0, s1 = t.stride()
        if s0 >= cols and (s1 == 1 or cols == 1):
            return s0
        if rows <= 1 and s1 == 1:
            return cols  # the pitch of one row says nothing
    _refuse(name, t, f"a {rows} x {cols} {dtype} tensor with contiguous rows that do not overlap, "
                     f"on CUDA device {device}")


def _dense(t, shape, dtype, device: int, name: str):
    if not (t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous()):
        _refuse(name, t, f"a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA device {device}")


def _matrix(t, name: str):
    if t.dim() != 2 or not t.is_cuda:
        _refuse(name, t, "a 2-D CUDA tensor")


def _stream(stream, device):
    """PyTorch's stream object for a stream object or a raw handle (None: the current stream)."""
    return torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream that the call runs on."""
    if stream is None:
        return _new(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream(stream, device)):
        return _new(shape, dtype=dtype, device=device)


def _call(function, device: int, stream, args, tensors):
    if stream is None:
        handle = _raw_stream(device)
    else:
        handle = _pkg._stream_handle(stream)
        user = _stream(stream, device)
        for t in tensors:
            if t is not None:
                t.record_stream(user)
    if device == _current_device():
        rc = function(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = function(*args, handle)
    if rc:
        raise _pkg.SptgError(rc, _pkg.last_error() or _pkg.status_string(rc))


def add_rms_norm(x, residual, weight, eps: float = 1e-6, out_dtype=None, h=None, y=None,
                 scales=None, stream=None, config=None):
    """Residual addition and root-mean-square norm: returns (h, y, scales).

    ``h = x + residual`` (the new residual stream, in x's type; may be x or
    residual itself), ``v = h * weight / sqrt(mean(h^2) + eps)`` in 32 bits.
    With ``out_dtype`` torch.int8 or torch.float8_e4m3fn, ``y * scales[:, None]``
    stands for v, each row scaled to the type's largest value; by default y is v
    in x's type and scales is None.  Rows without columns have scales of 0.  x,
    residual, h and y are 2-D with contiguous rows.  config: a Config, for its timeout_ms and inject_stall.
    """
    if x.dim() != 2 or not x.is_cuda:
        _refuse("x", x, "a 2-D CUDA tensor")
    dtype, device, shape = x.dtype, x.get_device(), x.shape
    rows, cols = shape
    if out_dtype is None:
        out_dtype = dtype if y is None else y.dtype
    in_code, code = TYPES.get(dtype, 9), TYPES.get(out_dtype, 9)
    if in_code > 1 or code > 3 or (code < 2 and code != in_code):
        raise ValueError(f"x must be float16 or bfloat16 and out_dtype int8, float8_e4m3fn or x's "
                         f"type, not {dtype} and {out_dtype}")
    ldx = cols if x.is_contiguous() else _pitch(x, rows, cols, dtype, device, "x")
    ldr = _pitch(residual, rows, cols, dtype, device, "residual")
    _dense(weight, (cols,), dtype, device, "weight")
    on = x.device
    if h is None:
        h, ldh = _empty(shape, dtype, on, stream), cols
    else:
        ldh = _pitch(h, rows, cols, dtype, device, "h")
    if y is None:
        y, ldy = _empty(shape, out_dtype, on, stream), cols
    else:
        ldy = _pitch(y, rows, cols, out_dtype, device, "y")
    if code < 2:
        if scales is not None:
            raise ValueError("a 16-bit y has no scales")
        s = None
    else:
        if scales is None:
            scales = _empty((rows,), _F32, on, stream)
        else:
            _dense(scales, (rows,), _F32, device, "scales")
        s = scales.data_ptr()
        if not cols:  # the library does nothing for rows without columns: their largest value is 0
            with torch.cuda.stream(_stream(stream, on)):
                scales.zero_()
    function = _norm
    if config is not None:
        function = lambda *args: _norm_ex(*args, ctypes.byref(config))  # noqa: E731
    _call(function, device, stream, (
        rows, cols, in_code, code, x.data_ptr(), ldx, residual.data_ptr(), ldr, weight.data_ptr(),
        eps, h.data_ptr(), ldh, y.data_ptr(), ldy, s), (x, residual, weight, h, y, scales))
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
    if x.dim() != 2 or codes.dim() != 2 or scales.dim() != 2 or not x.is_cuda:
        for name, t in (("x", x), ("codes", codes), ("scales", scales)):
            _matrix(t, name)
    device, dtype, (m, k), (n, groups) = x.get_device(), scales.dtype, x.shape, scales.shape
    code, out_code = TYPES.get(x.dtype, 9), TYPES.get(dtype, 9)
    if out_code > 1 or code > 3 or (code < 2 and code != out_code):
        raise ValueError("x must be of the scales' 16-bit type, int8 or float8_e4m3fn")
    group = k // groups if groups else 32
    if k % 2 or group * groups != k:
        raise ValueError(f"{groups} groups do not divide K = {k}")
    ldx = _pitch(x, m, k, x.dtype, device, "x")
    ldw = _pitch(codes, n, k // 2, _U8, device, "codes")
    _dense(scales, (n, groups), dtype, device, "scales")
    if zeros is not None:
        _dense(zeros, (n, groups), _U8, device, "zeros")
    if (code < 2) != (x_scales is None):
        raise ValueError("x_scales belong to 8-bit x, and to no other")
    if x_scales is not None:
        _dense(x_scales, (m,), _F32, device, "x_scales")
    if out is None:
        out, ldo = _empty((m, n), dtype, x.device, stream), n
    else:
        ldo = _pitch(out, m, n, dtype, device, "out")
    _call(_w4, device, stream, (
        m, n, k, group, code, out_code, x.data_ptr(), ldx,
        None if x_scales is None else x_scales.data_ptr(), codes.data_ptr(), ldw,
        scales.data_ptr(), None if zeros is None else zeros.data_ptr(), out.data_ptr(), ldo),
        (x, codes, scales, zeros, x_scales, out))
    return out


def _pair(dtype, out, out_dtype):
    """The library's dtype pair, and the output's type."""
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    pair = _PAIRS.get((dtype, out_dtype))
    if pair is None:
        raise ValueError(f"operands are float16 or bfloat16, the output their type or float32, not "
                         f"{dtype} and {out_dtype}")
    return pair, out_dtype


def _by_rows(function, rows, W, offsets, by_k, out, out_dtype, stream, name):
    """grouped_gemm and its gradient by X; by_k: the rows' length is K (else N)."""
    if W.dim() != 3 or not W.is_cuda:
        _refuse("W", W, "an experts x N x K CUDA tensor")
    _matrix(rows, name)
    (e, n, k), t = W.shape, rows.shape[0]
    width, cols = (k, n) if by_k else (n, k)
    dtype, device = W.dtype, W.get_device()
    pair, out_dtype = _pair(dtype, out, out_dtype)
    _dense(W, (e, n, k), dtype, device, "W")
    _dense(offsets, (e + 1,), _I32, device, "offsets")
    ld = _pitch(rows, t, width, dtype, device, name)
    if out is None:
        out, ldo = _empty((t, cols), out_dtype, W.device, stream), cols
    else:
        ldo = _pitch(out, t, cols, out_dtype, device, "out")
    _call(function, device, stream, (e, t, n, k, pair, offsets.data_ptr(), rows.data_ptr(), ld,
                                     W.data_ptr(), out.data_ptr(), ldo), (rows, W, offsets, out))
    return out


class _GroupedGemm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, offsets, out_dtype):
        ctx.save_for_backward(X, W, offsets)
        return _by_rows(_y, X, W, offsets, True, None, out_dtype, None, "X")

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        X, W, offsets = ctx.saved_tensors
        dY = dY.to(X.dtype)
        if not dY.is_contiguous() or dY.data_ptr() % 16:
            dY = dY.clone(memory_format=torch.contiguous_format)
        dX = grouped_gemm_dx(dY, W, offsets) if ctx.needs_input_grad[0] else None
        dW = grouped_gemm_dw(dY, X, offsets) if ctx.needs_input_grad[1] else None
        return dX, dW, None, None


def grouped_gemm(X, W, offsets, out=None, out_dtype=None, stream=None):
    """Products grouped by expert: ``Y[t] = X[t] @ W[e].T`` for the rows t of expert e.

    X: T x K; W: experts x N x K, contiguous; offsets: experts + 1 int32 on the
    GPU, rows ``offsets[e]`` to ``offsets[e + 1] - 1`` belonging to expert e
    (read there: the call does not wait for them).  Rows of no expert get
    zeros.  out_dtype: the operands' type (default) or float32.  Returns Y, T x N.

    Where X or W requires a gradient, backward runs grouped_gemm_dx and
    grouped_gemm_dw on Y's gradient in the operands' type, and gives gradients of
    that type; ``out`` is then refused.
    """
    if (X.requires_grad or W.requires_grad) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out cannot be given where X or W requires a gradient")
        if stream is None:
            return _GroupedGemm.apply(X, W, offsets, out_dtype)
        stream = _stream(stream, W.device)
        for t in (X, W, offsets):
            t.record_stream(stream)
        with torch.cuda.stream(stream):  # (backward runs there as well)
            return _GroupedGemm.apply(X, W, offsets, out_dtype)
    return _by_rows(_y, X, W, offsets, True, out, out_dtype, stream, "X")


def grouped_gemm_dx(dY, W, offsets, out=None, out_dtype=None, stream=None):
    """Gradient of grouped_gemm by X: ``dX[t] = dY[t] @ W[e]``; dY: T x N. Returns dX, T x K."""
    return _by_rows(_dx, dY, W, offsets, False, out, out_dtype, stream, "dY")


def grouped_gemm_dw(dY, X, offsets, out=None, out_dtype=None, stream=None):
    """Gradient of grouped_gemm by W: ``dW[e] = dY[rows of e].T @ X[rows of e]``.

    dY: T x N, X: T x K; returns dW, experts x N x K (zeros for an expert
    without rows), in the operands' type (default) or float32.
    """
    _matrix(X, "X")
    _matrix(dY, "dY")
    dtype, device, (t, k), n = X.dtype, X.get_device(), X.shape, dY.shape[1]
    pair, out_dtype = _pair(dtype, out, out_dtype)
    if offsets.dim() != 1 or not offsets.shape[0]:
        _refuse("offsets", offsets, "a 1-D tensor of experts + 1 values")
    e = offsets.shape[0] - 1
    _dense(offsets, (e + 1,), _I32, device, "offsets")
    ldx = _pitch(X, t, k, dtype, device, "X")
    ldy = _pitch(dY, t, n, dtype, device, "dY")
    if out is None:
        out = _empty((e, n, k), out_dtype, X.device, stream)
    else:
        _dense(out, (e, n, k), out_dtype, device, "out")
    _call(_dw, device, stream, (e, t, n, k, pair, offsets.data_ptr(), dY.data_ptr(), ldy,
                                X.data_ptr(), ldx, out.data_ptr()), (dY, X, offsets, out))
    return out
