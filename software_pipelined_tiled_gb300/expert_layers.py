"""Python binding of the operators around an expert layer.

Routing, rows sorted by expert and added up again, and the end of a block (norm,
gate, scaled residual, norm).  What ``layers`` says of streams, tensors and
checks holds here too.

``route_experts``, ``dispatch_rows``, ``combine_rows`` and ``gate_add_rms_norm``
take part in PyTorch's automatic differentiation: where an input requires a
gradient (and none of the outputs is given), backward runs the functions that
compute the gradients, which can also be called by themselves (tensors that carry
tangents of the forward mode are refused).  All of them can
be captured in a CUDA graph; a backward pass only while no other graph of the
same leaves is alive (PyTorch's rule: a leaf's node keeps to the stream that it was
made on, which may not join the capture).
"""
from __future__ import annotations

import ctypes

import torch

import software_pipelined_tiled_gb300 as _pkg

from .layers import (_16BIT, _F32, _I32, _call, _dense, _empty, _forward, _matrix, _pitch, _refuse,
                     _refuse_tangents, _stream)

_lib = _pkg.load()
_route, _route_grad = _lib.sptg_route_experts, _lib.sptg_route_experts_dlogits
_dispatch, _combine, _combine_grad = (_lib.sptg_dispatch_rows, _lib.sptg_combine_rows,
                                      _lib.sptg_combine_rows_grad_ex)
_gate_norm, _gate_norm_grad = _lib.sptg_gate_add_rms_norm, _lib.sptg_gate_add_rms_norm_grad
_workspace = _lib.sptg_gate_add_rms_norm_grad_workspace

# sptg_type values of include/sptgemm.h
_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 4}
_SCORES = {"softmax": 0, "sigmoid": 1}
_GATE_NONE, _GATE_COLS, _GATE_ROWS, _GATE_FULL = range(4)
_grad_enabled, _new_like = torch.is_grad_enabled, torch.empty_like


def _differentiated(function, stream, device, args, outputs):
    """A torch.autograd.Function's apply on the call's stream (backward runs there as well)."""
    for o in outputs:
        if o is not None:
            raise ValueError("outputs cannot be given where an input requires a gradient")
    if stream is None:
        return function.apply(*args)
    stream = _stream(stream, device)
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return function.apply(*args)


def _as_rows(t, dtype):
    """A gradient as autograd gives it (any type and strides) as rows of a type."""
    t = t.to(dtype)
    if t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) and t.stride(0) >= t.shape[1]:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _like(t, stream):
    """A new tensor of another's shape and type, dense, that belongs to the call's stream."""
    if stream is None and t.is_contiguous():
        return _new_like(t)
    return _empty(t.shape, t.dtype, t.device, stream)


def _row_type(t, name: str) -> int:
    if t.dim() != 2 or not t.is_cuda or t.dtype not in _16BIT:
        _refuse(name, t, "a 2-D float16 or bfloat16 CUDA tensor")
    return _TYPES[t.dtype]


# ------------------------------------------------------------------- routing
def _run_route(logits, top, bias, scores, groups, top_groups, group_best, renormalize, scale, weights,
               experts, stream):
    if logits.dim() != 2 or not logits.is_cuda:
        _refuse("logits", logits, "a 2-D CUDA tensor")
    rows, e = logits.shape
    dtype, device, on = logits.dtype, logits.get_device(), logits.device
    code, sigmoid = _TYPES.get(dtype), _SCORES.get(scores)
    if code is None:
        raise ValueError(f"logits must be float16, bfloat16 or float32, not {dtype}")
    if sigmoid is None:
        raise ValueError(f"scores must be 'softmax' or 'sigmoid', not {scores!r}")
    ld = e if logits.is_contiguous() else _pitch(logits, rows, e, dtype, device, "logits")
    if bias is not None:
        _dense(bias, (e,), _F32, device, "bias")
    if weights is None:
        weights = _empty((rows, top), _F32, on, stream)
    else:
        _dense(weights, (rows, top), _F32, device, "weights")
    if experts is None:
        experts = _empty((rows, top), _I32, on, stream)
    else:
        _dense(experts, (rows, top), _I32, device, "experts")
    _call(_route, device, stream, (
        rows, e, top, code, logits.data_ptr(), ld, None if bias is None else bias.data_ptr(), sigmoid,
        groups, top_groups, group_best, 1 if renormalize else 0, scale, weights.data_ptr(),
        experts.data_ptr()), (logits, bias, weights, experts))
    return weights, experts


class _RouteExperts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top, bias, scores, groups, top_groups, group_best, renormalize, scale):
        weights, experts = _run_route(logits, top, bias, scores, groups, top_groups, group_best,
                                      renormalize, scale, None, None, None)
        ctx.mark_non_differentiable(experts)
        ctx.save_for_backward(logits, experts)
        ctx.how = (scores, renormalize, scale)
        return weights, experts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dweights, _):
        logits, experts = ctx.saved_tensors
        scores, renormalize, scale = ctx.how
        dlogits = route_experts_dlogits(dweights.to(_F32).contiguous(), logits, experts, scores=scores,
                                        renormalize=renormalize, scale=scale)
        return (dlogits,) + (None,) * 8


def route_experts(logits, top: int, bias=None, scores: str = "softmax", groups: int = 1, top_groups: int = 1,
                  group_best: int = 2, renormalize: bool = True, scale: float = 1.0, weights=None,
                  experts=None, stream=None):
    """The experts of each row and their weights: returns (weights, experts), each T x top.

    ``scores``: "softmax" or "sigmoid" of the logits (T x E, float16, bfloat16
    or float32).  The ``top`` experts with the largest score + bias (E float32,
    or None) are chosen, largest first, of equal ones the lowest index.  With
    ``groups`` > 1 (equal groups of neighbouring experts) only those of the
    ``top_groups`` groups count whose ``group_best`` (1 or 2) best experts have
    the largest sum.  Keys are compared as exact arithmetic would compare them
    (without a bias for scores of any size, with one to 2^-42 of keys and biases).
    weights (float32): the chosen scores, without the bias, times ``scale``;
    with ``renormalize`` divided by their sum.  experts: int32.

    Experts whose logit or bias is -infinity are never chosen: where fewer than
    ``top`` are left, experts ends in -1 and weights in 0.  A row with a NaN (with a
    softmax: or +infinity) has weights NaN and experts 0 ... top - 1.

    weights is differentiable by the logits (route_experts_dlogits).
    """
    if _forward._current_level >= 0:
        _refuse_tangents(logits)
    if logits.requires_grad and _grad_enabled():
        return _differentiated(_RouteExperts, stream, logits.device,
                               (logits, top, bias, scores, groups, top_groups, group_best, renormalize,
                                scale), (weights, experts))
    return _run_route(logits, top, bias, scores, groups, top_groups, group_best, renormalize, scale,
                      weights, experts, stream)


def route_experts_dlogits(dweights, logits, experts, scores: str = "softmax", renormalize: bool = True,
                          scale: float = 1.0, out=None, stream=None):
    """Gradient of route_experts' weights by the logits: T x E, of the logits' type.

    dweights: T x top float32; experts, scores, renormalize, scale: as
    route_experts returned and took them.
    """
    _matrix(logits, "logits")
    _matrix(experts, "experts")
    rows, e = logits.shape
    top = experts.shape[1]
    dtype, device = logits.dtype, logits.get_device()
    code, sigmoid = _TYPES.get(dtype), _SCORES.get(scores)
    if code is None:
        raise ValueError(f"logits must be float16, bfloat16 or float32, not {dtype}")
    if sigmoid is None:
        raise ValueError(f"scores must be 'softmax' or 'sigmoid', not {scores!r}")
    ld = _pitch(logits, rows, e, dtype, device, "logits")
    _dense(experts, (rows, top), _I32, device, "experts")
    _dense(dweights, (rows, top), _F32, device, "dweights")
    if out is None:
        out, ldo = _like(logits, stream), e
    else:
        ldo = _pitch(out, rows, e, dtype, device, "out")
    _call(_route_grad, device, stream, (
        rows, e, top, code, logits.data_ptr(), ld, experts.data_ptr(), dweights.data_ptr(), sigmoid,
        1 if renormalize else 0, scale, out.data_ptr(), ldo), (dweights, logits, experts, out))
    return out


# ------------------------------------------------- rows to experts and back
def _run_dispatch(x, experts, num_experts, out, places, offsets, stream):
    code = _row_type(x, "x")
    if experts.dim() != 2:
        _refuse("experts", experts, "a 2-D tensor")
    (rows, cols), top = x.shape, experts.shape[1]
    dtype, device, on = x.dtype, x.get_device(), x.device
    ldx = cols if x.is_contiguous() else _pitch(x, rows, cols, dtype, device, "x")
    _dense(experts, (rows, top), _I32, device, "experts")
    if out is None:
        out, ldo = _empty((rows * top, cols), dtype, on, stream), cols
    else:
        ldo = _pitch(out, rows * top, cols, dtype, device, "out")
    if places is None:
        places = _empty((rows, top), _I32, on, stream)
    else:
        _dense(places, (rows, top), _I32, device, "places")
    if offsets is None:
        offsets = _empty((num_experts + 1,), _I32, on, stream)
    else:
        _dense(offsets, (num_experts + 1,), _I32, device, "offsets")
    _call(_dispatch, device, stream, (
        rows, cols, top, num_experts, code, x.data_ptr(), ldx, experts.data_ptr(), out.data_ptr(), ldo,
        places.data_ptr(), offsets.data_ptr()), (x, experts, out, places, offsets))
    return out, places, offsets


class _DispatchRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, experts, num_experts):
        out, places, offsets = _run_dispatch(x, experts, num_experts, None, None, None, None)
        ctx.mark_non_differentiable(places, offsets)
        ctx.save_for_backward(places)
        ctx.dtype = x.dtype
        return out, places, offsets

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, _places, _offsets):
        return dispatch_rows_dx(_as_rows(dout, ctx.dtype), ctx.saved_tensors[0]), None, None


def dispatch_rows(x, experts, num_experts: int, out=None, places=None, offsets=None, stream=None):
    """Rows sorted by expert: returns (rows, places, offsets), for grouped_gemm and combine_rows.

    x: T x C, float16 or bfloat16; experts: T x top int32, as route_experts
    returns them.  ``places[t, j]`` (int32) is the row that entry (t, j) went to:
    ``rows[places[t, j]] = x[t]``.  Entries are sorted by expert, those of one
    expert stay in their order, and those outside 0 ... num_experts - 1 come
    last.  ``offsets[e]`` (num_experts + 1 int32) is expert e's first row.

    rows is differentiable by x (dispatch_rows_dx).
    """
    if _forward._current_level >= 0:
        _refuse_tangents(x)
    if x.requires_grad and _grad_enabled():
        return _differentiated(_DispatchRows, stream, x.device, (x, experts, num_experts),
                               (out, places, offsets))
    return _run_dispatch(x, experts, num_experts, out, places, offsets, stream)


def _run_combine(y, places, weights, base, out, stream):
    code = _row_type(y, "y")
    if places.dim() != 2:
        _refuse("places", places, "a 2-D tensor")
    (y_rows, cols), (rows, top) = y.shape, places.shape
    dtype, device = y.dtype, y.get_device()
    ldy = cols if y.is_contiguous() else _pitch(y, y_rows, cols, dtype, device, "y")
    _dense(places, (rows, top), _I32, device, "places")
    if weights is not None:
        _dense(weights, (rows, top), _F32, device, "weights")
    ldb = cols if base is None else _pitch(base, rows, cols, dtype, device, "base")
    if out is None:
        out, ldo = _empty((rows, cols), dtype, y.device, stream), cols
    else:
        ldo = _pitch(out, rows, cols, dtype, device, "out")
    _call(_combine, device, stream, (
        rows, cols, top, y_rows, code, y.data_ptr(), ldy, places.data_ptr(),
        None if weights is None else weights.data_ptr(), None if base is None else base.data_ptr(), ldb,
        out.data_ptr(), ldo), (y, places, weights, base, out))
    return out


def dispatch_rows_dx(drows, places, out=None, stream=None):
    """Gradient of dispatch_rows by x: ``dx[t] = sum over j of drows[places[t, j]]``. Returns dx, T x C."""
    return _run_combine(drows, places, None, None, out, stream)


class _CombineRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, places, weights, base):
        ctx.save_for_backward(y, places, weights)
        return _run_combine(y, places, weights, base, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        y, places, weights = ctx.saved_tensors
        dy = dweights = None
        needs = ctx.needs_input_grad
        dout = _as_rows(dout, y.dtype)
        if needs[0] or needs[2]:
            dy, dweights = combine_rows_grad(dout, y, places, weights, need_weights=needs[2])
        return dy if needs[0] else None, None, dweights, dout if needs[3] else None


def combine_rows(y, places, weights=None, base=None, out=None, stream=None):
    """Rows added up: ``out[t] = base[t] + sum over j of weights[t, j] * y[places[t, j]]``.

    y: the experts' outputs in dispatch_rows' order, float16 or bfloat16;
    places: T x top int32, as dispatch_rows returns them (one outside of y's
    rows adds nothing); weights: T x top float32, or None for 1; base: T x C of
    y's type (the output of experts that every row goes through), or None.
    Sums are 32 bits, rounded once.  Returns out, T x C (it may be base).

    Differentiable by y, weights and base (combine_rows_grad); places then has to
    name no row of y twice.  Rows that none names have gradient 0.
    """
    if _forward._current_level >= 0:
        _refuse_tangents(y, weights, base)
    if ((y.requires_grad or (weights is not None and weights.requires_grad)
         or (base is not None and base.requires_grad)) and _grad_enabled()):
        return _differentiated(_CombineRows, stream, y.device, (y, places, weights, base), (out,))
    return _run_combine(y, places, weights, base, out, stream)


def combine_rows_grad(dout, y, places, weights=None, dy=None, dweights=None, need_weights: bool = True,
                      stream=None):
    """Gradients of combine_rows by y and weights: returns (dy, dweights).

    ``dy[places[t, j]] = weights[t, j] * dout[t]``, of y's type, and
    ``dweights[t, j] = <y[places[t, j]], dout[t]>``, float32 (None where weights is
    None or need_weights is false; y is then not read).  places has to name no row of
    y twice; rows that none names are 0 (in a given dy: left as they were).
    """
    code = _row_type(y, "y")
    if places.dim() != 2:
        _refuse("places", places, "a 2-D tensor")
    (y_rows, cols), (rows, top) = y.shape, places.shape
    dtype, device, on = y.dtype, y.get_device(), y.device
    ldy = _pitch(y, y_rows, cols, dtype, device, "y")
    ldd = _pitch(dout, rows, cols, dtype, device, "dout")
    _dense(places, (rows, top), _I32, device, "places")
    if weights is not None:
        _dense(weights, (rows, top), _F32, device, "weights")
    zeros = dy is None
    if zeros:
        dy, lddy = _like(y, stream), cols
    else:
        lddy = _pitch(dy, y_rows, cols, dtype, device, "dy")
    if weights is None or not need_weights:
        if dweights is not None:
            raise ValueError("dweights belong to weights")
    elif dweights is None:
        dweights = _empty((rows, top), _F32, on, stream)
    else:
        _dense(dweights, (rows, top), _F32, device, "dweights")
    _call(_combine_grad, device, stream, (
        rows, cols, top, y_rows, code, dout.data_ptr(), ldd, y.data_ptr(), ldy, places.data_ptr(),
        None if weights is None else weights.data_ptr(), dy.data_ptr(), lddy,
        None if dweights is None else dweights.data_ptr(), 1 if zeros else 0),
        (dout, y, places, weights, dy, dweights))
    return dy, dweights


# ---------------------------------------------------------- the end of a block
def _gate_of(gate, rows, cols, dtype, device):
    """A gate's kind and pitch."""
    if gate is None:
        return _GATE_NONE, 0
    shape = tuple(gate.shape)
    if shape == (cols,) or (shape == (1, cols) and rows != 1):
        _dense(gate, gate.shape, dtype, device, "gate")
        return _GATE_COLS, 0
    if shape == (rows, 1) and cols != 1 and gate.dtype is dtype and gate.get_device() == device:
        if rows == 1 or gate.stride(0) > 0:
            return _GATE_ROWS, max(1, gate.stride(0))
    if shape != (rows, cols):
        _refuse("gate", gate, f"a {dtype} tensor of {cols} values, {rows} x 1 or {rows} x {cols}, on CUDA "
                              f"device {device}")
    return _GATE_FULL, _pitch(gate, rows, cols, dtype, device, "gate")


def _tail(config):
    """The argument that follows the stream."""
    return (None if config is None else ctypes.byref(config),)


def _run_gate_norm(y, residual, weight, block_weight, gate, alpha, eps, h, v, stream, config=None):
    code = _row_type(y, "y")
    rows, cols = y.shape
    dtype, device = y.dtype, y.get_device()
    ldy = cols if y.is_contiguous() else _pitch(y, rows, cols, dtype, device, "y")
    ldr = _pitch(residual, rows, cols, dtype, device, "residual")
    _dense(weight, (cols,), dtype, device, "weight")
    if block_weight is not None:
        _dense(block_weight, (cols,), dtype, device, "block_weight")
    kind, ldg = _gate_of(gate, rows, cols, dtype, device)
    if h is None:
        h, ldh = _like(y, stream), cols
    else:
        ldh = _pitch(h, rows, cols, dtype, device, "h")
    if v is None:
        v, ldv = _like(y, stream), cols
    else:
        ldv = _pitch(v, rows, cols, dtype, device, "v")
    _call(_gate_norm, device, stream, (
        rows, cols, code, y.data_ptr(), ldy, residual.data_ptr(), ldr,
        None if block_weight is None else block_weight.data_ptr(), None if gate is None else gate.data_ptr(),
        kind, ldg, alpha, weight.data_ptr(), eps, h.data_ptr(), ldh, v.data_ptr(), ldv),
        (y, residual, weight, block_weight, gate, h, v), _tail(config))
    return h, v


class _GateAddRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, weight, block_weight, gate, alpha, eps, config):
        ctx.save_for_backward(y, residual, weight, block_weight, gate)
        ctx.how = (alpha, eps)
        # (backward has what forward was given, whatever becomes of the caller's object)
        ctx.config = None if config is None else type(config).from_buffer_copy(config)
        ctx.set_materialize_grads(False)
        return _run_gate_norm(y, residual, weight, block_weight, gate, alpha, eps, None, None, None, config)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dv):
        if dh is None and dv is None:
            return (None,) * 8
        y, residual, weight, block_weight, gate = ctx.saved_tensors
        dh, dv = (None if t is None else _as_rows(t, y.dtype) for t in (dh, dv))
        grads = gate_add_rms_norm_grad(dh, dv, y, residual, weight, block_weight, gate, *ctx.how,
                                       config=ctx.config)
        return tuple(g if n else None for g, n in zip(grads, ctx.needs_input_grad)) + (None,) * 3


def gate_add_rms_norm(y, residual, weight, block_weight=None, gate=None, alpha: float = 1.0,
                      eps: float = 1e-6, h=None, v=None, stream=None, config=None):
    """The end of a block: norm of its output, gate, scaled residual, norm before the next: returns (h, v).

    ``u = y * block_weight / sqrt(mean(y^2) + eps)`` (u = y without block_weight),
    ``h = alpha * residual + gate * u`` (the new residual stream; may be y or
    residual itself), ``v = h * weight / sqrt(mean(h^2) + eps)``, in 32 bits, h
    and v rounded once each.  y, residual: T x C, float16 or bfloat16; weights: C
    values; gate: None, C values (or 1 x C, where T is not 1), T x 1 or T x C, all of y's
    type.  A row's last bits may depend on T, which chooses among kernels.
    config: a Config, for its timeout_ms and inject_stall.

    Differentiable by all tensors (gate_add_rms_norm_grad, with the same config).
    """
    if _forward._current_level >= 0:
        _refuse_tangents(y, residual, weight, block_weight, gate)
    if ((y.requires_grad or residual.requires_grad or weight.requires_grad
         or (block_weight is not None and block_weight.requires_grad)
         or (gate is not None and gate.requires_grad)) and _grad_enabled()):
        return _differentiated(_GateAddRmsNorm, stream, y.device,
                               (y, residual, weight, block_weight, gate, alpha, eps, config), (h, v))
    return _run_gate_norm(y, residual, weight, block_weight, gate, alpha, eps, h, v, stream, config)


def gate_add_rms_norm_grad(dh, dv, y, residual, weight, block_weight=None, gate=None, alpha: float = 1.0,
                           eps: float = 1e-6, out_dtype=None, stream=None, config=None):
    """Gradients of gate_add_rms_norm: returns those of (y, residual, weight, block_weight, gate).

    dh, dv: gradients of h and v (T x C of y's type; either may be None).
    ``out_dtype``: of the gradients that are sums over rows or columns (weight,
    block_weight, a gate that is broadcast): y's type (default) or float32.
    Those of inputs that are None are None.  With one row, a gate of 1 x C is T x C: its
    gradient is no sum and of y's type (that of a gate of C values is of out_dtype always).
    """
    code = _row_type(y, "y")
    rows, cols = y.shape
    dtype, device, on = y.dtype, y.get_device(), y.device
    if out_dtype is None:
        out_dtype = dtype
    if out_dtype is not dtype and out_dtype is not _F32:
        raise ValueError(f"out_dtype must be {dtype} or float32, not {out_dtype}")
    ldy = _pitch(y, rows, cols, dtype, device, "y")
    ldr = _pitch(residual, rows, cols, dtype, device, "residual")
    _dense(weight, (cols,), dtype, device, "weight")
    if block_weight is not None:
        _dense(block_weight, (cols,), dtype, device, "block_weight")
    kind, ldg = _gate_of(gate, rows, cols, dtype, device)
    lddh = cols if dh is None else _pitch(dh, rows, cols, dtype, device, "dh")
    lddv = cols if dv is None else _pitch(dv, rows, cols, dtype, device, "dv")
    dy, dresidual = _like(y, stream), _like(y, stream)
    dweight = _empty((cols,), out_dtype, on, stream)
    dblock = None if block_weight is None else _empty((cols,), out_dtype, on, stream)
    dgate = None
    if gate is not None:
        dgate = _empty(gate.shape, dtype if kind == _GATE_FULL else out_dtype, on, stream)
    space = _workspace(rows, cols)
    workspace = _empty((space,), torch.uint8, on, stream)
    _call(_gate_norm_grad, device, stream, (
        rows, cols, code, None if dh is None else dh.data_ptr(), lddh, None if dv is None else dv.data_ptr(),
        lddv, y.data_ptr(), ldy, residual.data_ptr(), ldr,
        None if block_weight is None else block_weight.data_ptr(), None if gate is None else gate.data_ptr(),
        kind, ldg, alpha, weight.data_ptr(), eps, dy.data_ptr(), cols, dresidual.data_ptr(), cols,
        None if dgate is None else dgate.data_ptr(), cols, dweight.data_ptr(),
        None if dblock is None else dblock.data_ptr(), _TYPES[out_dtype], workspace.data_ptr(), space),
        (dh, dv, y, residual, weight, block_weight, gate, dy, dresidual, dweight, dblock, dgate, workspace),
        _tail(config))
    return dy, dresidual, dweight, dblock, dgate
