"""The operators around the product, on torch tensors: the root-mean-square norm with the residual's addition, 8-bit
rows with scales, the product with bias, activation and residual in its epilogue, and the backward passes.

As in the rest of the binding, every arithmetic step runs in the library's HIP kernels; torch supplies device memory
and the stream.  Leading dimensions count as rows: an input of shape (..., d) is (rows, d), and its results have its
leading dimensions.  The inputs of the norm and of the quantisation may have evenly spaced rows any number of elements
apart (a slice of a wider tensor's last dimension, say); other layouts, and every strided input of the product, are made
contiguous first.  Calls are asynchronous on torch's current stream, or on ``stream`` (a handle or torch's object), on
which their results are then allocated; inputs that another stream still writes have to be waited for by the caller, as
with torch's own operators.  The calls stand outside torch's autograd: results never require gradients, whatever the
inputs do, and a training step calls the backward functions itself.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import BF16, F16, F32, FP8_E4M3, FP8_E5M2, INT8, GemmBtError, _in_order_of, load, workspace_for

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_CODES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16, torch.float8_e4m3fn: FP8_E4M3,
          torch.float8_e5m2: FP8_E5M2, torch.int8: INT8}
_FLOAT_CODES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_EIGHT = (FP8_E4M3, INT8)


class Epilogue(ctypes.Structure):
    """gemm_bt_epilogue_t."""

    _fields_ = [("row_scale", ctypes.c_void_p), ("col_scale", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("preact", ctypes.c_void_p), ("bias_dtype", ctypes.c_int),
                ("residual_dtype", ctypes.c_int), ("preact_dtype", ctypes.c_int), ("activation", ctypes.c_int)]


class Normed(NamedTuple):
    """What add_rms_norm returns; None for what was not asked for."""

    y: torch.Tensor                 # the normalised rows
    scale: Optional[torch.Tensor]   # fp32, one per row, of 8-bit rows
    h: Optional[torch.Tensor]       # x + residual
    rstd: Optional[torch.Tensor]    # fp32, one per row


class Quantized(NamedTuple):
    q: torch.Tensor
    scale: torch.Tensor


class LinearGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


def _on_gpu(first, *others):
    if not first.is_cuda:
        raise ValueError("expected tensors on a GPU, got %s" % first.device)
    device = first.device
    for t in others:
        if t is not None and t.device != device:
            raise ValueError("all tensors must be on the same GPU")
    return device


def _rows(t, what):
    """(tensor, row stride, rows, elements per row) of (..., d) seen as (rows, d), without a copy where the rows are evenly
    spaced."""
    shape = t.shape
    if not shape:
        raise ValueError("%s needs at least one dimension" % what)
    d = shape[-1]
    rows = t.numel() // d if d else shape[:-1].numel()
    if t.is_contiguous():
        return t, d, rows, d
    strides = t.stride()
    if strides[-1] == 1:
        # the leading dimensions of more than one entry, from the last one on: each has to step over all of the one after it
        ld = step = None
        for n, s in zip(shape[-2::-1], strides[-2::-1]):
            if n == 1:
                continue
            if step is None:
                ld = s
            elif s != step:
                ld = 0
                break
            step = s * n
        if ld is not None and ld >= d:
            return t, ld, rows, d
    return t.contiguous(), d, rows, d


def _activation(name):
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(ACTIVATIONS), name))
    return act


def _term(t, shape, what, dtype=None):
    """An epilogue's operand, contiguous."""
    if t.shape != shape or (dtype is not None and t.dtype != dtype):
        raise ValueError("%s must be a %stensor of shape %s, got %s %s"
                         % (what, "" if dtype is None else "%s " % dtype, tuple(shape), t.dtype, tuple(t.shape)))
    return _dense(t)


def _dense(t):
    return t if t.is_contiguous() else t.contiguous()


def _chunked(t):
    """t with dense rows from a 16-byte boundary on."""
    t = _dense(t)
    return t if t.data_ptr() % 16 == 0 else t.clone()


_HERE = contextlib.nullcontext()


def _on(device):
    """The context of a call on `device`: one that switches to it only if it is not the current device."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


# The handle of a device's current stream: torch.cuda.current_stream would build a Stream object around it (1.9 us).
_stream = torch._C._cuda_getCurrentRawStream


def _on_stream(stream, like, call):
    """call() with `stream` (a handle, or torch's object) as the current stream of like's device, so that every copy and
    every allocation of the call is in its order too."""
    with _in_order_of(like.device, stream):
        return call()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _float_code(dtype, what):
    code = _FLOAT_CODES.get(dtype)
    if code is None:
        raise TypeError("%s must be float32, float16 or bfloat16, got %s" % (what, dtype))
    return code


def _same(t, x, what):
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError("%s must be a %s tensor of shape %s" % (what, x.dtype, tuple(x.shape)))


def _output(out, like, shape, dtype, what="out"):
    """`out` if it fits, or a new contiguous tensor (empty_like is the cheapest of torch's ways to make one)."""
    if out is None:
        if like.shape == shape and like.is_contiguous():
            return torch.empty_like(like) if like.dtype == dtype else torch.empty_like(like, dtype=dtype)
        return like.new_empty(shape, dtype=dtype)
    if out.shape != shape or out.dtype != dtype or not out.is_contiguous() or out.device != like.device:
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (what, dtype, tuple(shape), like.device))
    return out


def _workspace_query(name):
    """A workspace size of the library, remembered per sizes and device (it depends on nothing else)."""
    @functools.lru_cache(maxsize=1024)
    def query(*args):
        need = ctypes.c_size_t()
        st = getattr(load(), name)(*args[:-1], ctypes.byref(need))  # the last argument is the device, the current one
        if st:
            raise GemmBtError(st, name)
        return need.value

    return query


_epi_bytes = _workspace_query("gemm_bt_epi_workspace_size")
_norm_back_bytes = _workspace_query("gemm_bt_rms_norm_backward_workspace")
_linear_back_bytes = _workspace_query("gemm_bt_linear_backward_workspace")


# ---------------------------------------------------------------- norm and quantisation

def add_rms_norm(x, weight, residual=None, eps=1e-6, out_dtype=None, save_rstd=False, out=None, h_out=None, stream=None):
    """h = x + residual; y = h / sqrt(mean(h²) + eps) * weight, over the last dimension.

    x: float32, float16 or bfloat16; residual: as x, or None; weight: (d,) of x's type or float32.  ``out_dtype``: x's
    type (the default), another float type, or float8_e4m3fn or int8 for 8-bit rows with one float32 scale each (y is
    then q with y ≈ q * scale[..., None]).  Returns Normed(y, scale, h, rstd): scale for 8-bit rows, h where a residual
    is given (``h_out``, a contiguous tensor of x's type, receives it; it may be x or residual itself), rstd with
    ``save_rstd``.  h is used unrounded and returned rounded to x's type.
    """
    if stream is not None:
        return _on_stream(stream, x, lambda: add_rms_norm(x, weight, residual, eps, out_dtype, save_rstd, out, h_out))
    device = _on_gpu(x, weight, residual)
    dtype, shape = x.dtype, x.shape
    x_code = _float_code(dtype, "x")
    if weight.shape != shape[-1:]:
        raise ValueError("weight must have the shape of x's last dimension, got %s and %s" % (tuple(weight.shape), tuple(shape)))
    if weight.dtype != dtype and weight.dtype != torch.float32:
        raise TypeError("weight must be %s or float32, got %s" % (dtype, weight.dtype))
    y_dtype = dtype if out_dtype is None else out_dtype
    y_code = _CODES.get(y_dtype)
    if y_code is None or y_code == FP8_E5M2:
        raise TypeError("out_dtype must be a float type, float8_e4m3fn or int8, got %s" % y_dtype)
    xr, ldx, rows, d = _rows(x, "x")
    y = _output(out, xr, shape, y_dtype)
    scale = x.new_empty(shape[:-1], dtype=torch.float32) if y_code in _EIGHT else None
    rstd = x.new_empty(shape[:-1], dtype=torch.float32) if save_rstd else None
    rr, ldr, h = None, 0, None
    if residual is not None:
        _same(residual, x, "residual")
        rr, ldr, _, _ = _rows(residual, "residual")
        h = _output(h_out, xr, shape, dtype, "h_out")
    elif h_out is not None:
        raise ValueError("h_out needs a residual: without one h is x itself")
    weight = _dense(weight)
    with _on(device):
        st = load().gemm_bt_rms_norm(xr.data_ptr(), ldx, _ptr(rr), ldr, weight.data_ptr(), y.data_ptr(), _ptr(h), _ptr(scale),
                                     _ptr(rstd), rows, d, eps, x_code, _CODES[weight.dtype], y_code, _stream(device.index))
    if st:
        raise GemmBtError(st, "gemm_bt_rms_norm")
    return Normed(y, scale, h, rstd)


def quantize_rows(x, dtype=torch.float8_e4m3fn, stream=None):
    """The rows of x in 8 bits (float8_e4m3fn or int8) and one float32 scale each: Quantized(q, scale), x ≈ q * scale."""
    if stream is not None:
        return _on_stream(stream, x, lambda: quantize_rows(x, dtype))
    device = _on_gpu(x)
    x_code = _float_code(x.dtype, "x")
    q_code = _CODES.get(dtype)
    if q_code not in _EIGHT:
        raise TypeError("dtype must be float8_e4m3fn or int8, got %s" % dtype)
    xr, ldx, rows, d = _rows(x, "x")
    q = x.new_empty(x.shape, dtype=dtype)
    scale = x.new_empty(x.shape[:-1], dtype=torch.float32)
    with _on(device):
        st = load().gemm_bt_quantize_rows(xr.data_ptr(), ldx, q.data_ptr(), scale.data_ptr(), rows, d, x_code, q_code,
                                          _stream(device.index))
    if st:
        raise GemmBtError(st, "gemm_bt_quantize_rows")
    return Quantized(q, scale)


def add_rms_norm_backward(dy, h, weight, rstd, dh=None, stream=None):
    """(dx, dweight) of add_rms_norm: h and rstd as it returned them (h is x where there was no residual), dy the
    gradient of y, dh the gradient that reaches h from elsewhere.  dx is the gradient of x and of residual alike."""
    if stream is not None:
        return _on_stream(stream, dy, lambda: add_rms_norm_backward(dy, h, weight, rstd, dh))
    device = _on_gpu(dy, h, weight, rstd, dh)
    dtype, shape = dy.dtype, dy.shape
    code = _float_code(dtype, "dy")
    _same(h, dy, "h")
    if weight.shape != shape[-1:]:
        raise ValueError("weight must have the shape of dy's last dimension, got %s and %s" % (tuple(weight.shape), tuple(shape)))
    if weight.dtype != dtype and weight.dtype != torch.float32:
        raise TypeError("weight must be %s or float32, got %s" % (dtype, weight.dtype))
    if rstd.dtype != torch.float32 or rstd.shape != shape[:-1]:
        raise ValueError("rstd must be a float32 tensor of shape %s" % (tuple(shape[:-1]),))
    dyr, ld_dy, rows, d = _rows(dy, "dy")
    hr, ldh, _, _ = _rows(h, "h")
    dhr, ld_dh = None, 0
    if dh is not None:
        _same(dh, dy, "dh")
        dhr, ld_dh, _, _ = _rows(dh, "dh")
    weight, rstd = _dense(weight), _dense(rstd)
    dx = _output(None, dyr, shape, dtype)
    dw = torch.empty_like(weight)
    with _on(device):
        s = _stream(device.index)
        need = _norm_back_bytes(rows, d, device.index)
        ws = dyr.new_empty(need, dtype=torch.uint8) if need else None
        st = load().gemm_bt_rms_norm_backward(dyr.data_ptr(), ld_dy, hr.data_ptr(), ldh, weight.data_ptr(), rstd.data_ptr(),
                                              _ptr(dhr), ld_dh, dx.data_ptr(), dw.data_ptr(), rows, d, code, _CODES[weight.dtype],
                                              _ptr(ws), need, s)
    if st:
        raise GemmBtError(st, "gemm_bt_rms_norm_backward")
    return dx, dw


# ---------------------------------------------------------------- the product with its epilogue

def linear(x, weight, bias=None, activation="none", residual=None, x_scale=None, weight_scale=None, out_dtype=None,
           save_preact=False, out=None, stream=None):
    """act(x @ weight.T * x_scale[..., None] * weight_scale + bias) + residual in one kernel.

    x (..., K) and weight (N, K) of one input type: bfloat16, float16, float8_e4m3fn, float8_e5m2 or int8 (8-bit inputs
    need K % 16 == 0; int8 also K <= 131071).  bias (N,) and residual (..., N): float32, float16 or bfloat16; x_scale
    (...) and weight_scale (N,): float32.  ``activation``: one of ACTIVATIONS.  ``out_dtype``: float32, float16 or
    bfloat16; the default is x's type (bfloat16 for 8-bit inputs).  Everything between the product and the result is
    held in fp32.  With ``save_preact`` returns (y, z), z the argument of the activation (x's type, bfloat16 for 8-bit
    inputs) for linear_backward.  ``out`` may be residual itself.
    """
    if stream is not None:
        return _on_stream(stream, x, lambda: linear(x, weight, bias, activation, residual, x_scale, weight_scale, out_dtype, save_preact, out))
    device = _on_gpu(x, weight, bias, residual, x_scale, weight_scale)
    dtype = x.dtype
    in_code = _CODES.get(dtype)
    if in_code is None or in_code == F32:
        raise TypeError("unsupported input dtype %s" % dtype)
    if weight.dtype != dtype:
        raise TypeError("x and weight must share one dtype")
    x_shape, w_shape = x.shape, weight.shape
    if len(w_shape) != 2 or x_shape[-1:] != w_shape[1:]:
        raise ValueError("expected x (..., K) and weight (N, K), got %s and %s" % (tuple(x_shape), tuple(w_shape)))
    e = Epilogue()
    act = e.activation = _activation(activation)
    N, K = w_shape
    lead = x_shape[:-1]
    M = lead.numel()
    shape = lead + w_shape[:1]
    wide = dtype if in_code == BF16 or in_code == F16 else torch.bfloat16
    y_dtype = wide if out_dtype is None else out_dtype
    out_code = _float_code(y_dtype, "out_dtype")
    if in_code == BF16 or in_code == F16:
        x, weight = _dense(x), _dense(weight)
    else:  # 8-bit products read whole 16-byte chunks
        x, weight = _chunked(x), _chunked(weight)
    if bias is not None:
        bias = _term(bias, w_shape[:1], "bias")
        e.bias, e.bias_dtype = bias.data_ptr(), _float_code(bias.dtype, "bias")
    if residual is not None:
        residual = _term(residual, shape, "residual")
        e.residual, e.residual_dtype = residual.data_ptr(), _float_code(residual.dtype, "residual")
    if x_scale is not None:
        x_scale = _term(x_scale, lead, "x_scale", torch.float32)
        e.row_scale = x_scale.data_ptr()
    if weight_scale is not None:
        weight_scale = _term(weight_scale, w_shape[:1], "weight_scale", torch.float32)
        e.col_scale = weight_scale.data_ptr()
    y = _output(out, x, shape, y_dtype)
    z = None
    if save_preact:
        z = _output(None, y, shape, wide)
        e.preact, e.preact_dtype = z.data_ptr(), _CODES[wide]
    with _on(device):
        s = _stream(device.index)
        need = _epi_bytes(M, N, K, in_code, out_code, device.index)
        ws, ws_bytes = None, 0  # 16-bit products of few rows that need none: without one they stream their weight
        if need:
            t = workspace_for(device, s, need)
            ws, ws_bytes = t.data_ptr(), t.numel()
        st = load().gemm_bt_epi(x.data_ptr(), weight.data_ptr(), y.data_ptr(), M, N, K, in_code, out_code, ctypes.byref(e), ws,
                                ws_bytes, s)
    if st:
        raise GemmBtError(st, "gemm_bt_epi")
    return (y, z) if save_preact else y


def linear_backward(dy, x, weight, preact=None, activation="none", bias_grad=True, need_dx=True, need_dweight=True,
                    stream=None):
    """The gradients of linear's x, weight and bias for 16-bit x and weight: LinearGrads(dx, dweight, dbias).

    dy (..., N): the gradient of the result, of x's type; preact: what linear returned with save_preact (not needed
    for the activation "none").  All three are of x's type, a float32 bias's too.  The gradient of the residual is dy
    itself, and relu's slope at 0 is 0.
    """
    if stream is not None:
        return _on_stream(stream, dy, lambda: linear_backward(dy, x, weight, preact, activation, bias_grad, need_dx, need_dweight))
    device = _on_gpu(dy, x, weight, preact)
    dtype = x.dtype
    if dtype not in (torch.bfloat16, torch.float16) or weight.dtype != dtype or dy.dtype != dtype:
        raise TypeError("dy, x and weight must share float16 or bfloat16")
    act = _activation(activation)
    x_shape, w_shape = x.shape, weight.shape
    if len(w_shape) != 2 or x_shape[-1:] != w_shape[1:] or dy.shape != x_shape[:-1] + w_shape[:1]:
        raise ValueError("expected dy (..., N), x (..., K) and weight (N, K), got %s, %s and %s"
                         % (tuple(dy.shape), tuple(x_shape), tuple(w_shape)))
    code = z_code = _CODES[dtype]
    if act:
        if preact is None or preact.shape != dy.shape:
            raise ValueError("preact must be the pre-activation that linear returned, of shape %s" % (tuple(dy.shape),))
        z_code = _float_code(preact.dtype, "preact")
        preact = _dense(preact)
    N, K = w_shape
    M = x_shape[:-1].numel()
    dy, x, weight = _chunked(dy), _chunked(x), _chunked(weight)
    dx = torch.empty_like(x) if need_dx else None
    dw = torch.empty_like(weight) if need_dweight else None
    db = weight.new_empty(N) if bias_grad else None
    with _on(device):
        s = _stream(device.index)
        need = _linear_back_bytes(M, N, K, act, device.index)
        ws = dy.new_empty(need, dtype=torch.uint8) if need else None
        st = load().gemm_bt_linear_backward(dy.data_ptr(), x.data_ptr(), weight.data_ptr(), preact.data_ptr() if act else None,
                                            _ptr(dx), _ptr(dw), _ptr(db), M, N, K, act, code, z_code, _ptr(ws), need, s)
    if st:
        raise GemmBtError(st, "gemm_bt_linear_backward")
    return LinearGrads(dx, dw, db)
