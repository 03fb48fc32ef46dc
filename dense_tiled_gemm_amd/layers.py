"""The operators around the product, on torch tensors: the root-mean-square norm with the residual's addition, 8-bit
rows with scales, the product with bias, activation and residual in its epilogue, and the backward passes.

As in the rest of the binding, every arithmetic step runs in the library's HIP kernels; torch supplies device memory
and the stream.  Leading dimensions count as rows: an input of shape (..., d) is (rows, d), and its results have its
leading dimensions.  Rows may lie any number of elements apart; other layouts are made contiguous first.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import BF16, F16, F32, FP8_E4M3, FP8_E5M2, INT8, OK, GemmBtError, load, workspace_for

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_CODES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16, torch.float8_e4m3fn: FP8_E4M3,
          torch.float8_e5m2: FP8_E5M2, torch.int8: INT8}
_FLOATS = (torch.float32, torch.float16, torch.bfloat16)
_EIGHT = (torch.float8_e4m3fn, torch.int8)


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


def _check(status, what):
    if status != OK:
        raise GemmBtError(status, what)


def _rows(t, what="x"):
    """(tensor, row stride) of (..., d) seen as (rows, d) without a copy where the rows are evenly spaced."""
    if t.is_contiguous():
        if t.dim() == 0:
            raise ValueError("%s needs at least one dimension" % what)
        return t, t.shape[-1]
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
        return t, t.stride(0)
    return t.contiguous(), t.shape[-1]


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


def _stream(device, stream):
    # the handle alone: torch.cuda.current_stream would build a Stream object around it on every call (1.9 us)
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _float_code(t, what):
    if t.dtype not in _FLOATS:
        raise TypeError("%s must be float32, float16 or bfloat16, got %s" % (what, t.dtype))
    return _CODES[t.dtype]


def _same_shape(t, x, what):
    if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
        raise ValueError("%s must be a %s tensor of shape %s" % (what, x.dtype, tuple(x.shape)))


def _output(out, like, shape, dtype, device, what="out"):
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or not out.is_contiguous() or out.device != device:
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (what, dtype, tuple(shape), device))
    return out


# ---------------------------------------------------------------- norm and quantisation

def add_rms_norm(x, weight, residual=None, eps=1e-6, out_dtype=None, save_rstd=False, out=None, h_out=None, stream=None):
    """h = x + residual; y = h / sqrt(mean(h²) + eps) * weight, over the last dimension.

    x: float32, float16 or bfloat16; residual: as x, or None; weight: (d,) of x's type or float32.  ``out_dtype``: x's
    type (the default), another float type, or float8_e4m3fn or int8 for 8-bit rows with one float32 scale each (y is
    then q with y ≈ q * scale[..., None]).  Returns Normed(y, scale, h, rstd): scale for 8-bit rows, h where a residual
    is given (``h_out``, a contiguous tensor of x's type, receives it; it may be x or residual itself), rstd with
    ``save_rstd``.  h is used unrounded and returned rounded to x's type.
    """
    device = _on_gpu(x, weight, residual)
    x_code = _float_code(x, "x")
    _same_shape(residual, x, "residual")
    d = x.shape[-1] if x.dim() else 0
    if tuple(weight.shape) != (d,):
        raise ValueError("weight must have shape (%d,), got %s" % (d, tuple(weight.shape)))
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        raise TypeError("weight must be %s or float32, got %s" % (x.dtype, weight.dtype))
    y_dtype = x.dtype if out_dtype is None else out_dtype
    if y_dtype not in _FLOATS and y_dtype not in _EIGHT:
        raise TypeError("out_dtype must be a float type, float8_e4m3fn or int8, got %s" % y_dtype)
    lead = x.shape[:-1]
    xr, ldx = _rows(x)
    rr, ldr = (None, 0) if residual is None else _rows(residual, "residual")
    rows = x.numel() // d if d else 0
    y = _output(out, x, x.shape, y_dtype, device)
    h = None if residual is None else _output(h_out, x, x.shape, x.dtype, device, "h_out")
    scale = x.new_empty(lead, dtype=torch.float32) if y_dtype in _EIGHT else None
    rstd = x.new_empty(lead, dtype=torch.float32) if save_rstd else None
    with _on(device):
        _check(load().gemm_bt_rms_norm(xr.data_ptr(), ldx, _ptr(rr), ldr, _dense(weight).data_ptr(), y.data_ptr(), _ptr(h),
                                       _ptr(scale), _ptr(rstd), rows, d, eps, x_code, _CODES[weight.dtype],
                                       _CODES[y_dtype], _stream(device, stream)), "gemm_bt_rms_norm")
    return Normed(y, scale, h, rstd)


def quantize_rows(x, dtype=torch.float8_e4m3fn, stream=None):
    """The rows of x in 8 bits (float8_e4m3fn or int8) and one float32 scale each: Quantized(q, scale), x ≈ q * scale."""
    device = _on_gpu(x)
    x_code = _float_code(x, "x")
    if dtype not in _EIGHT:
        raise TypeError("dtype must be float8_e4m3fn or int8, got %s" % dtype)
    xr, ldx = _rows(x)
    d = x.shape[-1]
    q = x.new_empty(x.shape, dtype=dtype)
    scale = x.new_empty(x.shape[:-1], dtype=torch.float32)
    with _on(device):
        _check(load().gemm_bt_quantize_rows(xr.data_ptr(), ldx, q.data_ptr(), scale.data_ptr(), x.numel() // d if d else 0,
                                            d, x_code, _CODES[dtype], _stream(device, stream)), "gemm_bt_quantize_rows")
    return Quantized(q, scale)


def add_rms_norm_backward(dy, h, weight, rstd, dh=None, stream=None):
    """(dx, dweight) of add_rms_norm: h and rstd as it returned them (h is x where there was no residual), dy the
    gradient of y, dh the gradient that reaches h from elsewhere.  dx is the gradient of x and of residual alike."""
    device = _on_gpu(dy, h, weight, rstd, dh)
    code = _float_code(dy, "dy")
    _same_shape(h, dy, "h")
    _same_shape(dh, dy, "dh")
    d = dy.shape[-1] if dy.dim() else 0
    rows = dy.numel() // d if d else 0
    if tuple(weight.shape) != (d,):
        raise ValueError("weight must have shape (%d,), got %s" % (d, tuple(weight.shape)))
    if weight.dtype != dy.dtype and weight.dtype != torch.float32:
        raise TypeError("weight must be %s or float32, got %s" % (dy.dtype, weight.dtype))
    if rstd.dtype != torch.float32 or rstd.shape != dy.shape[:-1]:
        raise ValueError("rstd must be a float32 tensor of shape %s" % (tuple(dy.shape[:-1]),))
    dyr, ld_dy = _rows(dy, "dy")
    hr, ldh = _rows(h, "h")
    dhr, ld_dh = (None, 0) if dh is None else _rows(dh, "dh")
    dx = dy.new_empty(dy.shape)
    dw = weight.new_empty(d)
    lib = load()
    with _on(device):
        s = _stream(device, stream)
        need = ctypes.c_size_t()
        _check(lib.gemm_bt_rms_norm_backward_workspace(rows, d, ctypes.byref(need)), "gemm_bt_rms_norm_backward_workspace")
        ws = _scratch(dy, s, need.value)
        _check(lib.gemm_bt_rms_norm_backward(dyr.data_ptr(), ld_dy, hr.data_ptr(), ldh, _dense(weight).data_ptr(),
                                             _dense(rstd).data_ptr(), _ptr(dhr), ld_dh, dx.data_ptr(), dw.data_ptr(), rows,
                                             d, code, _CODES[weight.dtype], _ptr(ws), need.value, s),
               "gemm_bt_rms_norm_backward")
    return dx, dw


def _scratch(like, stream, nbytes):
    """Working memory of one call, on its stream: torch may hand it out again after that stream has passed the call."""
    if nbytes == 0:
        return None
    ws = like.new_empty(nbytes, dtype=torch.uint8)
    if stream != torch._C._cuda_getCurrentRawStream(like.device.index):
        ws.record_stream(torch.cuda.ExternalStream(stream, device=like.device))
    return ws


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
    device = _on_gpu(x, weight, bias, residual, x_scale, weight_scale)
    if x.dtype != weight.dtype:
        raise TypeError("x and weight must share one dtype")
    in_code = _CODES.get(x.dtype)
    if in_code is None or in_code == F32:
        raise TypeError("unsupported input dtype %s" % x.dtype)
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("expected x (..., K) and weight (N, K), got %s and %s" % (tuple(x.shape), tuple(weight.shape)))
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(ACTIVATIONS), activation))
    N, K = weight.shape
    lead = x.shape[:-1]
    M = lead.numel()
    shape = lead + (N,)
    wide = x.dtype if x.element_size() == 2 else torch.bfloat16
    y_dtype = wide if out_dtype is None else out_dtype
    if y_dtype not in _FLOATS:
        raise TypeError("out_dtype must be float32, float16 or bfloat16, got %s" % y_dtype)
    x, weight = _dense(x), _dense(weight)
    e = Epilogue()
    e.activation = act
    keep = []  # contiguous copies, alive until the launch
    for name, t, want in (("bias", bias, (N,)), ("residual", residual, shape)):
        if t is not None:
            if tuple(t.shape) != tuple(want):
                raise ValueError("%s must have shape %s, got %s" % (name, tuple(want), tuple(t.shape)))
            code = _float_code(t, name)
            t = _dense(t)
            keep.append(t)
            setattr(e, name, t.data_ptr())
            setattr(e, name + "_dtype", code)
    for name, t, want in (("row_scale", x_scale, lead), ("col_scale", weight_scale, (N,))):
        if t is not None:
            if tuple(t.shape) != tuple(want) or t.dtype != torch.float32:
                raise ValueError("%s must be a float32 tensor of shape %s"
                                 % ("x_scale" if name == "row_scale" else "weight_scale", tuple(want)))
            t = _dense(t)
            keep.append(t)
            setattr(e, name, t.data_ptr())
    y = _output(out, x, shape, y_dtype, device)
    z = None
    if save_preact:
        z = x.new_empty(shape, dtype=wide)
        e.preact = z.data_ptr()
        e.preact_dtype = _CODES[wide]
    out_code = _CODES[y_dtype]
    with _on(device):
        s = _stream(device, stream)
        lib, need = load(), ctypes.c_size_t()
        _check(lib.gemm_bt_epi_workspace_size(M, N, K, in_code, out_code, ctypes.byref(need)), "gemm_bt_epi_workspace_size")
        ws, ws_bytes = None, 0
        if need.value:
            t = workspace_for(device, s, need.value)
            ws, ws_bytes = t.data_ptr(), t.numel()
        _check(lib.gemm_bt_epi(x.data_ptr(), weight.data_ptr(), y.data_ptr(), M, N, K, in_code, out_code, ctypes.byref(e),
                                  ws, ws_bytes, s), "gemm_bt_epi")
    return (y, z) if save_preact else y


def linear_backward(dy, x, weight, preact=None, activation="none", bias_grad=True, need_dx=True, need_dweight=True,
                    stream=None):
    """The gradients of linear's x, weight and bias for 16-bit x and weight: LinearGrads(dx, dweight, dbias).

    dy (..., N): the gradient of the result, of x's type; preact: what linear returned with save_preact (not needed
    for the activation "none").  The gradient of the residual is dy itself.
    """
    device = _on_gpu(dy, x, weight, preact)
    if not (x.dtype == weight.dtype == dy.dtype) or x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("dy, x and weight must share float16 or bfloat16")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(ACTIVATIONS), activation))
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1] or dy.shape != x.shape[:-1] + weight.shape[:1]:
        raise ValueError("expected dy (..., N), x (..., K) and weight (N, K), got %s, %s and %s"
                         % (tuple(dy.shape), tuple(x.shape), tuple(weight.shape)))
    code = z_code = _CODES[dy.dtype]
    if act:
        if preact is None or preact.shape != dy.shape:
            raise ValueError("preact must be the pre-activation that linear returned, of shape %s" % (tuple(dy.shape),))
        z_code = _float_code(preact, "preact")
        preact = _dense(preact)
    N, K = weight.shape
    M = dy.shape[:-1].numel()
    dy, x, weight = _chunked(dy), _chunked(x), _chunked(weight)
    dx = x.new_empty(x.shape) if need_dx else None
    dw = weight.new_empty((N, K)) if need_dweight else None
    db = weight.new_empty(N) if bias_grad else None
    lib = load()
    with _on(device):
        s = _stream(device, stream)
        need = ctypes.c_size_t()
        _check(lib.gemm_bt_linear_backward_workspace(M, N, K, act, ctypes.byref(need)), "gemm_bt_linear_backward_workspace")
        ws = _scratch(dy, s, need.value)
        _check(lib.gemm_bt_linear_backward(dy.data_ptr(), x.data_ptr(), weight.data_ptr(), preact.data_ptr() if act else None,
                                           _ptr(dx), _ptr(dw), _ptr(db), M, N, K, act, code, z_code, _ptr(ws), need.value, s),
               "gemm_bt_linear_backward")
    return LinearGrads(dx, dw, db)
