"""Binding of the library's 8-bit linear-layer operators (C ABI in
``include/fp4q_linear.h``): root-mean-square norm with the residual's addition
and 8-bit output, its gradients, quantisation to 8 bits with a scale per 128
values, and the product of two 8-bit operands.

As in the rest of the package the functions carry the C entry points' names and
marshal arguments: torch tensors in, device pointers and the current HIP stream
out.  8-bit codes are float8 tensors whose rows begin at multiples of 16 bytes
(``stride(0) % 16 == 0``); scales are float32, [ceil(cols / 128), rows], or
[ceil(cols / 128), ceil(rows / 128)] for 128 x 128 tiles.

Autograd records none of these calls: their outputs require no gradients, and a call
whose inputs do, where gradients are recorded, warns.  A model calls forward and
backward functions in a ``torch.autograd.Function`` of its own.
"""
from __future__ import annotations

import ctypes
import functools
import warnings
from typing import NamedTuple, Optional

import torch

from . import FP4Q_ERR_SHAPE, FP4Q_OUT_BF16, FP4Q_OUT_F32, Fp4qError, _check, _stream
from . import lib as _base_lib

FP4Q_GROUP8 = 128
FP4Q_E4M3 = 0
FP4Q_E5M2 = 1
FP4Q_FLAG_TILES = 2
FP4Q_FLAG_ACCUMULATE = 4

_FORMATS = {torch.float8_e4m3fn: FP4Q_E4M3, torch.float8_e5m2: FP4Q_E5M2}
_TYPES = {torch.float32: FP4Q_OUT_F32, torch.bfloat16: FP4Q_OUT_BF16}
_bound = None


def _lib() -> ctypes.CDLL:
    global _bound
    L = _base_lib()
    if _bound is not L:
        P, I, I64, U32, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
        Z, SZ = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        L.fp4q_rmsnorm.argtypes = [P, P, P, F, I64, I64, I, P, P, P, I64, P, P, P]
        L.fp4q_rmsnorm_backward_workspace.argtypes = [I64, I64, SZ]
        L.fp4q_rmsnorm_backward.argtypes = [P, P, P, P, P, I64, I64, I, P, P, P, Z, P]
        L.fp4q_quantize8.argtypes = [P, I64, I64, I, I, P, I64, P, P, I64, P, U32, P]
        L.fp4q_gemm8_workspace.argtypes = [I64, I64, I64, I, U32, SZ]
        L.fp4q_gemm8.argtypes = [P, I64, I, P, P, I64, I, P, I64, I64, I64, P, I, U32, P, Z, P]
        _bound = L
    return L


# The checks and launches below run once per call of a serving step's smallest
# operators, whose kernels take a few microseconds: they are written to cost little.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# A launch on a default stream goes to the current GPU, whichever one the tensors are on:
# with tensors on another GPU, a function calls itself with that one current.
_current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch_stream(stream, index):
    """The address of the HIP stream to launch on (see _stream), on the GPU of that index."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(index)
    return _stream(stream, torch.device("cuda", index))


def _gpu(*tensors):
    """The index of the one GPU that every tensor argument (None apart) lies on."""
    first = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != first or first < 0:
            raise ValueError("fp4q: every tensor must be on the same GPU (%s, %s)" % (tensors[0].device, t.device))
    return first


def _unrecorded(name):
    """The warning that a gradient ends here (inputs of `name` require one)."""
    if torch.is_grad_enabled():
        warnings.warn("fp4q: autograd does not record %s: its outputs pass no gradient on to its inputs; call it "
                      "in a torch.autograd.Function, or under torch.no_grad()" % name, stacklevel=3)


@functools.lru_cache(maxsize=4096)
def _workspace(which, *sizes) -> int:
    """The workspace bytes that the C library asks for (a function of the sizes)."""
    need = ctypes.c_size_t()
    _check(getattr(_lib(), which)(*sizes, ctypes.byref(need)))
    return need.value


def _groups(n: int) -> int:
    return (n + FP4Q_GROUP8 - 1) // FP4Q_GROUP8


def _like(t, name, shape, dtype):
    """A tensor argument of exactly this shape and type, contiguous."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError("fp4q: %s must be a torch tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("fp4q: %s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("fp4q: %s must have shape %s, has %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("fp4q: %s must be contiguous" % name)


def _typed(t, name):
    """The type code of a 2-D contiguous float32 or bfloat16 tensor, and its shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("fp4q: %s must be a torch tensor" % name)
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError("fp4q: %s must be float32 or bfloat16, got %s" % (name, t.dtype))
    if t.dim() != 2:
        raise ValueError("fp4q: expected a 2-D tensor [rows, cols]")
    if not t.is_contiguous():
        raise ValueError("fp4q: expected a contiguous tensor")
    rows, cols = t.shape
    if cols == 0:
        raise Fp4qError(FP4Q_ERR_SHAPE)
    return code, rows, cols


def _new(like, shape, dtype, stream):
    """An uninitialised output on the GPU of `like`, allocated for the stream that the
    kernel will run on (so that its memory goes to no other work meanwhile)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _codes_out(like, rows, cols, dtype, stream):
    """Uninitialised codes [rows, cols] whose rows begin at multiples of 16 bytes."""
    pitch = (cols + 15) // 16 * 16
    t = _new(like, (rows, pitch), dtype, stream)
    return t if pitch == cols else t.as_strided((rows, cols), (pitch, 1))  # a slice costs the host twice as much


def _codes_in(t, name):
    """Format, rows, cols and pitch of an 8-bit operand; its rows must be readable up
    to a multiple of 16 bytes (the kernels load 16 bytes at a time)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("fp4q: %s must be a torch tensor" % name)
    fmt = _FORMATS.get(t.dtype)
    if fmt is None:
        raise TypeError("fp4q: %s must be float8_e4m3fn or float8_e5m2, got %s" % (name, t.dtype))
    if t.dim() != 2:
        raise ValueError("fp4q: expected a 2-D tensor [rows, cols]")
    rows, cols = t.shape
    if cols % 16 == 0 and t.is_contiguous():
        return fmt, rows, cols, cols
    wide = (cols + 15) // 16 * 16
    pitch = t.stride(0) if rows > 1 else wide
    if rows and cols:
        if cols > 1 and t.stride(1) != 1:
            raise ValueError("fp4q: the columns of %s must be contiguous" % name)
        if pitch % 16 or pitch < cols:
            raise ValueError("fp4q: the rows of %s must begin at multiples of 16 bytes" % name)
        if t.storage_offset() + (rows - 1) * pitch + wide > t.untyped_storage().nbytes():
            raise ValueError("fp4q: the last row of %s must be readable up to a multiple of 16 bytes" % name)
    else:
        pitch = wide
    return fmt, rows, cols, pitch


def _at(t):
    return None if t is None else t.data_ptr()


class RmsNorm(NamedTuple):
    """What :func:`fp4q_rmsnorm` returns; what was not asked for is None."""
    h: torch.Tensor
    y: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


def fp4q_rmsnorm(x, weight, eps: float, residual=None, h=None, want_y: bool = True,
                 want_codes: bool = False, want_rstd: bool = False, stream=None) -> RmsNorm:
    """h = x + residual (x itself without one), y = h / sqrt(mean(h^2) + eps) * weight of
    a float32 or bfloat16 tensor [rows, cols]: y in that type (want_y) and/or as E4M3
    codes [rows, cols] with scales [ceil(cols / 128), rows] (want_codes), and the
    reciprocal roots (want_rstd) that the backward pass takes.  ``h=residual`` updates
    the residual in place."""
    dtype, rows, cols = _typed(x, "input")
    kind = x.dtype
    _like(weight, "weight", (cols,), kind)
    if residual is not None:
        _like(residual, "residual", x.shape, kind)
        if h is not None:
            _like(h, "h", x.shape, kind)
    elif h is not None:
        raise ValueError("fp4q: h is an output of the sum with a residual")
    if not (want_y or want_codes):
        raise ValueError("fp4q: ask for y, codes or both")
    if x.requires_grad or weight.requires_grad or (residual is not None and residual.requires_grad):
        _unrecorded("fp4q_rmsnorm")
    gpu = _gpu(x, weight, residual, h)
    if _current_gpu() != gpu:
        with torch.cuda.device(gpu), torch.no_grad():
            return fp4q_rmsnorm(x, weight, eps, residual, h, want_y, want_codes, want_rstd, stream)
    if residual is not None and h is None:
        h = _new(x, (rows, cols), kind, stream)
    y = _new(x, (rows, cols), kind, stream) if want_y else None
    codes = scales = None
    if want_codes:
        codes = _codes_out(x, rows, cols, torch.float8_e4m3fn, stream)
        scales = _new(x, (_groups(cols), rows), torch.float32, stream)
    rstd = _new(x, (rows,), torch.float32, stream) if want_rstd else None
    status = (_bound or _lib()).fp4q_rmsnorm(_at(x), _at(residual), _at(weight), eps, rows, cols, dtype, _at(h), _at(y),
                                             _at(codes), (cols + 15) // 16 * 16, _at(scales), _at(rstd),
                                             _launch_stream(stream, gpu))
    if status:
        raise Fp4qError(status)
    return RmsNorm(x if residual is None else h, y, codes, scales, rstd)


def fp4q_rmsnorm_backward(dy, h, weight, rstd, dh=None, stream=None):
    """Gradients of :func:`fp4q_rmsnorm` -> (dx, dweight): dx is the gradient of x and of
    the residual alike, in the inputs' type; dweight is float32 [cols].  ``h`` is the
    forward's h, ``dh`` the gradient that reaches h by other paths."""
    dtype, rows, cols = _typed(dy, "dy")
    _like(h, "h", dy.shape, dy.dtype)
    _like(weight, "weight", (cols,), dy.dtype)
    _like(rstd, "rstd", (rows,), torch.float32)
    if dh is not None:
        _like(dh, "dh", dy.shape, dy.dtype)
    if dy.requires_grad or h.requires_grad or weight.requires_grad or (dh is not None and dh.requires_grad):
        _unrecorded("fp4q_rmsnorm_backward")
    gpu = _gpu(dy, h, weight, rstd, dh)
    if _current_gpu() != gpu:
        with torch.cuda.device(gpu), torch.no_grad():
            return fp4q_rmsnorm_backward(dy, h, weight, rstd, dh, stream)
    need = _workspace("fp4q_rmsnorm_backward_workspace", rows, cols)
    dx = _new(dy, (rows, cols), dy.dtype, stream)
    dweight = _new(dy, (cols,), torch.float32, stream)
    space = _new(dy, (need,), torch.uint8, stream)
    status = (_bound or _lib()).fp4q_rmsnorm_backward(_at(dy), _at(h), _at(weight), _at(rstd), _at(dh), rows, cols,
                                                      dtype, _at(dx), _at(dweight), _at(space), need,
                                                      _launch_stream(stream, gpu))
    if status:
        raise Fp4qError(status)
    return dx, dweight


class Quantized8(NamedTuple):
    """What :func:`fp4q_quantize8` returns; what was not asked for is None."""
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    codes_t: Optional[torch.Tensor]
    scales_t: Optional[torch.Tensor]


def fp4q_quantize8(x, dtype=torch.float8_e4m3fn, tiles: bool = False, straight: bool = True,
                   transposed: bool = False, stream=None) -> Quantized8:
    """8-bit codes and scales of a float32 or bfloat16 tensor [rows, cols]: of x
    (straight) and/or of its transpose (transposed), with one scale per 128
    neighbours of a row of what is written, or per 128 x 128 tile (tiles)."""
    kind, rows, cols = _typed(x, "input")
    fmt = _FORMATS.get(dtype)
    if fmt is None:
        raise TypeError("fp4q: codes are float8_e4m3fn or float8_e5m2, not %s" % (dtype,))
    if not (straight or transposed):
        raise ValueError("fp4q: ask for straight, transposed or both")
    if x.requires_grad:
        _unrecorded("fp4q_quantize8")
    gpu = _gpu(x)
    if _current_gpu() != gpu:
        with torch.cuda.device(gpu), torch.no_grad():
            return fp4q_quantize8(x, dtype, tiles, straight, transposed, stream)
    codes = scales = codes_t = scales_t = None
    gr, gc = _groups(rows), _groups(cols)
    if straight:
        codes = _codes_out(x, rows, cols, dtype, stream)
        scales = _new(x, (gc, gr if tiles else rows), torch.float32, stream)
    if transposed:
        codes_t = _codes_out(x, cols, rows, dtype, stream)
        scales_t = _new(x, (gr, gc if tiles else cols), torch.float32, stream)
    status = (_bound or _lib()).fp4q_quantize8(_at(x), rows, cols, kind, fmt, _at(codes), (cols + 15) // 16 * 16,
                                               _at(scales), _at(codes_t), (rows + 15) // 16 * 16, _at(scales_t),
                                               FP4Q_FLAG_TILES if tiles else 0, _launch_stream(stream, gpu))
    if status:
        raise Fp4qError(status)
    return Quantized8(codes, scales, codes_t, scales_t)


def fp4q_gemm8(a, a_scales, b, b_scales, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """The product of two 8-bit operands: a [M, K] with a_scales [ceil(K / 128), M] and
    b [N, K] with b_scales [ceil(K / 128), N] or, for tiles, [ceil(K / 128), ceil(N / 128)]
    -> [M, N] float32 or bfloat16 (bfloat16 when neither ``out`` nor ``out_dtype`` says
    otherwise).  ``accumulate`` adds the product to a float32 ``out``.  A bfloat16 product
    drops, of every 8 neighbouring products, what lies below 2^-13 of the largest: sums in
    which large products cancel want float32 output."""
    fa, M, K, a_pitch = _codes_in(a, "a")
    fb, N, kb, b_pitch = _codes_in(b, "b")
    if kb != K:
        raise ValueError("fp4q: a has %d columns, b %d" % (K, kb))
    groups, row_tiles = _groups(K), _groups(N)
    _like(a_scales, "a's scales", (groups, M), torch.float32)
    tiles = isinstance(b_scales, torch.Tensor) and b_scales.shape == (groups, row_tiles)
    _like(b_scales, "b's scales", (groups, row_tiles if tiles else N), torch.float32)
    dtype = out_dtype or torch.bfloat16
    if out is not None:
        if out_dtype is not None and out_dtype != out.dtype:
            raise TypeError("fp4q: out is %s, out_dtype %s" % (out.dtype, out_dtype))
        dtype = out.dtype
        _like(out, "out", (M, N), dtype)
    elif accumulate:
        raise ValueError("fp4q: accumulate needs out")
    code = _TYPES.get(dtype)
    if code is None or (accumulate and code != FP4Q_OUT_F32):
        raise TypeError("fp4q: out must be float32%s, got %s" % ("" if accumulate else " or bfloat16", dtype))
    if a.requires_grad or a_scales.requires_grad or b.requires_grad or b_scales.requires_grad:
        _unrecorded("fp4q_gemm8")
    gpu = _gpu(a, a_scales, b, b_scales, out)
    if _current_gpu() != gpu:
        with torch.cuda.device(gpu), torch.no_grad():
            return fp4q_gemm8(a, a_scales, b, b_scales, out, out_dtype, accumulate, stream)
    flags = (FP4Q_FLAG_TILES if tiles else 0) | (FP4Q_FLAG_ACCUMULATE if accumulate else 0)
    need = _workspace("fp4q_gemm8_workspace", M, N, K, code, flags)
    if out is None:
        out = _new(a_scales, (M, N), dtype, stream)
    space = _new(a_scales, (need,), torch.uint8, stream) if need else None
    status = (_bound or _lib()).fp4q_gemm8(_at(a), a_pitch, fa, _at(a_scales), _at(b), b_pitch, fb, _at(b_scales), M, N, K,
                                           _at(out), code, flags, _at(space), need, _launch_stream(stream, gpu))
    if status:
        raise Fp4qError(status)
    return out
