"""Binding of the library's operators for gated feed-forward layers (C ABI in
``include/fp4q_gated.h``): the gated product of 8-bit operands and its gradients, and
products of a few rows with weights held as FP4 payloads.

8-bit codes and scales are those of the 8-bit linear-layer operators, payloads those of
``fp4q_compress``.  The joined weight of :func:`fp4q_gated8` and the joined gradients of
:func:`fp4q_gated8_backward` hold the gate's N rows (columns), zeros up to the next multiple
of 128, and the up projection's N.

Autograd records none of these calls: a call whose inputs require gradients, where
gradients are recorded, warns.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import ctypes

import torch

from . import FP4Q_BLOCK, FP4Q_ERR_SHAPE, FP4Q_FLAG_NO_FWHT, FP4Q_GROUP, FP4Q_OUT_BF16, FP4Q_OUT_F32, Fp4qError
from . import lib as _base_lib
from .linear import (FP4Q_GROUP8, _FORMATS, _TYPES, _at, _codes_in, _codes_out, _current_gpu, _gpu, _groups,
                     _launch_stream, _like, _new, _typed, _unrecorded)
from . import linear as _linear

FP4Q_ACT_SILU = 0
FP4Q_ACT_GELU = 1
FP4Q_ACT_GELU_TANH = 2
FP4Q_ACT_RELU = 3

_ACTS = {"silu": FP4Q_ACT_SILU, "gelu": FP4Q_ACT_GELU, "gelu_tanh": FP4Q_ACT_GELU_TANH, "relu": FP4Q_ACT_RELU}
_bound = None


def _lib() -> ctypes.CDLL:
    global _bound
    L = _base_lib()
    if _bound is not L:
        P, I, I64, U32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32
        Z, SZ = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        L.fp4q_gated8_workspace.argtypes = [I64, I64, I64, SZ]
        L.fp4q_gated8.argtypes = [P, I64, I, P, P, I64, I, P, I64, I64, I64, I, P, P, P, P, Z, P]
        L.fp4q_gated8_backward.argtypes = [P, P, P, I64, I64, I, I, I, P, I64, P, P, I64, P, P, I64, P, P]
        L.fp4q_gemv4_workspace.argtypes = [I64, I64, I, U32, SZ]
        L.fp4q_gemv4.argtypes = [P, I, I64, P, P, P, I64, I64, P, I, U32, P, Z, P]
        L.fp4q_gated4.argtypes = [P, I, I64, P, P, P, P, P, P, I64, I64, I, P, I, U32, P, Z, P]
        _bound = L
    return L


def _act(activation) -> int:
    code = _ACTS.get(activation)
    if code is None:
        raise ValueError("fp4q: the activation is one of %s, not %r" % (", ".join(_ACTS), activation))
    return code


class Gated8(NamedTuple):
    """What :func:`fp4q_gated8` returns; what was not asked for is None."""
    y: torch.Tensor
    gate: Optional[torch.Tensor]
    up: Optional[torch.Tensor]


def fp4q_gated8(a, a_scales, gate_up, gate_up_scales, activation: str = "silu", want_pre: bool = False,
                stream=None) -> Gated8:
    """y = act(a gate^T) * (a up^T) as bfloat16 [M, N] of 8-bit operands: a [M, K] with
    a_scales [ceil(K / 128), M] and the joined weight gate_up [R, K] with tiles of scales
    [ceil(K / 128), ceil(R / 128)], R = N rounded up to a multiple of 128, plus N.
    ``want_pre`` also returns both products in bfloat16, for the backward pass.
    ``activation`` is "silu", "gelu" (erf), "gelu_tanh" or "relu"."""
    act = _act(activation)
    fa, M, K, a_pitch = _codes_in(a, "a")
    fw, R, kw, w_pitch = _codes_in(gate_up, "gate_up")
    if kw != K:
        raise ValueError("fp4q: a has %d columns, gate_up %d" % (K, kw))
    groups, tiles = _groups(K), _groups(R)
    if tiles % 2:
        raise ValueError("fp4q: gate_up has %d rows: not N rows of the gate, padded to a multiple of %d, "
                         "and N of the up projection" % (R, FP4Q_GROUP8))
    N = R - tiles // 2 * FP4Q_GROUP8
    _like(a_scales, "a's scales", (groups, M), torch.float32)
    _like(gate_up_scales, "gate_up's scales", (groups, tiles), torch.float32)
    if a.requires_grad or a_scales.requires_grad or gate_up.requires_grad or gate_up_scales.requires_grad:
        _unrecorded("fp4q_gated8")
    gpu = _gpu(a, a_scales, gate_up, gate_up_scales)
    if _current_gpu() != gpu:
        with torch.cuda.device(gpu), torch.no_grad():
            return fp4q_gated8(a, a_scales, gate_up, gate_up_scales, activation, want_pre, stream)
    L = _bound or _lib()
    need = _linear._workspace("fp4q_gated8_workspace", M, N, K)
    y = _new(a_scales, (M, N), torch.bfloat16, stream)
    gate = up = None
    if want_pre:
        gate, up = (_new(a_scales, (M, N), torch.bfloat16, stream) for _ in range(2))
    space = _new(a_scales, (need,), torch.uint8, stream) if need else None
    status = L.fp4q_gated8(_at(a), a_pitch, fa, _at(a_scales), _at(gate_up), w_pitch, fw, _at(gate_up_scales), M, N, K,
                           act, _at(y), _at(gate), _at(up), _at(space), need, _launch_stream(stream, gpu))
    if status:
        raise Fp4qError(status)
    return Gated8(y, gate, up)


class Gated8Grad(NamedTuple):
    """What :func:`fp4q_gated8_backward` returns; what was not asked for is None."""
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    codes_t: Optional[torch.Tensor]
    scales_t: Optional[torch.Tensor]
    y_codes_t: Optional[torch.Tensor]
    y_scales_t: Optional[torch.Tensor]


def fp4q_gated8_backward(dy, gate, up, activation: str = "silu", dtype=torch.float8_e5m2, straight: bool = True,
                         transposed: bool = True, want_y: bool = False, stream=None) -> Gated8Grad:
    """Gradients of :func:`fp4q_gated8` from dy, gate and up [M, N] (all float32 or all
    bfloat16) as 8-bit codes with a scale per 128: the joined [dgate | 0 | dup] along its
    rows (``straight``: codes [M, R], scales [ceil(R / 128), M]) and/or along its columns
    (``transposed``: codes_t [R, M], scales_t [ceil(M / 128), R]), in ``dtype``; with
    ``want_y`` also y = act(gate) * up along its columns, E4M3 (y_codes_t [N, M],
    y_scales_t [ceil(M / 128), N])."""
    act = _act(activation)
    kind, M, N = _typed(dy, "dy")
    _like(gate, "gate", dy.shape, dy.dtype)
    _like(up, "up", dy.shape, dy.dtype)
    fmt = _FORMATS.get(dtype)
    if fmt is None:
        raise TypeError("fp4q: codes are float8_e4m3fn or float8_e5m2, not %s" % (dtype,))
    if not (straight or transposed or want_y):
        raise ValueError("fp4q: ask for straight, transposed or y")
    if dy.requires_grad or gate.requires_grad or up.requires_grad:
        _unrecorded("fp4q_gated8_backward")
    gpu = _gpu(dy, gate, up)
    if _current_gpu() != gpu:
        with torch.cuda.device(gpu), torch.no_grad():
            return fp4q_gated8_backward(dy, gate, up, activation, dtype, straight, transposed, want_y, stream)
    R = _groups(N) * FP4Q_GROUP8 + N
    wide, high = (R + 15) // 16 * 16, (M + 15) // 16 * 16
    codes = scales = codes_t = scales_t = y_t = y_scales = None
    if straight:
        codes = _codes_out(dy, M, R, dtype, stream)
        scales = _new(dy, (_groups(R), M), torch.float32, stream)
    if transposed:
        codes_t = _codes_out(dy, R, M, dtype, stream)
        scales_t = _new(dy, (_groups(M), R), torch.float32, stream)
    if want_y:
        y_t = _codes_out(dy, N, M, torch.float8_e4m3fn, stream)
        y_scales = _new(dy, (_groups(M), N), torch.float32, stream)
    status = (_bound or _lib()).fp4q_gated8_backward(
        _at(dy), _at(gate), _at(up), M, N, kind, act, fmt, _at(codes), wide, _at(scales), _at(codes_t), high,
        _at(scales_t), _at(y_t), high, _at(y_scales), _launch_stream(stream, gpu))
    if status:
        raise Fp4qError(status)
    return Gated8Grad(codes, scales, codes_t, scales_t, y_t, y_scales)


def _payload(w, name, K):
    """The number of rows of a weight's payload (codes, micro-scales, block scales) with K columns."""
    try:
        codes, micro, block = w
    except (TypeError, ValueError):
        raise TypeError("fp4q: %s must be a payload (codes, micro-scales, block scales)" % name) from None
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise TypeError("fp4q: %s's codes must be a 2-D torch tensor" % name)
    N = codes.shape[0]
    _like(codes, name + "'s codes", (N, K // 2), torch.uint8)
    _like(micro, name + "'s micro-scales", (N, K // FP4Q_GROUP), torch.uint8)
    _like(block, name + "'s block scales", (N, K // FP4Q_BLOCK), torch.float32)
    return N, codes, micro, block


def _few_rows(x, out, out_dtype, N, flags):
    """What both 4-bit products do with x and out: x's and out's type codes, out's type, workspace bytes."""
    if flags & ~FP4Q_FLAG_NO_FWHT:
        raise ValueError("fp4q: flags are 0 or FP4Q_FLAG_NO_FWHT")
    dtype = out_dtype or (x.dtype if out is None else out.dtype)
    if out is not None:
        if out.dtype != dtype:
            raise TypeError("fp4q: out is %s, out_dtype %s" % (out.dtype, out_dtype))
        _like(out, "out", (x.shape[0], N), dtype)
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError("fp4q: out must be float32 or bfloat16, got %s" % (dtype,))
    return code, dtype


def _rows_in(x):
    kind, M, K = _typed(x, "x")
    if K % FP4Q_BLOCK:
        raise Fp4qError(FP4Q_ERR_SHAPE)
    return kind, M, K


def fp4q_gemv4(x, weight, flags: int = 0, out=None, out_dtype=None, stream=None):
    """x [M, K] (float32 or bfloat16) times the transpose of a weight [N, K] held as a
    payload (codes, micro-scales, block scales), as ``fp4q_compress`` with the same
    ``flags`` makes it -> [M, N] in x's type, ``out_dtype`` or ``out``'s.  Made for few
    rows: its time is that of reading the payload, once for every 32 of them or fewer."""
    kind, M, K = _rows_in(x)
    N, codes, micro, block = _payload(weight, "weight", K)
    code, dtype = _few_rows(x, out, out_dtype, N, flags)
    if x.requires_grad or block.requires_grad:
        _unrecorded("fp4q_gemv4")
    gpu = _gpu(x, codes, micro, block, out)
    if _current_gpu() != gpu:
        with torch.cuda.device(gpu), torch.no_grad():
            return fp4q_gemv4(x, weight, flags, out, out_dtype, stream)
    L = _bound or _lib()
    need = _linear._workspace("fp4q_gemv4_workspace", M, K, kind, flags)
    if out is None:
        out = _new(x, (M, N), dtype, stream)
    space = _new(x, (need,), torch.uint8, stream) if need else None
    status = L.fp4q_gemv4(_at(x), kind, M, _at(codes), _at(micro), _at(block), N, K, _at(out), code, flags, _at(space),
                          need, _launch_stream(stream, gpu))
    if status:
        raise Fp4qError(status)
    return out


def fp4q_gated4(x, gate, up, activation: str = "silu", flags: int = 0, out=None, out_dtype=None, stream=None):
    """act(x gate^T) * (x up^T) of x [M, K] (float32 or bfloat16) and two weights [N, K]
    held as payloads, as in :func:`fp4q_gemv4` -> [M, N] in x's type, ``out_dtype`` or
    ``out``'s."""
    act = _act(activation)
    kind, M, K = _rows_in(x)
    N, *gates = _payload(gate, "gate", K)
    n, *ups = _payload(up, "up", K)
    if n != N:
        raise ValueError("fp4q: the gate has %d rows, the up projection %d" % (N, n))
    code, dtype = _few_rows(x, out, out_dtype, N, flags)
    if x.requires_grad or gates[2].requires_grad or ups[2].requires_grad:
        _unrecorded("fp4q_gated4")
    gpu = _gpu(x, *gates, *ups, out)
    if _current_gpu() != gpu:
        with torch.cuda.device(gpu), torch.no_grad():
            return fp4q_gated4(x, gate, up, activation, flags, out, out_dtype, stream)
    L = _bound or _lib()
    need = _linear._workspace("fp4q_gemv4_workspace", M, K, kind, flags)
    if out is None:
        out = _new(x, (M, N), dtype, stream)
    space = _new(x, (need,), torch.uint8, stream) if need else None
    status = L.fp4q_gated4(_at(x), kind, M, *map(_at, gates), *map(_at, ups), N, K, act, _at(out), code, flags,
                           _at(space), need, _launch_stream(stream, gpu))
    if status:
        raise Fp4qError(status)
    return out
