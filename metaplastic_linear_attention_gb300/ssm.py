"""Binding of the state-space operators of ``libpalimpsa.so`` (``include/palimpsa.h``):
the short causal convolution and the selective scan, for prompts, packed batches, single
tokens and training. As in :mod:`.binding`, the functions keep the C names, marshal
device tensors, raise :class:`PalimpsaError` on a non-OK status, and have no fallback.

Token arrays are laid out row by row (``[B, T, D]``, or ``[rows, D]`` packed) and share
one dtype (bf16 or fp32). Input rows may be slices of wider rows (last dimension
contiguous, rows evenly spaced); outputs are dense.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import PALIMPSA_BF16, PALIMPSA_F32, PalimpsaError, _check, _packed_offsets

PALIMPSA_CONV_SILU = 1       # palimpsa_conv_flags
PALIMPSA_SCAN_SOFTPLUS = 1   # palimpsa_scan_flags
CHECKPOINT_TOKENS = 16
F32 = torch.float32


class _Strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_longlong) for n in ("x", "dt", "B", "C", "z", "dy")]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = binding.load_library()
        p, i, ll, u = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_uint
        st = ctypes.POINTER(_Strides)
        sig = {
            "palimpsa_causal_conv": [p, ll, p, p, p, p, p, p, i, i, i, i, i, u, i, p],
            "palimpsa_causal_conv_step": [p, ll, p, p, p, p, i, i, i, u, i, p],
            "palimpsa_causal_conv_backward": [p, ll, p, p, p, p, ll, p, p, p, p, p, p, i, i, i, i, i, u, i, p],
            "palimpsa_selective_scan": [p] * 12 + [st, p, i, i, i, i, i, i, u, i, p],
            "palimpsa_selective_scan_step": [p] * 10 + [st, i, i, i, i, u, i, p],
            "palimpsa_selective_scan_backward": [p] * 20 + [st, p, i, i, i, i, i, i, u, i, p],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = i, args
        lib.palimpsa_selective_scan_checkpoint_bytes.restype = ctypes.c_size_t
        lib.palimpsa_selective_scan_checkpoint_bytes.argtypes = [i, i, i, i, i]
        _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype(x, name):
    if x.dtype == torch.bfloat16:
        return PALIMPSA_BF16
    if x.dtype == F32:
        return PALIMPSA_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {x.dtype}")


def _rows(t, name, shape, dtype, dev, lead):
    """Checks a token array whose first `lead` dimensions count rows; returns its row
    stride in elements (0: dense)."""
    if t is None:
        return 0
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.is_contiguous():
        return 0
    st, width = t.stride(), 1
    for k in range(len(shape) - 1, lead - 1, -1):
        if shape[k] != 1 and st[k] != width:
            raise ValueError(f"{name}: a row must be contiguous, got strides {st}")
        width *= shape[k]
    if lead == 1:
        ld = st[0]
    elif shape[1] == 1:
        ld = st[0]
    else:
        ld = st[1]
        if shape[0] != 1 and st[0] != shape[1] * ld:
            raise ValueError(f"{name}: rows must be evenly spaced, got strides {st}")
    if ld < width:
        raise ValueError(f"{name}: rows overlap, got strides {st}")
    return ld


class _Call:
    """The device and stream of one call: the tensors' device, the caller's stream or
    the current one. Tensors used on a stream other than the current one are recorded
    there, so that the allocator keeps them until that stream is done."""

    def __init__(self, x, name, stream):
        if not x.is_cuda:
            raise ValueError(f"{name} takes device tensors")
        self.dev, self.stream, self.name = x.device, stream, name

    def __call__(self, fn, tensors, *args):
        if self.dev.index == torch.cuda.current_device():
            rc = self._run(fn, tensors, args)
        else:
            with torch.cuda.device(self.dev):
                rc = self._run(fn, tensors, args)
        if rc != 0:
            raise PalimpsaError(rc, self.name)

    def _run(self, fn, tensors, args):
        rc = fn(*args, binding._stream_handle(self.stream))
        if self.stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)
        return rc


def _batch(x, cu_seqlens, max_seqlen, dev, stream, name):
    """(B, T, max_seqlen, offsets on the device, row dimensions) of a token array x."""
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError(f"{name}: x must be [B, T, D], got {tuple(x.shape)}")
        return x.shape[0], x.shape[1], x.shape[1], None, 2
    if x.dim() != 2:
        raise ValueError(f"{name}: packed x must be [rows, D], got {tuple(x.shape)}")
    cu, n, longest = _packed_offsets(cu_seqlens, max_seqlen, dev, stream)
    return n, x.shape[0], longest, cu, 1


def _new(t, name, shape, dtype, dev, zero=False):
    """An output: checked when given, else allocated (zeroed where rows may stay unwritten)."""
    if t is None:
        return (torch.zeros if zero else torch.empty)(shape, dtype=dtype, device=dev)
    _check(t, name, shape, dtype, dev)
    return t


# ------------------------------------------------------------------ causal convolution

def _conv_params(x, weight, bias, dev):
    D, W = x.shape[-1], weight.shape[-1]
    _check(weight, "weight", (D, W), F32, dev)
    _check(bias, "bias", (D,), F32, dev)
    return D, W


def palimpsa_causal_conv(x, weight, bias=None, state0=None, *, silu=True, cu_seqlens=None, max_seqlen=None, y=None,
                         state_T=None, stream=None):
    """Depthwise causal convolution along the tokens (see palimpsa.h).

    x [B, T, D], or [rows, D] with cu_seqlens [B + 1] int32 (max_seqlen: the longest
    sequence, read from cu_seqlens when not given, which synchronises); weight [D, W],
    bias [D] fp32; state0 [B, W - 1, D]: the inputs before each sequence, or None for
    zeros. Returns (y, state_T), both in x's dtype; state_T may be given as state0."""
    name = "palimpsa_causal_conv"
    call = _Call(x, name, stream)
    dev = x.device
    B, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, stream, name)
    D, W = _conv_params(x, weight, bias, dev)
    ld = _rows(x, "x", tuple(x.shape), x.dtype, dev, lead)
    _check(state0, "state0", (B, W - 1, D), x.dtype, dev)
    y = _new(y, "y", tuple(x.shape), x.dtype, dev, cu is not None)
    state_T = _new(state_T, "state_T", (B, W - 1, D), x.dtype, dev)
    call(_library().palimpsa_causal_conv, (x, weight, bias, state0, y, state_T, cu),
         _ptr(x), ld, _ptr(weight), _ptr(bias), _ptr(state0), _ptr(y), _ptr(state_T), _ptr(cu), B, T, longest, D, W,
         PALIMPSA_CONV_SILU if silu else 0, _dtype(x, "x"))
    return y, state_T


def palimpsa_causal_conv_step(x, weight, bias, state, *, silu=True, y=None, stream=None):
    """One token of the convolution (see palimpsa.h): x [B, D], state [B, W - 1, D] updated in
    place. Returns y [B, D]."""
    name = "palimpsa_causal_conv_step"
    call = _Call(x, name, stream)
    dev = x.device
    if x.dim() != 2:
        raise ValueError(f"{name}: x must be [B, D], got {tuple(x.shape)}")
    B = x.shape[0]
    D, W = _conv_params(x, weight, bias, dev)
    ld = _rows(x, "x", (B, D), x.dtype, dev, 1)
    _check(state, "state", (B, W - 1, D), x.dtype, dev)
    y = _new(y, "y", (B, D), x.dtype, dev)
    call(_library().palimpsa_causal_conv_step, (x, weight, bias, state, y),
         _ptr(x), ld, _ptr(weight), _ptr(bias), _ptr(state), _ptr(y), B, D, W, PALIMPSA_CONV_SILU if silu else 0,
         _dtype(x, "x"))
    return y


def palimpsa_causal_conv_backward(x, weight, bias, state0, dy, dstate_T=None, *, silu=True, cu_seqlens=None,
                                  max_seqlen=None, want_state_grad=True, stream=None):
    """Gradients through palimpsa_causal_conv (see palimpsa.h). Returns a dict: dx (x's dtype; zero
    in rows outside every sequence), dweight [D, W], dbias [D] (fp32), and dstate0
    [B, W - 1, D] (x's dtype) when want_state_grad."""
    name = "palimpsa_causal_conv_backward"
    call = _Call(x, name, stream)
    dev = x.device
    B, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, stream, name)
    D, W = _conv_params(x, weight, bias, dev)
    ld = _rows(x, "x", tuple(x.shape), x.dtype, dev, lead)
    ldy = _rows(dy, "dy", tuple(x.shape), x.dtype, dev, lead)
    _check(state0, "state0", (B, W - 1, D), x.dtype, dev)
    _check(dstate_T, "dstate_T", (B, W - 1, D), x.dtype, dev)
    g = {"dx": _new(None, "dx", tuple(x.shape), x.dtype, dev, cu is not None),
         "dweight": _new(None, "dweight", (D, W), F32, dev), "dbias": _new(None, "dbias", (D,), F32, dev)}
    if want_state_grad:
        # a sequence that is skipped for its offsets leaves its rows as they are
        g["dstate0"] = _new(None, "dstate0", (B, W - 1, D), x.dtype, dev, cu is not None)
    call(_library().palimpsa_causal_conv_backward, (x, weight, bias, state0, dy, dstate_T, cu, *g.values()),
         _ptr(x), ld, _ptr(weight), _ptr(bias), _ptr(state0), _ptr(dy), ldy, _ptr(dstate_T), _ptr(g["dx"]),
         _ptr(g["dweight"]), _ptr(g["dbias"]), _ptr(g.get("dstate0")), _ptr(cu), B, T, longest, D, W,
         PALIMPSA_CONV_SILU if silu else 0, _dtype(x, "x"))
    return g


# ------------------------------------------------------------------ selective scan

def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, lead, dy=None):
    """Checks the scan's inputs; returns (channels, groups, states, strides or None)."""
    dev, kind, shape = x.device, x.dtype, tuple(x.shape)
    if A.dim() != 2 or B.dim() != lead + 2:
        raise ValueError(f"A must be [D, N] and B [..., G, N], got {tuple(A.shape)} and {tuple(B.shape)}")
    ch, n = A.shape
    groups = B.shape[-2]
    bc = shape[:-1] + (groups, n)
    ld = [_rows(x, "x", shape[:-1] + (ch,), kind, dev, lead), _rows(dt, "dt", shape, kind, dev, lead),
          _rows(B, "B", bc, kind, dev, lead), _rows(C, "C", bc, kind, dev, lead), _rows(z, "z", shape, kind, dev, lead),
          _rows(dy, "dy", shape, kind, dev, lead)]
    _check(A, "A", (ch, n), F32, dev)
    _check(D, "D", (ch,), F32, dev)
    _check(dt_bias, "dt_bias", (ch,), F32, dev)
    return ch, groups, n, ctypes.byref(_Strides(*ld)) if any(ld) else None


def palimpsa_selective_scan_checkpoint_shape(batch, tokens, channels, states, packed=False):
    """Shape of the checkpoints of a scan: one state per 16 tokens of every sequence
    (packed: rows // 16 + batch slots)."""
    if packed:
        return (tokens // CHECKPOINT_TOKENS + batch, channels, states)
    return (batch, -(-tokens // CHECKPOINT_TOKENS), channels, states)


def _scan(name, x, dt, A, B, C, D, z, dt_bias, h0, softplus, cu_seqlens, max_seqlen, y, h_T, want_ckpt, ckpt, stream):
    call = _Call(x, name, stream)
    dev = x.device
    nb, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, stream, name)
    ch, groups, n, strides = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, lead)
    _check(h0, "h0", (nb, ch, n), F32, dev)
    y = _new(y, "y", tuple(x.shape), x.dtype, dev, cu is not None)
    h_T = _new(h_T, "h_T", (nb, ch, n), F32, dev)
    if want_ckpt:
        ckpt = _new(ckpt, "ckpt", palimpsa_selective_scan_checkpoint_shape(nb, T, ch, n, cu is not None), F32, dev)
    call(_library().palimpsa_selective_scan, (x, dt, A, B, C, D, z, dt_bias, h0, y, h_T, ckpt, cu),
         _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(y), _ptr(h_T),
         _ptr(ckpt), strides, _ptr(cu), nb, T, longest, ch, groups, n, PALIMPSA_SCAN_SOFTPLUS if softplus else 0,
         _dtype(x, "x"))
    return y, h_T, ckpt


def palimpsa_selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, softplus=True, cu_seqlens=None,
                            max_seqlen=None, y=None, h_T=None, stream=None):
    """The selective scan (see palimpsa.h): s = softplus(dt + dt_bias), h = exp(-A s) h + s x B,
    y = (C h + D x) silu(z).

    x, dt, z [B, T, D] and B, C [B, T, G, N] (packed: [rows, D] and [rows, G, N] with
    cu_seqlens [B + 1] int32 and max_seqlen as for palimpsa_causal_conv), one dtype; A
    [D, N] > 0, D (the skip term), dt_bias [D], h0 [B, D, N] fp32; D, z, dt_bias, h0 may be
    None. Returns (y in x's dtype, h_T [B, D, N] fp32); h_T may be given as h0."""
    return _scan("palimpsa_selective_scan", x, dt, A, B, C, D, z, dt_bias, h0, softplus, cu_seqlens, max_seqlen, y, h_T,
                 False, None, stream)[:2]


def palimpsa_selective_scan_checkpointed(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, softplus=True,
                                         cu_seqlens=None, max_seqlen=None, ckpt=None, y=None, h_T=None, stream=None):
    """palimpsa_selective_scan for training: also the states that the backward reads. Returns
    (y, h_T, ckpt), ckpt of palimpsa_selective_scan_checkpoint_shape."""
    return _scan("palimpsa_selective_scan", x, dt, A, B, C, D, z, dt_bias, h0, softplus, cu_seqlens, max_seqlen, y, h_T,
                 True, ckpt, stream)


def palimpsa_selective_scan_backward(x, dt, A, B, C, D, z, dt_bias, h0, ckpt, dy, dh_T=None, *, softplus=True,
                                     cu_seqlens=None, max_seqlen=None, want_state_grad=True, stream=None):
    """Gradients through palimpsa_selective_scan_checkpointed (see palimpsa.h), with its ckpt on the
    same inputs. Returns a dict: dx, ddt, dz (with z), dB, dC in x's dtype; dA [D, N], dD
    (with D), ddt_bias (with dt_bias) fp32, and dh0 [B, D, N] fp32 when want_state_grad. Rows
    outside every sequence are zero."""
    name = "palimpsa_selective_scan_backward"
    call = _Call(x, name, stream)
    dev, kind = x.device, x.dtype
    nb, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, stream, name)
    ch, groups, n, strides = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, lead, dy)
    _check(h0, "h0", (nb, ch, n), F32, dev)
    _check(dh_T, "dh_T", (nb, ch, n), F32, dev)
    _check(ckpt, "ckpt", palimpsa_selective_scan_checkpoint_shape(nb, T, ch, n, cu is not None), F32, dev)
    packed = cu is not None
    g = {"dx": _new(None, "dx", tuple(x.shape), kind, dev, packed),
         "ddt": _new(None, "ddt", tuple(x.shape), kind, dev, packed),
         "dA": _new(None, "dA", (ch, n), F32, dev),
         "dB": _new(None, "dB", tuple(B.shape), kind, dev, packed),
         "dC": _new(None, "dC", tuple(B.shape), kind, dev, packed)}
    if D is not None:
        g["dD"] = _new(None, "dD", (ch,), F32, dev)
    if z is not None:
        g["dz"] = _new(None, "dz", tuple(x.shape), kind, dev, packed)
    if dt_bias is not None:
        g["ddt_bias"] = _new(None, "ddt_bias", (ch,), F32, dev)
    if want_state_grad:
        g["dh0"] = _new(None, "dh0", (nb, ch, n), F32, dev, packed)
    call(_library().palimpsa_selective_scan_backward,
         (x, dt, A, B, C, D, z, dt_bias, ckpt, dy, dh_T, cu, *g.values()),
         _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(ckpt), _ptr(dy),
         _ptr(dh_T), _ptr(g["dx"]), _ptr(g["ddt"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g.get("dD")),
         _ptr(g.get("dz")), _ptr(g.get("ddt_bias")), _ptr(g.get("dh0")), strides, _ptr(cu), nb, T, longest, ch, groups,
         n, PALIMPSA_SCAN_SOFTPLUS if softplus else 0, _dtype(x, "x"))
    return g


def palimpsa_selective_scan_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, softplus=True, y=None,
                                 stream=None):
    """One token of the selective scan (see palimpsa.h): x, dt, z [B, D], B and C [B, G, N], h
    [B, D, N] fp32 updated in place. Returns y [B, D]."""
    name = "palimpsa_selective_scan_step"
    call = _Call(x, name, stream)
    dev = x.device
    if x.dim() != 2:
        raise ValueError(f"{name}: x must be [B, D], got {tuple(x.shape)}")
    nb = x.shape[0]
    ch, groups, n, strides = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, 1)
    _check(h, "h", (nb, ch, n), F32, dev)
    y = _new(y, "y", (nb, ch), x.dtype, dev)
    call(_library().palimpsa_selective_scan_step, (x, dt, A, B, C, D, z, dt_bias, h, y),
         _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h), _ptr(y), strides, nb,
         ch, groups, n, PALIMPSA_SCAN_SOFTPLUS if softplus else 0, _dtype(x, "x"))
    return y
