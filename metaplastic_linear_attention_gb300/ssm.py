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
import functools
import inspect

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
            "palimpsa_zero_rows_outside": [p, p, i, p, i, i, i, p],
            "palimpsa_zero_unwritten": [p, p, i, p, p, i, p, i, i, i, p],
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


_functions = {}


def _function(name):
    _functions[name] = getattr(_library(), name)
    return _functions[name]


# The checks below run on every decode token, so they are written for speed: a tensor that
# passes costs a few comparisons, and only a refusal looks at what is wrong.

def _dtype(x):
    if x.dtype is torch.bfloat16:
        return PALIMPSA_BF16
    if x.dtype is F32:
        return PALIMPSA_F32
    raise TypeError(f"token arrays must be bfloat16 or float32, got {x.dtype}")


def _dense(t, name, shape, dtype, dev):
    """The address of a contiguous tensor of that shape and dtype on CUDA device `dev`, or None of None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _check(t, name, shape, dtype, torch.device("cuda", dev))
    raise ValueError(f"{name}: expected a tensor of {shape} on cuda:{dev}")


def _rows(t, name, shape, dtype, dev, lead):
    """Checks a token array whose first `lead` dimensions count rows; returns its row stride in
    elements (0: dense)."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return 0
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected device {dev}")
    st, width = t.stride(), 1
    for k in range(len(shape) - 1, lead - 1, -1):
        if shape[k] != 1 and st[k] != width:
            raise ValueError(f"{name}: a row must be contiguous, got strides {st}")
        width *= shape[k]
    if lead == 1 or shape[1] == 1:
        ld = st[0] if shape[0] != 1 else width
    else:
        ld = st[1]
        if shape[0] != 1 and st[0] != shape[1] * ld:
            raise ValueError(f"{name}: rows must be evenly spaced, got strides {st}")
    if ld < width:
        raise ValueError(f"{name}: rows overlap, got strides {st}")
    return ld


def _ptr(t):
    return None if t is None else t.data_ptr()


def _device(x, name):
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name} takes device tensors")
    return dev


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(name, dev, *args):
    """The library call on the tensors' device, on its current stream."""
    fn = _functions.get(name) or _function(name)
    if dev == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev))
    if rc != 0:
        raise PalimpsaError(rc, name)


def _on_stream(fn):
    """Adds the argument `stream` to an operator: the stream to run on, instead of the current one,
    whose queued work it first waits for (as every call of this package does: the inputs are
    usually made there). The caller waits for it before using the results elsewhere.
    What the call allocates and fills in belongs to that stream, so that nothing queued later on
    the current one can touch it. The inputs are recorded there and fresh outputs on the current
    stream, so that the allocator keeps either until both streams are done with it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        given = [t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor) and t.is_cuda]
        for t in given:
            if t.get_device() != stream.device_index:
                raise ValueError(f"{fn.__name__}: a tensor is on {t.device}, the stream on cuda:{stream.device_index}")
        home = torch.cuda.current_stream(stream.device)
        if stream == home:
            return fn(*args, **kw)
        binding._stream_handle(stream)  # waits for the current stream
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        for t in given:
            t.record_stream(stream)
        for t in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
            if t is not None:
                t.record_stream(home)
        return out

    sig = inspect.signature(fn)
    extra = inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)
    call.__signature__ = sig.replace(parameters=(*sig.parameters.values(), extra))
    return call


def _batch(x, cu_seqlens, max_seqlen, dev, name):
    """(B, T, max_seqlen, offsets on the device, row dimensions) of a token array x."""
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError(f"{name}: x must be [B, T, D], got {tuple(x.shape)}")
        return x.shape[0], x.shape[1], x.shape[1], None, 2
    if x.dim() != 2:
        raise ValueError(f"{name}: packed x must be [rows, D], got {tuple(x.shape)}")
    cu, n, longest = _packed_offsets(cu_seqlens, max_seqlen, x.device)
    return n, x.shape[0], longest, cu, 1


def _new(t, name, shape, dtype, x):
    """An output on x's device: checked when given, else allocated."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=x.device)
    _dense(t, name, shape, dtype, x.get_device())
    return t


def _like(t):
    """An uninitialised contiguous tensor of t's shape, dtype and device."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _zero_unwritten(outs, states, cu, nb, rows, longest, dev):
    """Zeros in what a packed call leaves as it is of its freshly allocated outputs: the rows (of
    `outs`) that no sequence covers, and the rows and `states` of sequences that are skipped for their
    offsets. (Where offsets are out of order, everything.)"""
    if cu is None:
        return
    outs = outs if rows else ()
    arrays = lambda ts: (ctypes.c_void_p * len(ts))(*(t.data_ptr() for t in ts))  # noqa: E731
    widths = lambda ts, n: (ctypes.c_longlong * len(ts))(*(t.numel() // n * t.element_size() for t in ts))  # noqa: E731
    _call("palimpsa_zero_unwritten", dev, arrays(outs), widths(outs, rows), len(outs), arrays(states), widths(states, nb),
          len(states), cu.data_ptr(), nb, rows, longest)


def _zero_fresh(given, outs, cu, nb, rows, longest, dev):
    """_zero_unwritten for a forward's (y, state) of which only those that the caller did not give are fresh."""
    if cu is not None and (given[0] is None or given[1] is None):
        _zero_unwritten(outs[:1] if given[0] is None else (), outs[1:] if given[1] is None else (), cu, nb, rows, longest, dev)


# ------------------------------------------------------------------ causal convolution

def _conv_params(x, weight, bias, dev):
    D, W = x.shape[-1], weight.shape[-1]
    return D, W, _dense(weight, "weight", (D, W), F32, dev), _dense(bias, "bias", (D,), F32, dev)


@_on_stream
def palimpsa_causal_conv(x, weight, bias=None, state0=None, *, silu=True, cu_seqlens=None, max_seqlen=None, y=None,
                         state_T=None):
    """Depthwise causal convolution along the tokens (see palimpsa.h).

    x [B, T, D], or [rows, D] with cu_seqlens [B + 1] int32 (max_seqlen: the longest
    sequence, read from cu_seqlens when not given, which synchronises; what no sequence
    writes of outputs that are not given is zero); weight [D, W], bias [D] fp32; state0
    [B, W - 1, D]: the inputs before each sequence, or None for zeros. Returns (y, state_T), both in x's dtype; state_T may be given as state0."""
    name = "palimpsa_causal_conv"
    dev = _device(x, name)
    B, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, name)
    D, W, pw, pb = _conv_params(x, weight, bias, dev)
    kind = _dtype(x)
    ld = _rows(x, "x", x.shape, x.dtype, dev, lead)
    ps = _dense(state0, "state0", (B, W - 1, D), x.dtype, dev)
    given = y, state_T
    if y is None:
        y = _like(x)
    else:
        _dense(y, "y", x.shape, x.dtype, dev)
    state_T = _new(state_T, "state_T", (B, W - 1, D), x.dtype, x)
    _zero_fresh(given, (y, state_T), cu, B, T, longest, dev)
    _call(name, dev, x.data_ptr(), ld, pw, pb, ps, y.data_ptr(), state_T.data_ptr(), _ptr(cu), B, T, longest, D, W,
          PALIMPSA_CONV_SILU if silu else 0, kind)
    return y, state_T


@_on_stream
def palimpsa_causal_conv_step(x, weight, bias, state, *, silu=True, y=None):
    """One token of the convolution (see palimpsa.h): x [B, D], state [B, W - 1, D] updated in
    place. Returns y [B, D]."""
    name = "palimpsa_causal_conv_step"
    dev = _device(x, name)
    if x.dim() != 2:
        raise ValueError(f"{name}: x must be [B, D], got {tuple(x.shape)}")
    D, W, pw, pb = _conv_params(x, weight, bias, dev)
    B, kind = x.shape[0], _dtype(x)
    ld = _rows(x, "x", x.shape, x.dtype, dev, 1)
    ps = _dense(state, "state", (B, W - 1, D), x.dtype, dev)
    if y is None:
        y = _like(x)
    else:
        _dense(y, "y", x.shape, x.dtype, dev)
    _call(name, dev, x.data_ptr(), ld, pw, pb, ps, y.data_ptr(), B, D, W, PALIMPSA_CONV_SILU if silu else 0, kind)
    return y


@_on_stream
def palimpsa_causal_conv_backward(x, weight, bias, state0, dy, dstate_T=None, *, silu=True, cu_seqlens=None,
                                  max_seqlen=None, want_state_grad=True):
    """Gradients through palimpsa_causal_conv (see palimpsa.h). Returns a dict: dx (x's dtype; zero
    in rows outside every sequence), dweight [D, W], dbias [D] (fp32), and dstate0
    [B, W - 1, D] (x's dtype) when want_state_grad."""
    name = "palimpsa_causal_conv_backward"
    dev = _device(x, name)
    B, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, name)
    D, W, pw, pb = _conv_params(x, weight, bias, dev)
    kind, dtype = _dtype(x), x.dtype
    ld = _rows(x, "x", x.shape, dtype, dev, lead)
    ldy = _rows(dy, "dy", x.shape, dtype, dev, lead)
    ps = _dense(state0, "state0", (B, W - 1, D), dtype, dev)
    pd = _dense(dstate_T, "dstate_T", (B, W - 1, D), dtype, dev)
    g = {"dx": _like(x), "dweight": _like(weight), "dbias": torch.empty(D, dtype=F32, device=x.device)}
    if want_state_grad:
        g["dstate0"] = torch.empty((B, W - 1, D), dtype=dtype, device=x.device)
    _zero_unwritten((g["dx"],), (g["dstate0"],) if want_state_grad else (), cu, B, T, longest, dev)
    _call(name, dev, x.data_ptr(), ld, pw, pb, ps, dy.data_ptr(), ldy, pd, g["dx"].data_ptr(),
          g["dweight"].data_ptr(), g["dbias"].data_ptr(), _ptr(g.get("dstate0")), _ptr(cu), B, T, longest, D, W,
          PALIMPSA_CONV_SILU if silu else 0, kind)
    return g


# ------------------------------------------------------------------ selective scan

def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, dev, lead, dy=None):
    """Checks the scan's inputs; returns (channels, groups, states, strides or None, the addresses
    of x, dt, A, B, C, D, z, dt_bias)."""
    kind, shape = x.dtype, x.shape
    if A.dim() != 2 or B.dim() != lead + 2:
        raise ValueError(f"A must be [D, N] and B [..., G, N], got {tuple(A.shape)} and {tuple(B.shape)}")
    ch, n = A.shape
    groups = B.shape[-2]
    bc = shape[:-1] + (groups, n)
    if (shape[-1] == ch and x.is_contiguous()
            and dt.dtype is kind and dt.shape == shape and dt.get_device() == dev and dt.is_contiguous()
            and B.dtype is kind and B.shape == bc and B.get_device() == dev and B.is_contiguous()
            and C.dtype is kind and C.shape == bc and C.get_device() == dev and C.is_contiguous()
            and (z is None or (z.dtype is kind and z.shape == shape and z.get_device() == dev and z.is_contiguous()))
            and (dy is None or (dy.dtype is kind and dy.shape == shape and dy.get_device() == dev
                                and dy.is_contiguous()))):
        ld = None
    else:
        ld = (_rows(x, "x", shape[:-1] + (ch,), kind, dev, lead), _rows(dt, "dt", shape, kind, dev, lead),
              _rows(B, "B", bc, kind, dev, lead), _rows(C, "C", bc, kind, dev, lead),
              _rows(z, "z", shape, kind, dev, lead), _rows(dy, "dy", shape, kind, dev, lead))
    ptrs = (x.data_ptr(), dt.data_ptr(), _dense(A, "A", (ch, n), F32, dev), B.data_ptr(), C.data_ptr(),
            _dense(D, "D", (ch,), F32, dev), _ptr(z), _dense(dt_bias, "dt_bias", (ch,), F32, dev))
    return ch, groups, n, None if ld is None else ctypes.byref(_Strides(*ld)), ptrs


def palimpsa_selective_scan_checkpoint_shape(batch, tokens, channels, states, packed=False):
    """Shape of the checkpoints of a scan: one state per 16 tokens of every sequence
    (packed: rows // 16 + batch slots)."""
    if packed:
        return (tokens // CHECKPOINT_TOKENS + batch, channels, states)
    return (batch, -(-tokens // CHECKPOINT_TOKENS), channels, states)


def _scan(name, x, dt, A, B, C, D, z, dt_bias, h0, softplus, cu_seqlens, max_seqlen, y, h_T, want_ckpt, ckpt):
    dev = _device(x, name)
    nb, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, name)
    ch, groups, n, strides, ptrs = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, dev, lead)
    kind = _dtype(x)
    p0 = _dense(h0, "h0", (nb, ch, n), F32, dev)
    given = y, h_T
    if y is None:
        y = _like(x)
    else:
        _dense(y, "y", x.shape, x.dtype, dev)
    h_T = _new(h_T, "h_T", (nb, ch, n), F32, x)
    _zero_fresh(given, (y, h_T), cu, nb, T, longest, dev)
    if want_ckpt:
        ckpt = _new(ckpt, "ckpt", palimpsa_selective_scan_checkpoint_shape(nb, T, ch, n, cu is not None), F32, x)
    _call(name, dev, *ptrs, p0, y.data_ptr(), h_T.data_ptr(), _ptr(ckpt), strides, _ptr(cu), nb, T, longest, ch,
          groups, n, PALIMPSA_SCAN_SOFTPLUS if softplus else 0, kind)
    return y, h_T, ckpt


@_on_stream
def palimpsa_selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, softplus=True, cu_seqlens=None,
                            max_seqlen=None, y=None, h_T=None):
    """The selective scan (see palimpsa.h): s = softplus(dt + dt_bias), h = exp(-A s) h + s x B,
    y = (C h + D x) silu(z).

    x, dt, z [B, T, D] and B, C [B, T, G, N] (packed: [rows, D] and [rows, G, N] with
    cu_seqlens [B + 1] int32 and max_seqlen as for palimpsa_causal_conv), one dtype; A
    [D, N] > 0, D (the skip term), dt_bias [D], h0 [B, D, N] fp32; D, z, dt_bias, h0 may be
    None. Returns (y in x's dtype, h_T [B, D, N] fp32); h_T may be given as h0."""
    return _scan("palimpsa_selective_scan", x, dt, A, B, C, D, z, dt_bias, h0, softplus, cu_seqlens, max_seqlen, y, h_T,
                 False, None)[:2]


@_on_stream
def palimpsa_selective_scan_checkpointed(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, softplus=True,
                                         cu_seqlens=None, max_seqlen=None, ckpt=None, y=None, h_T=None):
    """palimpsa_selective_scan for training: also the states that the backward reads. Returns
    (y, h_T, ckpt), ckpt of palimpsa_selective_scan_checkpoint_shape."""
    return _scan("palimpsa_selective_scan", x, dt, A, B, C, D, z, dt_bias, h0, softplus, cu_seqlens, max_seqlen, y, h_T,
                 True, ckpt)


@_on_stream
def palimpsa_selective_scan_backward(x, dt, A, B, C, D, z, dt_bias, h0, ckpt, dy, dh_T=None, *, softplus=True,
                                     cu_seqlens=None, max_seqlen=None, want_state_grad=True):
    """Gradients through palimpsa_selective_scan_checkpointed (see palimpsa.h), with its ckpt on the
    same inputs. Returns a dict: dx, ddt, dz (with z), dB, dC in x's dtype; dA [D, N], dD
    (with D), ddt_bias (with dt_bias) fp32, and dh0 [B, D, N] fp32 when want_state_grad. Rows
    outside every sequence are zero."""
    name = "palimpsa_selective_scan_backward"
    dev = _device(x, name)
    nb, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, name)
    ch, groups, n, strides, ptrs = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, dev, lead, dy)
    kind, dtype, packed = _dtype(x), x.dtype, cu is not None
    _dense(h0, "h0", (nb, ch, n), F32, dev)
    pg = _dense(dh_T, "dh_T", (nb, ch, n), F32, dev)
    pc = _dense(ckpt, "ckpt", palimpsa_selective_scan_checkpoint_shape(nb, T, ch, n, packed), F32, dev)
    g = {"dx": _like(x), "ddt": _like(x), "dA": _like(A), "dB": _like(B), "dC": _like(B)}
    if D is not None:
        g["dD"] = _like(D)
    if z is not None:
        g["dz"] = _like(x)
    if dt_bias is not None:
        g["ddt_bias"] = _like(dt_bias)
    if want_state_grad:
        g["dh0"] = torch.empty((nb, ch, n), dtype=F32, device=x.device)
    _zero_unwritten([g[k] for k in ("dx", "ddt", "dz", "dB", "dC") if k in g], (g["dh0"],) if want_state_grad else (), cu,
                    nb, T, longest, dev)
    at = {k: v.data_ptr() for k, v in g.items()}
    _call(name, dev, *ptrs, pc, dy.data_ptr(), pg, at["dx"], at["ddt"], at["dA"], at["dB"], at["dC"], at.get("dD"),
          at.get("dz"), at.get("ddt_bias"), at.get("dh0"), strides, _ptr(cu), nb, T, longest, ch, groups, n,
          PALIMPSA_SCAN_SOFTPLUS if softplus else 0, kind)
    return g


@_on_stream
def palimpsa_selective_scan_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, softplus=True, y=None):
    """One token of the selective scan (see palimpsa.h): x, dt, z [B, D], B and C [B, G, N], h
    [B, D, N] fp32 updated in place. Returns y [B, D]."""
    name = "palimpsa_selective_scan_step"
    dev = _device(x, name)
    if x.dim() != 2:
        raise ValueError(f"{name}: x must be [B, D], got {tuple(x.shape)}")
    ch, groups, n, strides, ptrs = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, dev, 1)
    kind, nb = _dtype(x), x.shape[0]
    ph = _dense(h, "h", (nb, ch, n), F32, dev)
    if y is None:
        y = _like(x)
    else:
        _dense(y, "y", x.shape, x.dtype, dev)
    _call(name, dev, *ptrs, ph, y.data_ptr(), strides, nb, ch, groups, n,
          PALIMPSA_SCAN_SOFTPLUS if softplus else 0, kind)
    return y
