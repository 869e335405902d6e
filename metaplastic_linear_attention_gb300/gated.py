"""Binding of the gated scan of ``libpalimpsa.so`` (``include/palimpsa.h``): a linear recurrence
with one state per channel and gates from the token, for prompts, packed batches, single
tokens and training. Conventions as in :mod:`.ssm`.
"""
from __future__ import annotations

import ctypes

import torch

from .ssm import F32, _batch, _call, _dense, _device, _dtype, _like, _new, _on_stream, _ptr, _rows

PALIMPSA_GATE_ZERO_ROWS, PALIMPSA_GATE_ZERO_STATES = 1, 2   # palimpsa_gate_flags
CHECKPOINT_TOKENS = 8


class _Strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_longlong) for n in ("x", "r", "i", "z", "dy")]


def _inputs(x, r, A, i, z, r_bias, i_bias, dev, lead, dy=None):
    """Checks the inputs; returns (channels, strides or None, the addresses of x, r, A, i, z, r_bias, i_bias)."""
    kind, shape = x.dtype, x.shape
    if i is None and i_bias is not None:
        raise ValueError("i_bias without i")
    ch = shape[-1]
    dense = x.is_contiguous()
    for t in (r, i, z, dy):
        if not (t is None or (t.dtype is kind and t.shape == shape and t.get_device() == dev and t.is_contiguous())):
            dense = False
    strides = None
    if not dense:
        strides = ctypes.byref(_Strides(*(_rows(t, name, shape, kind, dev, lead) for name, t in
                                          (("x", x), ("r", r), ("i", i), ("z", z), ("dy", dy)))))
    per = (ch,)
    return ch, strides, (x.data_ptr(), r.data_ptr(), _dense(A, "A", per, F32, dev), _ptr(i), _ptr(z),
                         _dense(r_bias, "r_bias", per, F32, dev), _dense(i_bias, "i_bias", per, F32, dev))


def palimpsa_gated_scan_checkpoint_shape(batch, tokens, channels, packed=False):
    """Shape of the checkpoints of a gated scan: one state per 8 tokens of every sequence
    (packed: rows // 8 + batch slots)."""
    if packed:
        return (tokens // CHECKPOINT_TOKENS + batch, channels)
    return (batch, -(-tokens // CHECKPOINT_TOKENS), channels)


def _scan(name, x, r, A, i, z, r_bias, i_bias, h0, cu_seqlens, max_seqlen, y, h_T, want_ckpt, ckpt):
    dev = _device(x, name)
    nb, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, name)
    ch, strides, ptrs = _inputs(x, r, A, i, z, r_bias, i_bias, dev, lead)
    kind = _dtype(x)
    p0 = _dense(h0, "h0", (nb, ch), F32, dev)
    fill = 0    # of a packed call's fresh outputs, what it leaves unwritten
    if y is None:
        y, fill = _like(x), PALIMPSA_GATE_ZERO_ROWS
    else:
        _dense(y, "y", x.shape, x.dtype, dev)
    if h_T is None:
        fill |= PALIMPSA_GATE_ZERO_STATES
    h_T = _new(h_T, "h_T", (nb, ch), F32, x)
    if want_ckpt:
        ckpt = _new(ckpt, "ckpt", palimpsa_gated_scan_checkpoint_shape(nb, T, ch, cu is not None), F32, x)
    _call(name, dev, *ptrs, p0, y.data_ptr(), h_T.data_ptr(), _ptr(ckpt), strides, _ptr(cu), nb, T, longest, ch, fill,
          kind)
    return y, h_T, ckpt


@_on_stream
def palimpsa_gated_scan(x, r, A, i=None, z=None, r_bias=None, i_bias=None, h0=None, *, cu_seqlens=None, max_seqlen=None,
                        y=None, h_T=None):
    """The gated scan (see palimpsa.h): a = exp(-A sigmoid(r + r_bias)),
    h = a h + sqrt(1 - a^2) sigmoid(i + i_bias) x, y = h silu(z).

    x, r, i, z [B, T, D] (packed: [rows, D] with cu_seqlens [B + 1] int32 and max_seqlen as for
    palimpsa_causal_conv), one dtype; A [D] > 0, r_bias, i_bias [D], h0 [B, D] fp32; i (no input
    gate), z, the biases and h0 may be None. Returns (y in x's dtype, h_T [B, D] fp32); h_T may be given as h0."""
    return _scan("palimpsa_gated_scan", x, r, A, i, z, r_bias, i_bias, h0, cu_seqlens, max_seqlen, y, h_T, False, None)[:2]


@_on_stream
def palimpsa_gated_scan_checkpointed(x, r, A, i=None, z=None, r_bias=None, i_bias=None, h0=None, *, cu_seqlens=None,
                                     max_seqlen=None, ckpt=None, y=None, h_T=None):
    """palimpsa_gated_scan for training: also the states that the backward reads. Returns
    (y, h_T, ckpt), ckpt of palimpsa_gated_scan_checkpoint_shape."""
    return _scan("palimpsa_gated_scan", x, r, A, i, z, r_bias, i_bias, h0, cu_seqlens, max_seqlen, y, h_T, True, ckpt)


@_on_stream
def palimpsa_gated_scan_backward(x, r, A, i, z, r_bias, i_bias, ckpt, dy, dh_T=None, *, cu_seqlens=None, max_seqlen=None,
                                 want_state_grad=True):
    """Gradients through palimpsa_gated_scan_checkpointed (see palimpsa.h), with its ckpt on the same
    inputs. Returns a dict: dx, dr, di (with i), dz (with z) in x's dtype; dA, dr_bias (always: the
    sum of dr over the tokens), di_bias (with i) [D] fp32, and dh0 [B, D] fp32 when
    want_state_grad. Rows outside every sequence are zero."""
    name = "palimpsa_gated_scan_backward"
    dev = _device(x, name)
    nb, T, longest, cu, lead = _batch(x, cu_seqlens, max_seqlen, dev, name)
    ch, strides, ptrs = _inputs(x, r, A, i, z, r_bias, i_bias, dev, lead, dy)
    kind = _dtype(x)
    pg = _dense(dh_T, "dh_T", (nb, ch), F32, dev)
    pc = _dense(ckpt, "ckpt", palimpsa_gated_scan_checkpoint_shape(nb, T, ch, cu is not None), F32, dev)
    g = {"dx": _like(x), "dr": _like(x), "dA": _like(A), "dr_bias": _like(A)}
    if i is not None:
        g["di"], g["di_bias"] = _like(x), _like(A)
    if z is not None:
        g["dz"] = _like(x)
    if want_state_grad:
        g["dh0"] = torch.empty((nb, ch), dtype=F32, device=x.device)
    at = {k: v.data_ptr() for k, v in g.items()}
    _call(name, dev, *ptrs, pc, dy.data_ptr(), pg, at["dx"], at["dr"], at["dA"], at.get("di"), at.get("dz"), at["dr_bias"],
          at.get("di_bias"), at.get("dh0"), strides, _ptr(cu), nb, T, longest, ch,
          PALIMPSA_GATE_ZERO_ROWS | PALIMPSA_GATE_ZERO_STATES, kind)
    return g


@_on_stream
def palimpsa_gated_scan_step(x, r, A, h, i=None, z=None, r_bias=None, i_bias=None, *, y=None):
    """One token of the gated scan (see palimpsa.h): x, r, i, z [B, D], h [B, D] fp32 updated in
    place. Returns y [B, D]."""
    name = "palimpsa_gated_scan_step"
    dev = _device(x, name)
    if x.dim() != 2:
        raise ValueError(f"{name}: x must be [B, D], got {tuple(x.shape)}")
    ch, strides, ptrs = _inputs(x, r, A, i, z, r_bias, i_bias, dev, 1)
    kind, nb = _dtype(x), x.shape[0]
    ph = _dense(h, "h", (nb, ch), F32, dev)
    if y is None:
        y = _like(x)
    else:
        _dense(y, "y", x.shape, x.dtype, dev)
    _call(name, dev, *ptrs, ph, y.data_ptr(), strides, nb, ch, kind)
    return y
