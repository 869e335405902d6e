"""Binding of the layer norm of ``libpalimpsa.so`` (``include/palimpsa.h``), with the addition
in front of it and its backward. Conventions as in :mod:`.ssm`.
"""
from __future__ import annotations

import torch

from .ssm import F32, _call, _dense, _device, _dtype, _like, _new, _on_stream, _ptr, _rows


def _token_rows(t, name, like, dev):
    """Checks a row array of like's shape and dtype; returns its row stride in elements (0: dense)."""
    shape, kind = like.shape, like.dtype
    if t is None or (t.dtype is kind and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return 0
    if t.shape == shape and t.dim() > 3:
        raise ValueError(f"{name}: rows of more than three dimensions must be contiguous, got strides {t.stride()}")
    return _rows(t, name, shape, kind, dev, max(1, len(shape) - 1))


def _shape(x, name):
    if x.dim() < 2:
        raise ValueError(f"{name}: rows of D values expected, got {tuple(x.shape)}")
    D = x.shape[-1]
    return x.shape[:-1].numel(), D


@_on_stream
def palimpsa_layer_norm(x, weight=None, bias=None, residual=None, *, eps=1e-5, want_stats=False, y=None, s=None,
                        stats=None):
    """Layer norm of rows, after an addition (see palimpsa.h): s = x + residual (rounded to x's dtype),
    y = (s - mean) / sqrt(variance + eps) weight + bias over the last dimension.

    x, residual [..., D], one dtype (up to three dimensions they may be slices of wider rows); weight,
    bias [D] fp32. Returns (y, s, stats): s is x itself without a residual, stats [..., 2] fp32
    (mean, 1 / deviation; for the backward) or None unless want_stats. s may be given as residual
    or x, which then receives the sum."""
    name = "palimpsa_layer_norm"
    dev = _device(x, name)
    rows, D = _shape(x, name)
    kind = _dtype(x)
    ldx, ldr = _token_rows(x, "x", x, dev), _token_rows(residual, "residual", x, dev)
    pw, pb = _dense(weight, "weight", (D,), F32, dev), _dense(bias, "bias", (D,), F32, dev)
    if y is None:
        y = _like(x)
    else:
        _dense(y, "y", x.shape, x.dtype, dev)
    if residual is None:
        if s is not None:
            raise ValueError("s without residual: the rows are x itself")
        s, ps = x, None
    else:
        if s is None:
            s = _like(x)
        else:
            _dense(s, "s", x.shape, x.dtype, dev)
        ps = s.data_ptr()
    if want_stats:
        stats = _new(stats, "stats", (*x.shape[:-1], 2), F32, x)
    elif stats is not None:
        raise ValueError("stats without want_stats")
    _call(name, dev, x.data_ptr(), ldx, _ptr(residual), ldr, pw, pb, y.data_ptr(), ps, _ptr(stats), rows, D, eps, kind)
    return y, s, stats


@_on_stream
def palimpsa_layer_norm_backward(s, weight, stats, dy, ds=None, *, want_weight_grad=True, want_bias_grad=True, dx=None):
    """Gradients through palimpsa_layer_norm (see palimpsa.h) from dy and, where s is used past the norm, ds, with
    the s and stats that the forward returned. Returns a dict: dx in s's dtype (the gradient of x and
    of residual alike), dweight [D] (with weight, when want_weight_grad) and dbias [D] (when
    want_bias_grad) fp32. dx may be given as dy or ds."""
    name = "palimpsa_layer_norm_backward"
    dev = _device(s, name)
    rows, D = _shape(s, name)
    kind = _dtype(s)
    lds, ldy, ldd = _token_rows(s, "s", s, dev), _token_rows(dy, "dy", s, dev), _token_rows(ds, "ds", s, dev)
    pw, pst = _dense(weight, "weight", (D,), F32, dev), _dense(stats, "stats", (*s.shape[:-1], 2), F32, dev)
    if dx is None:
        dx = _like(s)
    else:
        _dense(dx, "dx", s.shape, s.dtype, dev)
    g = {"dx": dx}
    if weight is not None and want_weight_grad:
        g["dweight"] = _like(weight)
    if want_bias_grad:
        g["dbias"] = torch.empty(D, dtype=F32, device=s.device)
    _call(name, dev, s.data_ptr(), lds, pw, pst, dy.data_ptr(), ldy, _ptr(ds), ldd, dx.data_ptr(), _ptr(g.get("dweight")),
          _ptr(g.get("dbias")), rows, D, kind)
    return g
