"""ORACLE — test infrastructure only (see ``oracle/__init__``).

Plain fp64 statements of the state-space operators and the layer norm, one sequence and one token at a
time, in torch so that torch.autograd (a library routine) differentiates them exactly. They
share no code with the CUDA library.

* ``conv``: u_t = bias + sum_j w_j x_{t-(W-1)+j}, y = silu(u) (or u), the inputs before the
  first token taken from the state.
* ``scan``: s = softplus(dt + dt_bias) (or dt + dt_bias), h_t = exp(-A s_t) h_{t-1} +
  s_t x_t B_t, y_t = (C_t h_t + D x_t) silu(z_t), every channel reading the B and C of its
  group.
* ``gate``: a_t = exp(-A sigmoid(r_t + r_bias)), h_t = a_t h_{t-1} + sqrt(1 - a_t^2)
  sigmoid(i_t + i_bias) x_t, y_t = h_t silu(z_t).
* ``layer_norm``: s = x + residual as it is stored, y = (s - mean) / sqrt(variance + eps) weight + bias.

Token arrays are [rows, ...]; ``cu`` gives the sequences' row ranges. Rows outside every
sequence come back as zeros.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def conv(x, weight, bias, state0, cu, silu=True):
    """x [rows, D], weight [D, W], bias [D] or None, state0 [n, W-1, D] or None ->
    (y [rows, D], state_T [n, W-1, D])."""
    D, W = weight.shape
    ys, lasts, at = [], [], 0
    for n in range(len(cu) - 1):
        s0, s1 = int(cu[n]), int(cu[n + 1])
        ys.append(torch.zeros(s0 - at, D, dtype=F64))
        at = s1
        old = [torch.zeros(D, dtype=F64)] * (W - 1) if state0 is None else [state0[n, j] for j in range(W - 1)]
        rows = []
        for t in range(s0, s1):
            taps = old + [x[t]]
            u = sum(weight[:, j] * taps[j] for j in range(W))
            u = u if bias is None else u + bias
            rows.append(u * torch.sigmoid(u) if silu else u)
            old = taps[1:]
        ys.append(torch.stack(rows) if rows else torch.zeros(0, D, dtype=F64))
        lasts.append(torch.stack(old))
    ys.append(torch.zeros(x.shape[0] - at, D, dtype=F64))
    return torch.cat(ys), torch.stack(lasts)


def scan(x, dt, A, B, C, D, z, dt_bias, h0, cu, softplus=True):
    """x, dt, z [rows, ch], B, C [rows, G, N], A [ch, N], D, dt_bias [ch], h0 [n, ch, N]
    (D, z, dt_bias, h0 may be None) -> (y [rows, ch], h_T [n, ch, N])."""
    ch, N = A.shape
    per = ch // B.shape[1]
    ys, lasts, at = [], [], 0
    for n in range(len(cu) - 1):
        s0, s1 = int(cu[n]), int(cu[n + 1])
        ys.append(torch.zeros(s0 - at, ch, dtype=F64))
        at = s1
        h = torch.zeros(ch, N, dtype=F64) if h0 is None else h0[n]
        rows = []
        for t in range(s0, s1):
            raw = dt[t] if dt_bias is None else dt[t] + dt_bias
            s = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
            b, c = (m[t].repeat_interleave(per, 0) for m in (B, C))
            h = torch.exp(-A * s[:, None]) * h + (s * x[t])[:, None] * b
            y = (c * h).sum(-1)
            y = y if D is None else y + D * x[t]
            rows.append(y if z is None else y * z[t] * torch.sigmoid(z[t]))
        ys.append(torch.stack(rows) if rows else torch.zeros(0, ch, dtype=F64))
        lasts.append(h)
    ys.append(torch.zeros(x.shape[0] - at, ch, dtype=F64))
    return torch.cat(ys), torch.stack(lasts)


def gate(x, r, A, i, z, r_bias, i_bias, h0, cu):
    """x, r, i, z [rows, D], A, r_bias, i_bias [D], h0 [n, D] (i, z, r_bias, i_bias, h0 may be None)
    -> (y [rows, D], h_T [n, D])."""
    D = x.shape[1]
    ys, lasts, at = [], [], 0
    for n in range(len(cu) - 1):
        s0, s1 = int(cu[n]), int(cu[n + 1])
        ys.append(torch.zeros(s0 - at, D, dtype=F64))
        at = s1
        h = torch.zeros(D, dtype=F64) if h0 is None else h0[n]
        rows = []
        for t in range(s0, s1):
            rate = A * torch.sigmoid(r[t] if r_bias is None else r[t] + r_bias)
            u = torch.sqrt(-torch.expm1(-2 * rate)) * x[t]
            if i is not None:
                u = u * torch.sigmoid(i[t] if i_bias is None else i[t] + i_bias)
            h = torch.exp(-rate) * h + u
            rows.append(h if z is None else h * z[t] * torch.sigmoid(z[t]))
        ys.append(torch.stack(rows) if rows else torch.zeros(0, D, dtype=F64))
        lasts.append(h)
    ys.append(torch.zeros(x.shape[0] - at, D, dtype=F64))
    return torch.cat(ys), torch.stack(lasts)


def layer_norm(s, weight, bias, eps):
    """s [rows, D] (the sum as it is stored), weight, bias [D] or None -> y [rows, D]."""
    rows = []
    for v in s:
        mean = v.sum() / v.numel()
        t = (v - mean) / torch.sqrt(((v - mean) ** 2).sum() / v.numel() + eps)
        t = t if weight is None else t * weight
        rows.append(t if bias is None else t + bias)
    return torch.stack(rows) if rows else torch.zeros_like(s)


def gradients(fn, inputs, dy, dlast, cu, **kw):
    """Values and gradients of fn(*inputs, cu): `inputs` an ordered dict of fp64 tensors or None.
    Returns (y, last, {name: gradient of <dy, y> + <dlast, last>})."""
    leaves = {k: None if v is None else v.detach().clone().requires_grad_() for k, v in inputs.items()}
    y, last = fn(*leaves.values(), cu, **kw)
    loss = (y * dy).sum()
    if dlast is not None:
        loss = loss + (last * dlast).sum()
    names = [k for k, v in leaves.items() if v is not None]
    got = (torch.autograd.grad(loss, [leaves[k] for k in names], allow_unused=True) if loss.requires_grad
           else [None] * len(names))
    grads = {k: torch.zeros_like(leaves[k]) if g is None else g for k, g in zip(names, got)}
    return y.detach(), last.detach(), grads
