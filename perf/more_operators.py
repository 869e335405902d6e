"""Cases of the gated scan (a linear recurrence with one state per channel: a prompt, a
packed batch, one token, training) and of the layer norm with its residual addition
(forward, training), with their plain forms.

With ``own`` false, ``run`` computes an operator from elementary torch operations in 32
bits (64 where 32 lose what matters); with ``own`` true it makes the calls a user of
``metaplastic_linear_attention_gb300`` makes.
"""
import math

import torch

own = False

DEV = "cuda"
F32, F64 = torch.float32, torch.float64
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One layer's recurrence at the 760M layer's sizes (24 heads of 64 values, 8 x 4096 tokens).
        dict(name="gate_layer", op="gate", batch=8, tokens=4096, width=1536, type="bf16", input=True, gate=False,
             state=False),
        # One long context: few channels, so the sequence itself has to be shared out (32 heads of 64 values).
        dict(name="gate_long", op="gate", batch=1, tokens=32768, width=2048, type="bf16", input=True, gate=True,
             state=True),
        # A serving prefill: 24 prompts of different lengths in one call, continued from their states.
        dict(name="gate_packed", op="gate_packed", batch=24, tokens=32768, width=2048, type="bf16", input=True,
             gate=True, state=True),
        # A training step of the small layer (16 heads of 64 values): forward with checkpoints, then the gradients.
        dict(name="gate_train", op="gate_train", batch=4, tokens=2048, width=1024, type="bf16", input=True, gate=True,
             state=False),
        # A packed training step in 32 bits with odd sizes: a small experiment.
        dict(name="gate_train_packed", op="gate_train_packed", batch=5, tokens=3003, width=520, type="f32", input=True,
             gate=False, state=True),
        # One decode token for the decode job's batch (256 sequences, 32 heads of 64 values).
        dict(name="gate_token", op="gate_token", batch=256, tokens=1, width=2048, type="bf16", input=True, gate=True,
             state=True),
        # One decode token of one sequence: latency alone.
        dict(name="gate_token_one", op="gate_token", batch=1, tokens=1, width=1024, type="bf16", input=True, gate=True,
             state=True),
        # The norm between two layers of the 760M model: the mixer's output joins the residual stream.
        dict(name="norm_layer", op="norm", rows=32768, width=1536, type="bf16", residual=True, affine=True),
        # A norm over each head's 64 values of the recurrence's fp32 output (4 x 16 heads x 2048 tokens).
        dict(name="norm_heads", op="norm", rows=131072, width=64, type="f32", residual=False, affine=True),
        # The layer's norm in a training step: forward, then the gradients with the residual stream's.
        dict(name="norm_train", op="norm_train", rows=32768, width=1536, type="bf16", residual=True, affine=True),
        # The same in 32 bits with odd sizes.
        dict(name="norm_train_odd", op="norm_train", rows=1001, width=520, type="f32", residual=False, affine=True),
        # The norm of a decode step.
        dict(name="norm_token", op="norm", rows=256, width=2048, type="bf16", residual=True, affine=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate_packed", "gate_train", "gate_train_packed", "gate_token", "norm", "norm", "norm_train"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    cells = 32 << 20 if kind == "bf16" else 16 << 20  # channel-tokens, at most
    if op.startswith("norm"):
        width = 8 * _log(rng, 4, 1024)
        return dict(op=op, rows=_log(rng, 1, min(131072, cells // width)), width=width, type=kind,
                    residual=rng.random() < 0.6, affine=rng.random() < 0.8)
    width = 8 * _log(rng, 4, 512)
    batch, tokens = _log(rng, 1, 256 if op == "gate_token" else 24), 1
    if op in ("gate", "gate_train"):
        longest = 32768 if op == "gate" else 8192
        tokens = _log(rng, 1, max(1, min(longest, cells // (width * batch))))
    elif op != "gate_token":
        tokens = _log(rng, batch, max(batch, min(32768 if op == "gate_packed" else 8192, cells // width)))
    return dict(op=op, batch=batch, tokens=tokens, width=width, type=kind, input=rng.random() < 0.8,
                gate=rng.random() < 0.5, state=bool(op == "gate_token" or rng.random() < 0.5))


def _lengths(total, n, seed):
    """n ragged lengths that sum to `total`, each at least 1 where there are tokens enough."""
    g = torch.Generator().manual_seed(seed * 37 + 11)
    w = 0.05 + torch.rand((n,), generator=g, dtype=F64)
    if total < n:
        return [1] * total + [0] * (n - total)
    got = ((w / w.sum() * (total - n)).floor().to(torch.int64) + 1).tolist()
    got[-1] += total - sum(got)
    return got


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1013 + 29)
    kind = torch.bfloat16 if case["type"] == "bf16" else F32
    op, w = case["op"], case["width"]
    train, packed, token = "train" in op, "packed" in op, "token" in op

    def randn(*shape, scale=1.0, dtype=kind):
        return (scale * torch.randn(shape, generator=g, device=DEV, dtype=F32)).to(dtype)

    s = dict(case=dict(case))
    if op.startswith("norm"):
        # A residual stream some layers deep: larger than a layer's output, its channels off centre.
        rows = case["rows"]
        s["x"] = randn(rows, w)
        s["residual"] = (randn(rows, w, scale=3.0, dtype=F32) + randn(w, dtype=F32)).to(kind) if case["residual"] else None
        s["weight"] = 1 + randn(w, scale=0.1, dtype=F32) if case["affine"] else None
        s["bias"] = randn(w, scale=0.1, dtype=F32) if case["affine"] else None
        if train:
            s["dy"] = randn(rows, w)
            s["ds"] = randn(rows, w) if case["residual"] else None
        return s
    nb, t = case["batch"], case["tokens"]
    rows = (t,) if packed else (nb,) if token else (nb, t)
    s["cu"] = s["longest"] = None
    if packed:
        ls = _lengths(t, nb, int(seed) % 1000)
        cu = [0]
        for n in ls:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["longest"] = max(ls)
    s["x"] = randn(*rows, w)
    s["r"] = randn(*rows, w)
    # Rates log-uniform over [0.002, 2]: memories of half a token to a thousand.
    s["A"] = torch.exp(math.log(2e-3) + math.log(1e3) * torch.rand((w,), generator=g, device=DEV, dtype=F32))
    s["r_bias"] = randn(w, scale=0.5, dtype=F32)
    s["i"] = randn(*rows, w) if case["input"] else None
    s["i_bias"] = randn(w, scale=0.5, dtype=F32) if case["input"] else None
    s["z"] = randn(*rows, w) if case["gate"] else None
    s["h"] = randn(nb, w, scale=0.5, dtype=F32) if case["state"] else None
    if train:
        s["dy"] = randn(*rows, w)
    return s


# ------------------------------------------------------------------ the framework's calls

def _own_run(s):
    import metaplastic_linear_attention_gb300 as pal
    op = s["case"]["op"]
    if op.startswith("norm"):
        train = op == "norm_train"
        y, total, stats = pal.palimpsa_layer_norm(s["x"], s["weight"], s["bias"], s["residual"], eps=EPS,
                                                  want_stats=train)
        out = dict(y=y)
        if s["residual"] is not None:
            out["s"] = total
        if train:
            out.update(pal.palimpsa_layer_norm_backward(total, s["weight"], stats, s["dy"], s["ds"],
                                                        want_bias_grad=s["bias"] is not None))
        return out
    a = (s["x"], s["r"], s["A"])
    rest = (s["i"], s["z"], s["r_bias"], s["i_bias"])
    if op == "gate_token":
        return dict(y=pal.palimpsa_gated_scan_step(*a, s["h"], *rest), h_T=s["h"])
    kw = {} if s["cu"] is None else dict(cu_seqlens=s["cu"], max_seqlen=s["longest"])
    if "train" not in op:
        y, h = pal.palimpsa_gated_scan(*a, *rest, s["h"], **kw)
        return dict(y=y, h_T=h)
    y, h, ckpt = pal.palimpsa_gated_scan_checkpointed(*a, *rest, s["h"], **kw)
    g = pal.palimpsa_gated_scan_backward(*a, *rest, ckpt, s["dy"], want_state_grad=s["h"] is not None, **kw)
    return dict(g, y=y, h_T=h)


# ------------------------------------------------------------------ the plain forms

def _sigmoid(u):
    return 1 / (1 + torch.exp(-u))


def _norm(s):
    kind = s["x"].dtype
    total = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(kind)
    x = total.float()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS)
    hat = (x - mean) * rstd
    y = hat if s["weight"] is None else hat * s["weight"] + s["bias"]
    out = dict(y=y.to(kind))
    if s["residual"] is not None:
        out["s"] = total
    if s["case"]["op"] != "norm_train":
        return out
    dy = s["dy"].float()
    dhat = dy if s["weight"] is None else dy * s["weight"]
    dx = rstd * (dhat - dhat.mean(-1, keepdim=True) - hat * (dhat * hat).mean(-1, keepdim=True))
    out["dx"] = (dx if s["ds"] is None else dx + s["ds"].float()).to(kind)
    if s["weight"] is not None:
        out["dweight"] = (dy * hat).sum(0)
        out["dbias"] = dy.sum(0)
    return out


def _places(s):
    """(offsets, place of each token in its sequence, tokens behind it in its sequence, longest sequence)."""
    if s["cu"] is None:
        t = s["x"].shape[1]
        pos = torch.arange(t, device=DEV)
        return None, pos, pos.flip(0), t
    cu = s["cu"].long()
    t = torch.arange(s["x"].shape[0], device=DEV)
    q = torch.searchsorted(cu, t, right=True) - 1
    return cu, t - cu[q], cu[q + 1] - 1 - t, s["longest"]


def _doubled(h, total, pos, longest, forward):
    """h_t + the decayed h of the earlier (with forward false, the later) tokens of its sequence, by doubling: h [.., T, D],
    total [.., T, D] the running sum of the rates in 64 bits, pos [T] the tokens before (behind) each in its sequence."""
    axis, step = h.dim() - 2, 1
    while step < longest:
        m = h.shape[axis] - step
        gap = (total.narrow(axis, step, m) - total.narrow(axis, 0, m)).float()
        near, far = (step, 0) if forward else (0, step)
        add = torch.exp(-gap) * h.narrow(axis, far, m) * (pos >= step).narrow(0, near, m)[:, None]
        h = torch.cat([h.narrow(axis, 0, step), h.narrow(axis, step, m) + add] if forward
                      else [h.narrow(axis, 0, m) + add, h.narrow(axis, m, step)], axis)
        step *= 2
    return h


def _gates(s):
    """(sigmoid of r, rate, decay, norm sqrt(1 - decay^2), sigmoid of i or 1, x) in 32 bits."""
    sr = _sigmoid(s["r"].float() + s["r_bias"])
    rate = s["A"] * sr
    p = _sigmoid(s["i"].float() + s["i_bias"]) if s["i"] is not None else 1.0
    return sr, rate, torch.exp(-rate), torch.sqrt(-torch.expm1(-2 * rate)), p, s["x"].float()


def _scan(s):
    op, kind = s["case"]["op"], s["x"].dtype
    sr, rate, decay, norm, p, x = _gates(s)
    sz = _sigmoid(s["z"].float()) if s["z"] is not None else None
    gate = s["z"].float() * sz if s["z"] is not None else None
    b = norm * p * x
    if op == "gate_token":
        h = decay * s["h"] + b
        s["h"].copy_(h)
        return dict(y=(h if gate is None else h * gate).to(kind), h_T=s["h"])
    cu, pos, back, longest = _places(s)
    total = torch.cumsum(rate.double(), dim=-2)
    nb, w = s["case"]["batch"], x.shape[-1]
    h0 = s["h"] if s["h"] is not None else torch.zeros((nb, w), device=DEV)
    if cu is None:
        b[:, 0] += decay[:, 0] * h0
    else:
        some = (cu[1:] > cu[:-1]).nonzero()[:, 0]
        b[cu[some]] += decay[cu[some]] * h0[some]
    h = _doubled(b, total, pos, longest, True)
    if cu is None:
        last = h[:, -1].contiguous()
    else:
        last = h0.clone()
        last[some] = h[cu[some + 1] - 1]
    out = dict(y=(h if gate is None else h * gate).to(kind), h_T=last)
    if "train" not in op:
        return out
    # gradients: g_t = dy_t silu(z_t) + decay_{t+1} g_{t+1}
    dy = s["dy"].float()
    # (the running sum up to the token: from t to a later u the gradient decays by the rates of t + 1 .. u)
    g = _doubled(dy if gate is None else dy * gate, total, back, longest, False)
    before = torch.cat([torch.zeros_like(h[..., :1, :]), h[..., :-1, :]], -2)
    if cu is None:
        before[:, 0] = h0
    else:
        before[cu[some]] = h0[some]
    keep = 1.0 / norm
    drate = g * (p * x * (decay * decay) * keep - decay * before)
    draw_ = drate * rate * (1 - sr)
    lead = tuple(range(x.dim() - 1))
    out.update(dx=(g * norm * p).to(kind), dr=draw_.to(kind), dA=(drate * sr).sum(lead), dr_bias=draw_.sum(lead))
    if s["i"] is not None:
        di = g * norm * x * p * (1 - p)
        out.update(di=di.to(kind), di_bias=di.sum(lead))
    if gate is not None:
        out["dz"] = (dy * h * sz * (1 + s["z"].float() * (1 - sz))).to(kind)
    if s["h"] is not None:
        if cu is None:
            out["dh0"] = decay[:, 0] * g[:, 0]
        else:
            out["dh0"] = torch.zeros_like(h0)
            out["dh0"][some] = decay[cu[some]] * g[cu[some]]
    return out


def run(state):
    if own:
        return _own_run(state)
    return _norm(state) if state["case"]["op"].startswith("norm") else _scan(state)


# ------------------------------------------------------------------ work

def work(case):
    e = 2 if case["type"] == "bf16" else 4
    op, w = case["op"], case["width"]
    train = "train" in op
    if op.startswith("norm"):
        cells, extra = case["rows"] * w, 2 if case["residual"] else 0
        params = 2 * w * 4 if case["affine"] else 0
        moved, flops = cells * e * (2 + extra) + params, cells * (7 + extra / 2)
        if train:  # dy (and the residual stream's gradient) in, dx out, the parameters' gradients
            moved += cells * e * (2 + extra / 2) + params
            flops += cells * 12
        return dict(bytes=int(moved), flops=int(flops))
    nb = case["batch"]
    cells = (case["tokens"] if "packed" in op else nb * case["tokens"]) * w
    i, z = int(case["input"]), int(case["gate"])
    # The parameters once, the states in and out, x, r, i, z in, y out.
    moved = cells * e * (3 + i + z) + w * 4 * (2 + i) + nb * w * 4 * (2 if case["state"] else 1)
    flops = cells * (12 + 6 * i + 6 * z)
    if train:  # dy in; dx, dr, di, dz and the gradients of the parameters and the first state out
        moved += cells * e * (3 + i + z) + w * 4 * (2 + i) + (nb * w * 4 if case["state"] else 0)
        flops += cells * (24 + 8 * i + 10 * z)
    return dict(bytes=moved, flops=flops)


# ------------------------------------------------------------------ 64 bits, token by token

def _exact_norm(s):
    kind = s["x"].dtype
    x = s["x"].to(F64)
    if s["residual"] is not None:  # the rows that are normalised are the sum as it is stored
        x = (x + s["residual"].to(F64)).to(kind).to(F64)
    n = x.shape[1]
    centred = x - (x.sum(1) / n)[:, None]
    sd = torch.sqrt((centred * centred).sum(1) / n + EPS)[:, None]
    hat = centred / sd
    wt = torch.ones(n, dtype=F64, device=DEV) if s["weight"] is None else s["weight"].to(F64)
    y = hat * wt
    out = dict(y=y if s["bias"] is None else y + s["bias"].to(F64))
    if s["residual"] is not None:
        out["s"] = x
    if s["case"]["op"] != "norm_train":
        return out
    dy = s["dy"].to(F64)
    u = dy * wt
    c1, c2 = u.sum(1) / n, (u * hat).sum(1) / n
    dx = (u - c1[:, None] - c2[:, None] * hat) / sd
    out["dx"] = dx if s["ds"] is None else dx + s["ds"].to(F64)
    if s["weight"] is not None:
        out["dweight"], out["dbias"] = torch.einsum("rd,rd->d", dy, hat), dy.sum(0)
    return out


def _exact_scan(s):
    """The recurrence in 64 bits, one token after the other; a packed batch's sequences side by side, the longest first."""
    op = s["case"]["op"]
    up = lambda m: None if m is None else m.to(F64)  # noqa: E731
    x, r = up(s["x"]), up(s["r"]) + up(s["r_bias"])
    i = up(s["i"]) + up(s["i_bias"]) if s["i"] is not None else None
    z, A, dy = up(s["z"]), up(s["A"]), up(s.get("dy"))
    nb, w = s["case"]["batch"], s["case"]["width"]
    h = up(s["h"]) if s["h"] is not None else torch.zeros((nb, w), dtype=F64, device=DEV)
    h = h.clone()
    if op == "gate_token":
        first, lens = list(range(nb)), [1] * nb
    elif s["cu"] is not None:
        cu = s["cu"].tolist()
        first, lens = cu[:-1], [cu[k + 1] - cu[k] for k in range(nb)]
    else:
        t = x.shape[1]
        first, lens = [k * t for k in range(nb)], [t] * nb
    flat = lambda m: None if m is None else m.reshape(-1, w)  # noqa: E731
    fx, fr, fi, fz, fdy = flat(x), flat(r), flat(i), flat(z), flat(dy)
    order = sorted(range(nb), key=lambda k: -lens[k])
    rank = torch.tensor(order, device=DEV)
    start = torch.tensor([first[k] for k in order], device=DEV)
    alive = [sum(1 for n in lens if n > t) for t in range(max(lens))]
    h = h[rank]
    sig = torch.sigmoid

    def parts(at):
        rho = sig(fr[at])
        a = torch.exp(-A * rho)
        n2 = -torch.expm1(-2 * A * rho)
        return rho, a, torch.sqrt(n2), sig(fi[at]) if fi is not None else torch.ones_like(a)

    train = "train" in op
    y, prior = torch.empty_like(fx), torch.empty_like(fx) if train else None
    hs = torch.empty_like(fx) if train else None
    for t, m in enumerate(alive):
        at = start[:m] + t
        _, a, n, p = parts(at)
        if train:
            prior[at] = h[:m]
        h[:m] = a * h[:m] + n * p * fx[at]
        if train:
            hs[at] = h[:m]
        y[at] = h[:m] if fz is None else h[:m] * (fz[at] * sig(fz[at]))
    last = torch.empty_like(h)
    last[rank] = h
    out = dict(y=y.reshape(x.shape), h_T=last)
    if not train:
        return out
    dx, dr, di, dz = (torch.empty_like(fx) for _ in range(4))
    dA = torch.zeros((w,), dtype=F64, device=DEV)
    c = torch.zeros((nb, w), dtype=F64, device=DEV)  # the gradient that comes back from the next token
    for t in range(len(alive) - 1, -1, -1):
        m = alive[t]
        at = start[:m] + t
        rho, a, n, p = parts(at)
        g = fdy[at]
        if fz is not None:
            q = sig(fz[at])
            dz[at] = g * hs[at] * (q + fz[at] * q * (1 - q))
            g = g * fz[at] * q
        g = g + c[:m]
        dx[at] = g * n * p
        di[at] = g * n * fx[at] * p * (1 - p)
        da = g * (prior[at] - p * fx[at] * a / n)
        drate = -a * da
        dA += (drate * rho).sum(0)
        dr[at] = drate * A * rho * (1 - rho)
        c[:m] = a * g
    out.update(dx=dx.reshape(x.shape), dr=dr.reshape(x.shape), dA=dA, dr_bias=dr.sum(0))
    if fi is not None:
        out.update(di=di.reshape(x.shape), di_bias=di.sum(0))
    if fz is not None:
        out["dz"] = dz.reshape(x.shape)
    if s["h"] is not None:
        out["dh0"] = torch.empty_like(c)
        out["dh0"][rank] = c
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"].startswith("norm") else _exact_scan(s)
