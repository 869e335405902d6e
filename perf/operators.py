"""Cases of the state-space operators that stand next to the Palimpsa recurrence:
the short causal convolution (a prompt, a packed batch, one token, training) and
the selective scan (the same four), with their plain forms.

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits; with ``own`` true it makes the calls a user of
``metaplastic_linear_attention_gb300`` makes.
"""
import math

import torch

own = False

DEV = "cuda"
F32, F64 = torch.float32, torch.float64


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One layer's convolution at the 760M layer's sizes (24 heads of 64 values, 8 x 4096 tokens).
        dict(name="conv_layer", op="conv", batch=8, tokens=4096, width=1536, taps=4, type="bf16", state=False),
        # A serving prefill: 24 prompts of different lengths in one call, some of them continued from a state.
        dict(name="conv_packed", op="conv_packed", batch=24, tokens=32768, width=2048, taps=4, type="bf16", state=True),
        # A training step of the small layer (16 heads of 64 values): forward and gradients.
        dict(name="conv_train", op="conv_train", batch=4, tokens=2048, width=1024, taps=4, type="bf16", state=False),
        # The same in 32 bits with odd sizes and three taps: a small experiment.
        dict(name="conv_train_odd", op="conv_train", batch=3, tokens=1001, width=520, taps=3, type="f32", state=True),
        # One decode token for the decode job's batch (256 sequences, 32 heads of 64 values).
        dict(name="conv_token", op="conv_token", batch=256, tokens=1, width=2048, taps=4, type="bf16", state=True),
        # One layer's scan at the 760M layer's sizes.
        dict(name="scan_layer", op="scan", batch=8, tokens=4096, width=1536, d_state=16, groups=1, type="bf16",
             gate=True, state=False),
        # One long context: few channels, so time itself has to be split (32 heads of 64 values, 32768 tokens).
        dict(name="scan_long", op="scan", batch=1, tokens=32768, width=2048, d_state=16, groups=1, type="bf16",
             gate=True, state=True),
        # A serving prefill of 13 prompts with a wide state and two groups of B and C.
        dict(name="scan_packed", op="scan_packed", batch=13, tokens=8195, width=1024, d_state=64, groups=2,
             type="bf16", gate=False, state=True),
        # A training step of the small layer: forward with checkpoints, then the gradients.
        dict(name="scan_train", op="scan_train", batch=4, tokens=2048, width=1024, d_state=16, groups=1, type="bf16",
             gate=True, state=False),
        # The same in 32 bits with odd sizes.
        dict(name="scan_train_odd", op="scan_train", batch=2, tokens=777, width=520, d_state=8, groups=1, type="f32",
             gate=False, state=True),
        # One decode token for the decode job's batch.
        dict(name="scan_token", op="scan_token", batch=256, tokens=1, width=2048, d_state=16, groups=1, type="bf16",
             gate=True, state=True),
        # One decode token of one sequence: latency alone.
        dict(name="scan_token_one", op="scan_token", batch=1, tokens=1, width=1024, d_state=16, groups=1, type="bf16",
             gate=True, state=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_packed", "conv_train", "conv_token", "scan", "scan_packed", "scan_train",
                     "scan_token"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    width = 8 * _log(rng, 8, 256)
    if op.startswith("conv"):
        batch = _log(rng, 1, 16 if op != "conv_token" else 256)
        tokens = 1 if op == "conv_token" else _log(rng, batch, max(batch, min(32768, (24 << 20) // (width * batch))))
        if op == "conv_packed":
            tokens = _log(rng, batch, 16384)
        return dict(op=op, batch=batch, tokens=tokens, width=width, taps=rng.choice([2, 3, 4, 4]), type=kind,
                    state=bool(op == "conv_token" or rng.random() < 0.5))
    n = rng.choice([8, 16, 16, 32, 64, 128])
    groups = rng.choice([1, 1, 2, 4])
    width = max(groups * 8, width // (8 * groups) * (8 * groups))
    if op == "scan_token":
        batch, tokens = _log(rng, 1, 256), 1
        width = max(groups * 8, min(width, (8 << 20) // (batch * n)) // (8 * groups) * (8 * groups))
    else:
        most = (64 << 20) if op == "scan_train" else (256 << 20)   # states of all tokens
        batch = _log(rng, 1, 13)
        tokens = _log(rng, 1, max(1, min(16384, most // (width * n * batch))))
        if op == "scan_packed":
            tokens = _log(rng, batch, max(batch, min(16384, most // (width * n))))
    return dict(op=op, batch=batch, tokens=tokens, width=width, d_state=n, groups=groups, type=kind,
                gate=rng.random() < 0.5, state=bool(op == "scan_token" or rng.random() < 0.5))


def _lengths(total, n, seed):
    """n ragged lengths that sum to `total`, each at least 1 where there are tokens enough."""
    g = torch.Generator().manual_seed(seed * 31 + 7)
    w = 0.05 + torch.rand((n,), generator=g, dtype=F64)
    if total < n:
        return [1] * total + [0] * (n - total)
    got = ((w / w.sum() * (total - n)).floor().to(torch.int64) + 1).tolist()
    got[-1] += total - sum(got)
    return got


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1009 + 17)
    dt_ = torch.bfloat16 if case["type"] == "bf16" else F32
    op, nb, t, w = case["op"], case["batch"], case["tokens"], case["width"]
    packed, token, train = op.endswith("packed"), op.endswith("token"), op.endswith("train")

    def randn(*shape, scale=1.0, dtype=dt_):
        return (scale * torch.randn(shape, generator=g, device=DEV, dtype=F32)).to(dtype)

    rows = (t,) if packed else (nb,) if token else (nb, t)
    s = dict(case=dict(case), cu=None, longest=None)
    if packed:
        ls = _lengths(t, nb, int(seed) % 1000)
        cu = [0]
        for n in ls:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["longest"] = max(ls)
    if op.startswith("conv"):
        k = case["taps"]
        s["x"] = randn(*rows, w)
        s["weight"] = randn(w, k, scale=k ** -0.5, dtype=F32)
        s["bias"] = randn(w, scale=0.1, dtype=F32)
        s["state"] = randn(nb, k - 1, w) if case["state"] else None
        if train:
            s["dy"] = randn(*rows, w)
        return s
    n, gr = case["d_state"], case["groups"]
    # x as it leaves the convolution's SiLU; step sizes log-uniform over [0.001, 0.1], moved by the token;
    # A the integers 1 .. N with a jitter of a tenth.
    s["x"] = torch.nn.functional.silu(torch.randn(rows + (w,), generator=g, device=DEV, dtype=F32)).to(dt_)
    d0 = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((w,), generator=g, device=DEV, dtype=F32))
    s["dt_bias"] = d0 + torch.log(-torch.expm1(-d0))
    s["dt"] = randn(*rows, w, scale=0.5)
    s["A"] = torch.arange(1, n + 1, device=DEV, dtype=F32) * (1 + 0.1 * torch.rand((w, n), generator=g, device=DEV))
    s["B"] = randn(*rows, gr, n)
    s["C"] = randn(*rows, gr, n)
    s["D"] = 1 + randn(w, scale=0.1, dtype=F32)
    s["z"] = randn(*rows, w) if case["gate"] else None
    s["h"] = randn(nb, w, n, scale=0.1, dtype=F32) if case["state"] else None
    if train:
        s["dy"] = randn(*rows, w)
    return s


# ------------------------------------------------------------------ the framework's calls

def _own_run(s):
    import metaplastic_linear_attention_gb300 as pal
    op = s["case"]["op"]
    if op in ("conv", "conv_packed"):
        return pal.palimpsa_causal_conv(s["x"], s["weight"], s["bias"], s["state"], cu_seqlens=s["cu"],
                                        max_seqlen=s["longest"])
    if op == "conv_token":
        return pal.palimpsa_causal_conv_step(s["x"], s["weight"], s["bias"], s["state"]), s["state"]
    if op == "conv_train":
        y, last = pal.palimpsa_causal_conv(s["x"], s["weight"], s["bias"], s["state"])
        g = pal.palimpsa_causal_conv_backward(s["x"], s["weight"], s["bias"], s["state"], s["dy"],
                                              want_state_grad=s["state"] is not None)
        return dict(g, y=y, state_T=last)
    a = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    if op in ("scan", "scan_packed"):
        return pal.palimpsa_selective_scan(*a, s["D"], s["z"], s["dt_bias"], s["h"], cu_seqlens=s["cu"],
                                           max_seqlen=s["longest"])
    if op == "scan_token":
        return pal.palimpsa_selective_scan_step(*a, s["h"], s["D"], s["z"], s["dt_bias"]), s["h"]
    y, h, ckpt = pal.palimpsa_selective_scan_checkpointed(*a, s["D"], s["z"], s["dt_bias"], s["h"])
    g = pal.palimpsa_selective_scan_backward(*a, s["D"], s["z"], s["dt_bias"], s["h"], ckpt, s["dy"],
                                             want_state_grad=s["h"] is not None)
    return dict(g, y=y, h_T=h)


# ------------------------------------------------------------------ the plain forms

def _silu(u):
    return u / (1 + torch.exp(-u))


def _dsilu(u):
    p = 1 / (1 + torch.exp(-u))
    return p * (1 + u * (1 - p))


def _softplus(u):
    return torch.clamp(u, min=0) + torch.log1p(torch.exp(-torch.abs(u)))


def _places(s):
    """(sequence of each token, its place in it, end of its sequence) of a packed batch."""
    cu = s["cu"].long()
    t = torch.arange(s["x"].shape[0], device=DEV)
    q = torch.searchsorted(cu, t, right=True) - 1
    return cu, q, t - cu[q]


def _taps(s):
    """The K shifted inputs of every token, in 32 bits, [K] + x.shape, and the last K - 1 inputs."""
    x, k = s["x"].float(), s["weight"].shape[1]
    nb, w = s["case"]["batch"], x.shape[-1]
    st = s["state"].float() if s["state"] is not None else torch.zeros((nb, k - 1, w), device=DEV)
    if s["cu"] is None:
        full = torch.cat([st, x], 1)
        t = x.shape[1]
        return torch.stack([full[:, j:j + t] for j in range(k)]), full[:, t:]
    cu, q, pos = _places(s)
    row = torch.arange(x.shape[0], device=DEV)
    got = []
    for j in range(k):
        back = k - 1 - j
        inside = (pos >= back)[:, None]
        got.append(torch.where(inside, x[(row - back).clamp(min=0)], st[q, (pos + j).clamp(max=k - 2)]))
    ends = (cu[1:] - cu[:-1])[:, None] + torch.arange(k - 1, device=DEV)          # place in [state, inputs]
    inputs = x[(cu[:-1, None] + ends - (k - 1)).clamp(0, max(0, x.shape[0] - 1))]
    olds = torch.gather(st, 1, ends.clamp(max=k - 2)[..., None].expand(-1, -1, w))
    return torch.stack(got), torch.where((ends >= k - 1)[..., None], inputs, olds)


def _conv(s):
    kind = s["x"].dtype
    if s["case"]["op"] == "conv_token":
        full = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
        u = (full * s["weight"].t()).sum(1) + s["bias"]
        s["state"].copy_(full[:, 1:].to(kind))
        return _silu(u).to(kind), s["state"]
    taps, last = _taps(s)
    wt = s["weight"].t()
    u = (taps * wt.reshape((wt.shape[0],) + (1,) * (taps.dim() - 2) + (-1,))).sum(0) + s["bias"]
    y, last = _silu(u).to(kind), last.to(kind)
    if s["case"]["op"] != "conv_train":
        return y, last
    du = s["dy"].float() * _dsilu(u)
    k, t = wt.shape[0], u.shape[1]
    full = torch.zeros((u.shape[0], t + k - 1, u.shape[2]), device=DEV)
    for j in range(k):
        full[:, j:j + t] += wt[j] * du
    out = dict(dx=full[:, k - 1:].to(kind), dweight=(taps * du).sum((1, 2)).t().contiguous(), dbias=du.sum((0, 1)),
               y=y, state_T=last)
    if s["state"] is not None:
        out["dstate0"] = full[:, :k - 1].to(kind)
    return out


def _spread(m, w):
    """B or C of the channels: [..., G, N] -> [..., D, N], in 32 bits."""
    return m.float().repeat_interleave(w // m.shape[-2], dim=-2)


def _doubled(h, total, a, pos, longest, forward):
    """h_t + the decayed h of the earlier (or, with forward false, the later) tokens of its sequence, by doubling:
    h [.., T, D, N], total [.., T, D] the running sum of the step sizes in 64 bits, pos [T] the tokens before (after), `longest` the longest sequence."""
    axis, step = h.dim() - 3, 1
    while step < longest:
        m = h.shape[axis] - step
        gap = (total.narrow(axis, step, m) - total.narrow(axis, 0, m)).float()
        near, far = (step, 0) if forward else (0, step)
        reach = (pos >= step).narrow(0, near, m).to(F32).reshape((m, 1, 1))
        add = torch.exp(-a * gap[..., None])
        add *= h.narrow(axis, far, m)
        add *= reach
        h = torch.cat([h.narrow(axis, 0, step), h.narrow(axis, step, m) + add] if forward
                      else [h.narrow(axis, 0, m) + add, h.narrow(axis, m, step)], axis)
        step *= 2
    return h


def _scan(s):
    op, kind = s["case"]["op"], s["x"].dtype
    x, a, skip = s["x"].float(), s["A"], s["D"]
    w = x.shape[-1]
    raw = s["dt"].float() + s["dt_bias"]
    dt = _softplus(raw)
    b, c = _spread(s["B"], w), _spread(s["C"], w)
    if op == "scan_token":
        h = torch.exp(-a * dt[..., None]) * s["h"] + (dt * x)[..., None] * b
        s["h"].copy_(h)
        y = (h * c).sum(-1) + skip * x
        y = y * _silu(s["z"].float()) if s["z"] is not None else y
        return y.to(kind), s["h"]
    total = torch.cumsum(dt.double(), dim=-2)
    h = (dt * x)[..., None] * b
    if s["cu"] is None:
        pos = torch.arange(x.shape[1], device=DEV)
        if s["h"] is not None:
            h[:, 0] += torch.exp(-a * dt[:, 0, :, None]) * s["h"]
    else:
        cu, _, pos = _places(s)
        some = (cu[1:] > cu[:-1]).nonzero()[:, 0]
        if s["h"] is not None:
            first = cu[some]
            h[first] += torch.exp(-a * dt[first][..., None]) * s["h"][some]
    h = _doubled(h, total, a, pos, s["longest"] or x.shape[1], True)
    pre = (h * c).sum(-1) + skip * x
    gate = _silu(s["z"].float()) if s["z"] is not None else None
    y = (pre if gate is None else pre * gate).to(kind)
    if s["cu"] is not None:
        last = s["h"].clone() if s["h"] is not None else torch.zeros((cu.numel() - 1, w, a.shape[1]), device=DEV)
        last[some] = h[cu[some + 1] - 1]
        return y, last
    if op == "scan":
        return y, h[:, -1].contiguous()
    # gradients: dh_t = C_t dy_t + alpha_{t+1} dh_{t+1}
    dy = s["dy"].float()
    dpre = dy if gate is None else dy * gate
    dh = _doubled(dpre[..., None] * c, total, a, pos.flip(0), x.shape[1], False)
    alpha = torch.exp(-a * dt[..., None])
    before = torch.cat([s["h"][:, None] if s["h"] is not None else torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    old = dh * (alpha * before)                        # the gradient of -A dt
    write = (dh * b).sum(-1)                           # the gradient of dt x
    ddt = write * x - (old * a).sum(-1)
    draw_ = ddt * torch.exp(raw - dt)                  # softplus' = sigmoid = exp(raw - softplus(raw))
    g = s["B"].shape[-2]
    per = lambda m: m.reshape(m.shape[:2] + (g, w // g, m.shape[-1])).sum(3)  # noqa: E731
    out = dict(y=y, h_T=h[:, -1].contiguous(), dx=(write * dt + dpre * skip).to(kind), ddt=draw_.to(kind),
               dA=-(old * dt[..., None]).sum((0, 1)), dB=per(dh * (dt * x)[..., None]).to(kind),
               dC=per(h * dpre[..., None]).to(kind), dD=(dpre * x).sum((0, 1)), ddt_bias=draw_.sum((0, 1)))
    if gate is not None:
        out["dz"] = (dy * pre * _dsilu(s["z"].float())).to(kind)
    if s["h"] is not None:
        out["dh0"] = alpha[:, 0] * dh[:, 0]
    return out


def run(state):
    if own:
        return _own_run(state)
    return _conv(state) if state["case"]["op"].startswith("conv") else _scan(state)


# ------------------------------------------------------------------ work

def work(case):
    e = 2 if case["type"] == "bf16" else 4
    op, nb, w = case["op"], case["batch"], case["width"]
    rows = case["tokens"] if op.endswith("packed") else nb * case["tokens"]
    cells = rows * w
    if op.startswith("conv"):
        k = case["taps"]
        flops, moved = cells * (2 * k + 6), 2 * cells * e + w * (k + 1) * 4
        moved += nb * w * (k - 1) * e * (2 if case["state"] else 1)
        if op == "conv_train":  # x and dy in, dx out; x and y of the forward are counted above
            moved += 2 * cells * e + w * (k + 1) * 4
            flops += cells * (4 * k + 12)
        return dict(bytes=moved, flops=flops)
    n, g = case["d_state"], case["groups"]
    z = 1 if case["gate"] else 0
    moved = cells * e * (3 + z) + rows * 2 * g * n * e + w * n * 4 + 2 * w * 4
    moved += nb * w * n * 4 * (2 if case["state"] else 1)
    flops = cells * (7 * n + 12 + 6 * z)
    if op == "scan_train":      # dy in; dx, ddt, dz, dB, dC and the parameters' gradients out
        moved += cells * e * (3 + z) + rows * 2 * g * n * e + w * n * 4 + 2 * w * 4
        moved += nb * w * n * 4 if case["state"] else 0
        flops += cells * (20 * n + 20 + 10 * z)
    return dict(bytes=moved, flops=flops)


# ------------------------------------------------------------------ 64 bits, token by token

def _walk_conv(s):
    """The convolution in 64 bits, one sequence after the other."""
    x, wt, bias, k = s["x"].to(F64), s["weight"].to(F64), s["bias"].to(F64), s["weight"].shape[1]
    nb, w = s["case"]["batch"], x.shape[-1]
    if s["case"]["op"] == "conv_token":
        seqs = [x[i:i + 1] for i in range(nb)]
    elif s["cu"] is not None:
        cu = s["cu"].tolist()
        seqs = [x[cu[i]:cu[i + 1]] for i in range(nb)]
    else:
        seqs = list(x)
    ys, lasts, grads = [], [], []
    dweight, dbias = torch.zeros((w, k), dtype=F64, device=DEV), torch.zeros((w,), dtype=F64, device=DEV)
    for i, xi in enumerate(seqs):
        st = s["state"][i].to(F64) if s["state"] is not None else torch.zeros((k - 1, w), dtype=F64, device=DEV)
        full = torch.cat([st, xi])
        t = xi.shape[0]
        u = bias.expand(t, w).clone()
        for j in range(k):
            u += full[j:j + t] * wt[:, j]
        sig = torch.sigmoid(u)
        ys.append(u * sig)
        lasts.append(full[t:])
        if "dy" in s:
            du = s["dy"][i].to(F64) * (sig + u * sig * (1 - sig))
            d = torch.zeros_like(full)
            for j in range(k):
                d[j:j + t] += du * wt[:, j]
                dweight[:, j] += (du * full[j:j + t]).sum(0)
            dbias += du.sum(0)
            grads.append(d)
    last = torch.stack(lasts)
    if s["case"]["op"] != "conv_train":
        return (torch.cat(ys) if s["case"]["op"] != "conv" else torch.stack(ys)), last
    d = torch.stack(grads)
    out = dict(y=torch.stack(ys), state_T=last, dx=d[:, k - 1:], dweight=dweight, dbias=dbias)
    if s["state"] is not None:
        out["dstate0"] = d[:, :k - 1]
    return out


def _walk_scan(s):
    """The selective scan in 64 bits, one token after the other (all sequences of a dense batch at once)."""
    op = s["case"]["op"]
    nb, w, n = s["case"]["batch"], s["case"]["width"], s["case"]["d_state"]
    up = lambda t: None if t is None else t.to(F64)  # noqa: E731
    x, dt_raw, a, z, skip = up(s["x"]), up(s["dt"]) + up(s["dt_bias"]), up(s["A"]), up(s["z"]), up(s["D"])
    dt = torch.logaddexp(dt_raw, torch.zeros_like(dt_raw))
    per = w // s["case"]["groups"]
    wide = lambda m: up(m).repeat_interleave(per, dim=-2)  # noqa: E731
    h0 = up(s["h"]) if s["h"] is not None else torch.zeros((nb, w, n), dtype=F64, device=DEV)
    gate = z * torch.sigmoid(z) if z is not None else None

    def token(h, xt, dtt, bt, ct):
        h = torch.exp(-dtt[..., None] * a) * h + (dtt * xt)[..., None] * wide(bt)
        return h, (h * wide(ct)).sum(-1) + skip * xt

    if op == "scan_token":
        h, y = token(h0, x, dt, s["B"], s["C"])
        return (y if gate is None else y * gate), h
    if op == "scan_packed":
        cu = s["cu"].tolist()
        y, ends = torch.empty_like(x), []
        for i in range(nb):
            h = h0[i]
            for t in range(cu[i], cu[i + 1]):
                h, y[t] = token(h, x[t], dt[t], s["B"][t], s["C"][t])
            ends.append(h)
        return (y if gate is None else y * gate), torch.stack(ends)
    length, h = x.shape[1], h0
    pre, kept = torch.empty_like(x), []
    for t in range(length):
        if op == "scan_train":
            kept.append(h)
        h, pre[:, t] = token(h, x[:, t], dt[:, t], s["B"][:, t], s["C"][:, t])
    y = pre if gate is None else pre * gate
    if op == "scan":
        return y, h
    dy = up(s["dy"])
    dpre = dy if gate is None else dy * gate
    z8 = lambda *shape: torch.zeros(shape, dtype=F64, device=DEV)  # noqa: E731
    dx, ddt, da = torch.empty_like(x), torch.empty_like(x), z8(w, n)
    db, dc = z8(*s["B"].shape), z8(*s["B"].shape)
    grouped = lambda m: m.reshape(nb, s["case"]["groups"], per, n).sum(2)  # noqa: E731
    g = z8(nb, w, n)
    for t in range(length - 1, -1, -1):
        bt, ct = wide(s["B"][:, t]), wide(s["C"][:, t])
        decay = torch.exp(-dt[:, t, :, None] * a)
        carried = decay * kept[t]
        ht = carried + (dt[:, t] * x[:, t])[..., None] * bt
        dc[:, t] = grouped(ht * dpre[:, t, :, None])
        g = g + dpre[:, t, :, None] * ct
        db[:, t] = grouped(g * (dt[:, t] * x[:, t])[..., None])
        into = (g * bt).sum(-1)
        dx[:, t] = into * dt[:, t] + dpre[:, t] * skip
        ddt[:, t] = into * x[:, t] - (g * carried * a).sum(-1)
        da -= (g * carried * dt[:, t, :, None]).sum(0)
        g = g * decay
    ddt = ddt * torch.sigmoid(dt_raw)
    out = dict(y=y, h_T=h, dx=dx, ddt=ddt, dA=da, dB=db, dC=dc, dD=(dpre * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))
    if z is not None:
        sig = torch.sigmoid(z)
        out["dz"] = dy * pre * (sig + z * sig * (1 - sig))
    if s["h"] is not None:
        out["dh0"] = g
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _walk_conv(s) if case["op"].startswith("conv") else _walk_scan(s)
