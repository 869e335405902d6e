"""The state-space operators on the GPU against the fp64 oracle on the same (rounded) inputs.

Bars, relative L2 per output. A value that is rounded once to the input type is off by at most half a
step, 2^-8 relative in bf16. What is computed in fp32: step sizes here are at least 0.02 and A at
least 0.3, so a state remembers at most 170 tokens; each adds at most 2^-22 (the exponential,
2 ulp) + 2^-23 (two roundings) + 2^-23 |A s| (the exponent's rounding, |A s| < 1 wherever the state
survives a token) < 6e-7 relative, in all 1e-4. Sums add their terms' errors, so the bar holds for them
relative to the terms; a gradient that sums over tokens or channels keeps it because random signs do
not make the sum smaller than a term's share times the root of their number, and neither the errors.
The convolution adds at most W + 2 roundings: 1e-6."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from oracle import ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _rel(got, want):
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    d = float((got - want).norm())
    n = float(want.norm())
    return d / n if n else d


def _near(got, want, bar, what=""):
    r = _rel(got, want)
    assert r <= bar, f"{what}: relative L2 {r:.3g} over {bar:.3g}"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _r(g, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _up(d):
    return {k: None if v is None else v.to(F64) for k, v in d.items()}


def _dev(d):
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}


def _conv_inputs(seed, rows, n, D, W, dtype, bias=True, state=True):
    g = _gen(seed)
    return dict(x=_r(g, rows, D, dtype=dtype), weight=_r(g, D, W, scale=W ** -0.5), bias=_r(g, D) if bias else None,
                state0=_r(g, n, W - 1, D, dtype=dtype) if state else None)


def _scan_inputs(seed, rows, n, D, G, N, dtype, gate=True, state=True, extras=True):
    g = _gen(seed)
    dt = _r(g, rows, D, dtype=dtype, scale=0.5)
    bias = -2.0 + 0.3 * torch.randn((D,), generator=g)
    return dict(x=_r(g, rows, D, dtype=dtype), dt=dt if extras else (dt.float() - 2).to(dtype),
                A=0.3 + 2 * torch.rand((D, N), generator=g), B=_r(g, rows, G, N, dtype=dtype),
                C=_r(g, rows, G, N, dtype=dtype), D=_r(g, D) if extras else None,
                z=_r(g, rows, D, dtype=dtype) if gate else None, dt_bias=bias if extras else None,
                h0=_r(g, n, D, N) if state else None)


def _dense(i, B, names=("x", "dt", "z", "B", "C", "dy")):
    return {k: v.reshape((B, -1) + tuple(v.shape[1:])) if v is not None and k in names else v for k, v in i.items()}


def _status():
    assert pal.palimpsa_get_device_status() == 0


# ------------------------------------------------------------------ convolution

CONV_SHAPES = [(1, 1, 8, 4), (2, 3, 64, 4), (3, 1, 8, 2), (1, 130, 2048, 4), (2, 33, 520, 3), (5, 8, 264, 2), (1, 2, 16, 4),
               (2, 65, 136, 4)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D,W", CONV_SHAPES)
@pytest.mark.parametrize("silu,bias,state", [(True, True, True), (False, False, False), (True, False, True)])
def test_conv_dense(dtype, B, T, D, W, silu, bias, state):
    i = _conv_inputs(B * T + D, B * T, B, D, W, dtype, bias, state)
    cu = _cu([T] * B)
    g = _gen(9)
    dy, dl = _r(g, B * T, D, dtype=dtype), _r(g, B, W - 1, D, dtype=dtype)
    y, last, grads = ssm.gradients(ssm.conv, _up(i), dy.to(F64), dl.to(F64), cu, silu=silu)
    d = _dev(_dense(i, B, ("x",)))
    gy, gs = pal.palimpsa_causal_conv(*d.values(), silu=silu)
    bar = HALF[dtype] + 1e-6
    _near(gy.reshape(-1, D), y, bar, "y")
    assert torch.equal(gs.cpu().to(F64), last)
    got = pal.palimpsa_causal_conv_backward(*d.values(), dy.reshape(B, T, D).to(DEV), dl.to(DEV), silu=silu)
    _near(got["dx"].reshape(-1, D), grads["x"], bar, "dx")
    _near(got["dweight"], grads["weight"], 1e-5, "dweight")   # sums of up to 130 x 2 terms of either sign
    if bias:
        _near(got["dbias"], grads["bias"], 1e-5, "dbias")
    if state:
        _near(got["dstate0"], grads["state0"], bar, "dstate0")
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[5, 0, 1, 130, 2, 3], [1], [0, 0, 7], [700, 3, 1]])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_packed(dtype, lens, W):
    D, n, tail = 136, len(lens), 3
    cu = _cu(lens)
    i = _conv_inputs(sum(lens), cu[-1] + tail, n, D, W, dtype)
    g = _gen(8)
    dy, dl = _r(g, cu[-1] + tail, D, dtype=dtype), _r(g, n, W - 1, D, dtype=dtype)
    y, last, grads = ssm.gradients(ssm.conv, _up(i), dy.to(F64), dl.to(F64), cu)
    d, cud = _dev(i), torch.tensor(cu, dtype=torch.int32, device=DEV)
    mine = torch.full((cu[-1] + tail, D), 7.0, dtype=dtype, device=DEV)
    gy, gs = pal.palimpsa_causal_conv(*d.values(), cu_seqlens=cud, max_seqlen=max(lens), y=mine)
    bar = HALF[dtype] + 1e-6
    _near(gy[:cu[-1]], y[:cu[-1]], bar, "y")
    assert (gy[cu[-1]:] == 7).all()         # rows behind the last sequence stay as they were
    assert torch.equal(gs.cpu().to(F64), last)
    got = pal.palimpsa_causal_conv_backward(*d.values(), dy.to(DEV), dl.to(DEV), cu_seqlens=cud, max_seqlen=max(lens))
    _near(got["dx"], grads["x"], bar, "dx")
    _near(got["dstate0"], grads["state0"], bar, "dstate0")
    _near(got["dweight"], grads["weight"], 1e-5, "dweight")
    _near(got["dbias"], grads["bias"], 1e-5, "dbias")
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_conv_steps_continue_a_prompt(dtype):
    """A prompt, then tokens one by one, equals the whole sequence; state and y bit for bit."""
    B, T, D, W = 3, 21, 72, 4
    i = _dev(_dense(_conv_inputs(3, B * T, B, D, W, dtype), B, ("x",)))
    y, last = pal.palimpsa_causal_conv(*i.values())
    state = i["state0"].clone()
    y1, _ = pal.palimpsa_causal_conv(i["x"][:, :9].contiguous(), i["weight"], i["bias"], state, state_T=state)  # in place
    ys = [y1]
    for t in range(9, T):
        ys.append(pal.palimpsa_causal_conv_step(i["x"][:, t], i["weight"], i["bias"], state)[:, None])
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(state, last)


# ------------------------------------------------------------------ selective scan

SCAN_SHAPES = [  # B, T, D, G, N
    (1, 1, 8, 1, 16), (2, 17, 64, 1, 16), (1, 33, 40, 1, 8), (3, 15, 72, 3, 32), (2, 50, 48, 2, 64), (1, 40, 16, 2, 128),
    (2, 300, 96, 1, 16), (1, 600, 32, 1, 16), (1, 259, 64, 1, 64), (1, 290, 24, 1, 8)]


def _scan_case(dtype, lens, dense, D, G, N, gate, state, extras, tail=0):
    n, cu = len(lens), _cu(lens)
    rows = cu[-1] + tail
    i = _scan_inputs(rows + D + N, rows, n, D, G, N, dtype, gate, state, extras)
    g = _gen(7)
    dy, dl = _r(g, rows, D, dtype=dtype), _r(g, n, D, N)
    y, last, grads = ssm.gradients(ssm.scan, _up(i), dy.to(F64), dl.to(F64), cu)
    cud = None if dense else torch.tensor(cu, dtype=torch.int32, device=DEV)
    kw = {} if dense else dict(cu_seqlens=cud, max_seqlen=max(lens))
    d = _dev(_dense(i, n) if dense else i)
    gdy = _dense(dict(dy=dy), n)["dy"].to(DEV) if dense else dy.to(DEV)
    gy, gh = pal.palimpsa_selective_scan(*d.values(), **kw)
    cy, chh, ckpt = pal.palimpsa_selective_scan_checkpointed(*d.values(), **kw)
    assert torch.equal(gy, cy) and torch.equal(gh, chh)
    fine, bar = 1e-4, HALF[dtype] + 1e-4
    _near(gy.reshape(-1, D), y, bar, "y")
    _near(gh, last, fine, "h_T")
    got = pal.palimpsa_selective_scan_backward(*d.values(), ckpt, gdy, dl.to(DEV), **kw)
    again = pal.palimpsa_selective_scan_backward(*d.values(), ckpt, gdy, dl.to(DEV), **kw)
    for k, v in got.items():
        assert torch.equal(v, again[k]), f"{k} differs from run to run"
    flat = lambda t: t.reshape((-1,) + tuple(t.shape[2:])) if dense else t  # noqa: E731
    for k, name in (("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dz", "z")):
        if k in got:
            _near(flat(got[k]), grads[name], bar, k)
    for k, name in (("dA", "A"), ("dD", "D"), ("ddt_bias", "dt_bias"), ("dh0", "h0")):
        if name in grads:
            _near(got[k], grads[name], fine, k)
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D,G,N", SCAN_SHAPES)
@pytest.mark.parametrize("gate,state,extras", [(True, True, True), (False, False, False)])
def test_scan_dense(dtype, B, T, D, G, N, gate, state, extras):
    _scan_case(dtype, [T] * B, True, D, G, N, gate, state, extras)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[5, 0, 1, 130, 16, 3], [0], [0, 0, 7], [400, 3, 1, 129], [32, 16, 48]])
@pytest.mark.parametrize("D,G,N", [(40, 1, 16), (48, 2, 32), (8, 1, 8)])
def test_scan_packed(dtype, lens, D, G, N):
    _scan_case(dtype, lens, False, D, G, N, True, True, True, tail=2)


# One long sequence among hundreds of short ones: the grids cover the batch's rows, not the
# longest sequence's length times the number of sequences (which would be over 16384 CTAs more).
def _one_long(count, long, at):
    return [long if k == at else (0, 1, 3, 2)[k % 4] for k in range(count)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("at", [0, 333, 599])
@pytest.mark.parametrize("W", [3, 4])
def test_conv_packed_one_long(dtype, at, W):
    test_conv_packed(dtype, _one_long(600, 2000, at), W)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("count,long,at,D,G,N", [
    (600, 900, 599, 40, 1, 16), (1200, 500, 700, 40, 1, 16), (600, 900, 1, 48, 2, 32), (1100, 900, 0, 16, 1, 128),
    (1100, 500, 1030, 64, 1, 8)])
def test_scan_packed_one_long(dtype, count, long, at, D, G, N):
    _scan_case(dtype, _one_long(count, long, at), False, D, G, N, True, True, True, tail=2)


def test_packed_one_long_with_bad_offsets():
    """As above with a sequence over max_seqlen in the middle and one past the rows at the end: both are skipped."""
    lens = _one_long(700, 900, 20)
    lens[400], lens[-1] = 901, 50
    D, N, cu = 136, 16, _cu(lens)
    rows, ok = cu[-1] - 5, [k not in (400, 699) for k in range(700)]
    i, c = _scan_inputs(3, rows, 700, D, 1, N, F32), _conv_inputs(3, rows, 700, D, 4, F32)
    dy = torch.ones(rows, D)
    keep = torch.zeros(rows, dtype=torch.bool)
    for n in range(700):
        if ok[n]:
            keep[cu[n]:cu[n + 1]] = True
    cug = _cu([n for n, fine in zip(lens, ok) if fine])
    okt = torch.tensor(ok)
    pick = lambda v: (v[keep] if v.shape[0] == rows else v[okt] if v.shape[0] == 700 else v).to(F64)  # noqa: E731
    sub = lambda d: {k: pick(v) for k, v in d.items()}  # noqa: E731
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=900)
    zero = torch.zeros(int(okt.sum()), D, N, dtype=F64)
    y, last, want = ssm.gradients(ssm.scan, sub(i), dy[keep].to(F64), zero, cug)
    h = torch.full((700, D, N), 7.0, device=DEV)
    gy, _, ckpt = pal.palimpsa_selective_scan_checkpointed(*_dev(i).values(), h_T=h, **kw)
    assert pal.palimpsa_get_device_status() == 5
    g = pal.palimpsa_selective_scan_backward(*_dev(i).values(), ckpt, dy.to(DEV), **kw)
    assert pal.palimpsa_get_device_status() == 5
    _near(gy[keep], y, 1e-4, "y")
    _near(h[okt], last, 1e-4, "h_T")
    assert (h[~okt] == 7).all() and not gy[~keep].any()
    for k, name in (("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dz", "z")):
        _near(g[k][keep], want[name], 1e-4, k)
        assert not g[k][~keep].any()
    for k, name in (("dA", "A"), ("dD", "D"), ("ddt_bias", "dt_bias")):
        _near(g[k], want[name], 1e-4, k)
    _near(g["dh0"][okt], want["h0"], 1e-4, "dh0")
    y, last, want = ssm.gradients(ssm.conv, sub(c), dy[keep].to(F64), torch.zeros(int(okt.sum()), 3, D, dtype=F64), cug)
    gy, gs = pal.palimpsa_causal_conv(*_dev(c).values(), **kw)
    assert pal.palimpsa_get_device_status() == 5
    g = pal.palimpsa_causal_conv_backward(*_dev(c).values(), dy.to(DEV), **kw)
    assert pal.palimpsa_get_device_status() == 5
    _near(gy[keep], y, 2e-6, "y")
    assert torch.equal(gs[okt].cpu().to(F64), last) and not gy[~keep].any()
    _near(g["dx"][keep], want["x"], 2e-6, "dx")
    _near(g["dweight"], want["weight"], 1e-5, "dweight")
    _near(g["dbias"], want["bias"], 1e-5, "dbias")


def test_scan_leaves_rows_behind_the_last_sequence():
    lens, D, N = [5, 300], 32, 16
    cu = torch.tensor(_cu(lens), dtype=torch.int32, device=DEV)
    i = _dev(_scan_inputs(1, 310, 2, D, 1, N, BF))
    y = torch.full((310, D), 7.0, dtype=BF, device=DEV)
    pal.palimpsa_selective_scan(*i.values(), cu_seqlens=cu, max_seqlen=300, y=y)
    assert (y[305:] == 7).all() and not (y[:305] == 7).all(1).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,G,N", [(64, 1, 16), (40, 1, 8), (48, 3, 32), (32, 2, 64), (24, 1, 128)])
@pytest.mark.parametrize("gate", [True, False])
def test_scan_steps_continue_a_prompt(dtype, D, G, N, gate):
    B, T, cut = 3, 25, 18
    flat = _scan_inputs(5, B * T, B, D, G, N, dtype, gate)
    y, last = ssm.scan(*_up(flat).values(), _cu([T] * B))
    d = _dev(_dense(flat, B))
    tok = ("x", "dt", "B", "C", "z")
    head = {k: v[:, :cut].contiguous() if k in tok and v is not None else v for k, v in d.items()}
    h = d["h0"].clone()
    gy, _ = pal.palimpsa_selective_scan(*dict(head, h0=h).values(), h_T=h)      # in place
    got = [gy]
    for t in range(cut, T):
        s = {k: (None if d[k] is None else d[k][:, t]) for k in tok}             # strided rows
        got.append(pal.palimpsa_selective_scan_step(s["x"], s["dt"], d["A"], s["B"], s["C"], h, d["D"], s["z"],
                                                    d["dt_bias"])[:, None])
    _near(torch.cat(got, 1).reshape(-1, D), y, HALF[dtype] + 1e-4, "y")
    _near(h, last, 1e-4, "h")
    _status()


def test_long_in_place_state_with_a_time_split():
    """Few channels over many tokens (time is split): h_T may be h0, and a cut sequence continues."""
    T, D, N = 4096, 32, 16
    i = _dev(_dense(_scan_inputs(6, T, 1, D, 1, N, F32), 1))
    y, h = pal.palimpsa_selective_scan(*i.values())
    tok = ("x", "dt", "B", "C", "z")
    state = i["h0"].clone()
    ys = []
    for a, b in ((0, 1000), (1000, 1001), (1001, T)):
        part = {k: v[:, a:b].contiguous() if k in tok else v for k, v in i.items()}
        ys.append(pal.palimpsa_selective_scan(*dict(part, h0=state).values(), h_T=state)[0])
    _near(torch.cat(ys, 1).cpu(), y.cpu(), 1e-4, "y")
    _near(state, h.cpu(), 1e-4, "h")
    _status()


# ------------------------------------------------------------------ both

def test_rows_of_a_wider_projection():
    """x and z are halves of one projection, B and C slices of another: same bits as dense copies."""
    B, T, D, N = 2, 70, 64, 16
    g = _gen(4)
    xz, xbc = _r(g, B, T, 2 * D, dtype=BF).to(DEV), _r(g, B, T, D + 32 + 2 * N, dtype=BF).to(DEV)
    w, bias = _r(g, D, 4).to(DEV), _r(g, D).to(DEV)
    A, skip = (0.3 + torch.rand((D, N), generator=g)).to(DEV), _r(g, D).to(DEV)
    x, z = xz[..., :D], xz[..., D:]
    dt, Bm, Cm = xbc[..., :D], xbc[..., D + 32:D + 32 + N].unflatten(-1, (1, N)), xbc[..., D + 32 + N:].unflatten(-1, (1, N))
    assert not x.is_contiguous()
    c = [t.contiguous() for t in (x, z, dt, Bm, Cm)]
    assert torch.equal(pal.palimpsa_causal_conv(x, w, bias)[0], pal.palimpsa_causal_conv(c[0], w, bias)[0])
    a = pal.palimpsa_causal_conv_backward(x, w, bias, None, z)
    b = pal.palimpsa_causal_conv_backward(c[0], w, bias, None, c[1])
    assert all(torch.equal(a[k], b[k]) for k in a)
    a = pal.palimpsa_selective_scan_checkpointed(x, dt, A, Bm, Cm, skip, z)
    b = pal.palimpsa_selective_scan_checkpointed(c[0], c[2], A, c[3], c[4], skip, c[1])
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = pal.palimpsa_selective_scan_backward(x, dt, A, Bm, Cm, skip, z, None, None, a[2], dt)
    b = pal.palimpsa_selective_scan_backward(c[0], c[2], A, c[3], c[4], skip, c[1], None, None, b[2], c[2])
    assert all(torch.equal(a[k], b[k]) for k in a)
    h1, h2 = torch.zeros(B, D, N, device=DEV), torch.zeros(B, D, N, device=DEV)
    y1 = pal.palimpsa_selective_scan_step(x[:, 3], dt[:, 3], A, Bm[:, 3], Cm[:, 3], h1, skip, z[:, 3])
    y2 = pal.palimpsa_selective_scan_step(*(t[:, 3].contiguous() for t in (x, dt)), A, *(t[:, 3].contiguous() for t in (Bm, Cm)),
                                          h2, skip, z[:, 3].contiguous())
    assert torch.equal(y1, y2) and torch.equal(h1, h2)
    _status()


@pytest.mark.parametrize("cu", [[0, 5, 20], [3, 9, 17], [4, 4, 4], [0, 0, 0], [20, 20, 20]])
def test_fresh_packed_outputs_are_zero_outside_the_sequences(cu):
    rows, D, N = 20, 16, 16
    junk = torch.full((1 << 20,), float("nan"), device=DEV)       # what the allocator hands out again
    del junk
    i = _dev(_scan_inputs(2, rows, 2, D, 1, N, BF))
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=20)
    y, _, ck = pal.palimpsa_selective_scan_checkpointed(*i.values(), **kw)
    g = pal.palimpsa_selective_scan_backward(*i.values(), ck, i["x"], **kw)
    w = torch.randn(D, 4, device=DEV)
    u, _ = pal.palimpsa_causal_conv(i["x"], w, **kw)
    c = pal.palimpsa_causal_conv_backward(i["x"], w, None, None, i["x"], **kw)
    for t in (y, u, g["dx"], g["ddt"], g["dz"], g["dB"], g["dC"], c["dx"]):
        assert not t[:cu[0]].any() and not t[cu[-1]:].any()
        assert torch.isfinite(t).all()
    _status()


def test_offsets_beyond_32_bits():
    """Rows 2^20 elements apart: the last ones lie beyond 2^31 elements (and 2^32 bytes)."""
    T, D, N, ld = 2200, 64, 16, 1 << 20
    wide = torch.empty(T, ld, dtype=BF, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    parts = [torch.randn((T, D), generator=g, device=DEV).to(BF) for _ in range(4)]
    bc = [torch.randn((T, N), generator=g, device=DEV).to(BF) for _ in range(2)]
    views = []
    for k, t in enumerate(parts + bc):
        v = wide[:, 64 * k:64 * k + t.shape[1]]
        v.copy_(t)
        views.append(v)
    w, A = torch.randn(D, 4, device=DEV), 0.3 + torch.rand(D, N, device=DEV)
    out = []
    for x, dt, z, dy, b, c in (views, parts + bc):
        bm, cm = b.unflatten(-1, (1, N)), c.unflatten(-1, (1, N))
        one = lambda t: t[None]  # noqa: E731
        y, st = pal.palimpsa_causal_conv(one(x), w)
        gc = pal.palimpsa_causal_conv_backward(one(x), w, None, None, one(dy))
        a = (one(x), one(dt), A, one(bm), one(cm), None, one(z))
        ys, h, ck = pal.palimpsa_selective_scan_checkpointed(*a)
        gs = pal.palimpsa_selective_scan_backward(*a, None, None, ck, one(dy))
        cs, hs = torch.zeros(T, 3, D, dtype=BF, device=DEV), torch.zeros(T, D, N, device=DEV)
        y1 = pal.palimpsa_causal_conv_step(x, w, None, cs)
        y2 = pal.palimpsa_selective_scan_step(x, dt, A, bm, cm, hs, None, z)
        out.append([y, st, ys, h, y1, y2, cs, hs, *gc.values(), *gs.values()])
    assert all(torch.equal(p, q) for p, q in zip(*out))
    _status()


@pytest.mark.parametrize("gate", [True, False])
def test_gradients_equal_differences_of_the_kernels(gate):
    """Along a random direction, (L(p + e m) - L(p - e m)) / 2e of the fp32 kernels against <grad, m>. With e = 2^-6 the
    differences are off by e^2 / 6 = 4e-5 of the third derivative along m, and by the roundings of L, at most
    1e-6 |y| |dy| / e; both are held against |grad| |m|."""
    T, D, N, e = 150, 40, 16, 2.0 ** -6
    i = _dev(_dense(_scan_inputs(17, T, 1, D, 1, N, F32, gate=gate), 1))
    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda t: torch.randn(t.shape, generator=g, device=DEV)  # noqa: E731
    dy, dh = rnd(i["x"]), rnd(i["h0"])

    def loss(v):
        y, h = pal.palimpsa_selective_scan(*v.values())
        return float((y.double() * dy).sum() + (h.double() * dh).sum()), float(y.double().norm() * dy.norm())

    _, _, ck = pal.palimpsa_selective_scan_checkpointed(*i.values())
    got = pal.palimpsa_selective_scan_backward(*i.values(), ck, dy, dh)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", dt_bias="ddt_bias", h0="dh0")
    for k, v in i.items():
        if v is None:
            continue
        m = rnd(v)
        m = m / m.norm() * min(1.0, 0.25 * float(v.norm()) if k == "A" else 1.0)
        (up, scale), (down, _) = loss(dict(i, **{k: v + e * m})), loss(dict(i, **{k: v - e * m}))
        grad = got[names[k]].double()
        diff = (up - down) / (2 * e)
        bar = 1e-3 * float(grad.norm() * m.norm()) + 1e-6 * scale / e
        assert abs(diff - float((grad * m).sum())) <= bar, k
    x, w, b = i["x"], rnd(torch.empty(D, 4)), rnd(torch.empty(D))
    st = rnd(torch.empty(1, 3, D))
    gc = pal.palimpsa_causal_conv_backward(x, w, b, st, dy)
    for k, name in ((0, "dx"), (1, "dweight"), (2, "dbias"), (3, "dstate0")):
        args = [x, w, b, st]
        m = rnd(args[k])
        m = m / m.norm()
        y = []
        for s in (1, -1):
            moved = list(args)
            moved[k] = args[k] + s * e * m
            y.append(pal.palimpsa_causal_conv(*moved)[0].double())
        diff = float(((y[0] - y[1]) * dy).sum()) / (2 * e)
        bar = 1e-3 * float(gc[name].norm()) + 1e-6 * float(y[0].norm() * dy.norm()) / e
        assert abs(diff - float((gc[name].double() * m).sum())) <= bar, name
    _status()


def test_calls_on_two_streams_at_once():
    """Split scans and their backward, running side by side, do not share scratch."""
    cases = [_dev(_dense(_scan_inputs(40 + k, 3000, 1, 64, 1, 16, BF), 1)) for k in range(2)]

    def work(i, stream=None):
        y, h, ck = pal.palimpsa_selective_scan_checkpointed(*i.values(), stream=stream)
        return [y, h, *pal.palimpsa_selective_scan_backward(*i.values(), ck, i["x"], stream=stream).values()]

    want = [[t.clone() for t in work(i)] for i in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [work(i, s) for i, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    _status()


def test_empty_prompt_passes_the_state_through():
    h = torch.randn(2, 16, 16, device=DEV)
    e = torch.empty(2, 0, 16, device=DEV)
    bc = torch.empty(2, 0, 1, 16, device=DEV)
    A = torch.ones(16, 16, device=DEV)
    y, last, ckpt = pal.palimpsa_selective_scan_checkpointed(e, e, A, bc, bc, h0=h)
    assert y.numel() == 0 and torch.equal(last, h)
    got = pal.palimpsa_selective_scan_backward(e, e, A, bc, bc, None, None, None, h, ckpt, e, h)
    assert torch.equal(got["dh0"], h) and not got["dA"].any()
    st = torch.randn(2, 3, 16, device=DEV)
    w = torch.randn(16, 4, device=DEV)
    y, last = pal.palimpsa_causal_conv(e, w, None, st)
    assert torch.equal(last, st)
    got = pal.palimpsa_causal_conv_backward(e, w, None, st, e, st)
    assert torch.equal(got["dstate0"], st) and not got["dweight"].any() and not got["dbias"].any()
    _status()


@pytest.mark.parametrize("cu", [[0, 9, 5, 20], [0, 5, 30, 30], [-1, 4, 8, 12], [0, 18, 19, 20]])
def test_bad_offsets_are_reported_and_touch_nothing(cu):
    """Offsets out of order or range, or a sequence longer than max_seqlen: that sequence is skipped."""
    rows, D, N, longest = 20, 16, 16, 12
    i = _dev(_scan_inputs(2, rows, 3, D, 1, N, F32))
    ok = [0 <= a <= b <= rows and b - a <= longest for a, b in zip(cu, cu[1:])]
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    y = torch.full((rows, D), 7.0, device=DEV)
    h = torch.full((3, D, N), 7.0, device=DEV)
    _, _, ckpt = pal.palimpsa_selective_scan_checkpointed(*i.values(), cu_seqlens=cud, max_seqlen=longest, y=y, h_T=h)
    assert pal.palimpsa_get_device_status() == 5
    for n, fine in enumerate(ok):
        assert (h[n] == 7).all() != fine
    g = pal.palimpsa_selective_scan_backward(*i.values(), ckpt, torch.ones(rows, D, device=DEV), cu_seqlens=cud, max_seqlen=longest)
    assert pal.palimpsa_get_device_status() == 5
    for n, fine in enumerate(ok):
        assert g["dh0"][n].any() == fine
    c = _dev(_conv_inputs(2, rows, 3, D, 4, F32))
    y = torch.full((rows, D), 7.0, device=DEV)
    _, st = pal.palimpsa_causal_conv(*c.values(), cu_seqlens=cud, max_seqlen=longest, y=y)
    assert pal.palimpsa_get_device_status() == 5
    pal.palimpsa_causal_conv_backward(*c.values(), torch.ones(rows, D, device=DEV), cu_seqlens=cud, max_seqlen=longest)
    assert pal.palimpsa_get_device_status() == 5
    written = torch.zeros(rows, dtype=torch.bool)
    for (a, b), fine in zip(zip(cu, cu[1:]), ok):
        if fine:
            written[a:b] = True
    assert torch.equal((y == 7).all(1).cpu(), ~written)


def test_fresh_outputs_are_zero_in_the_rows_of_skipped_sequences():
    cu, rows, D, N, longest = [0, 18, 19, 40, 44, 50], 40, 16, 16, 12  # too long, whole, too long, out of range twice
    i = _dev(_scan_inputs(2, rows, 5, D, 1, N, F32))
    c = _dev(_conv_inputs(2, rows, 5, D, 4, F32))
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    kw = dict(cu_seqlens=cud, max_seqlen=longest)
    dy = torch.ones(rows, D, device=DEV)

    def used(*shape):
        """Leaves the allocator with blocks that hold NaN."""
        held = [torch.full(shape, float("nan"), device=DEV) for _ in range(8)]
        del held

    used(rows, D)
    outs = [pal.palimpsa_causal_conv(*c.values(), **kw)[0]]
    used(rows, D)
    outs.append(pal.palimpsa_causal_conv_backward(*c.values(), dy, **kw)["dx"])
    used(rows, D)
    y, _, ckpt = pal.palimpsa_selective_scan_checkpointed(*i.values(), **kw)
    outs.append(y)
    used(rows, D)
    g = pal.palimpsa_selective_scan_backward(*i.values(), ckpt, dy, **kw)
    outs += [g[k] for k in ("dx", "ddt", "dz", "dB", "dC")]
    assert pal.palimpsa_get_device_status() == 5
    for o in outs:
        o = o.reshape(rows, -1)
        assert o[18].abs().sum() > 0 and not o[:18].any() and not o[19:].any()


def test_state_gradients_of_a_packed_batch_on_another_stream():
    """The zeros that a packed batch's state gradients start from are filled in on the call's stream: work that is
    still queued on the current one does not put them over the results."""
    rows, D, N = 20, 16, 16
    i = _dev(_scan_inputs(2, rows, 2, D, 1, N, F32))
    c = _dev(_conv_inputs(2, rows, 2, D, 4, F32))
    kw = dict(cu_seqlens=torch.tensor([0, 9, 20], dtype=torch.int32, device=DEV), max_seqlen=11)
    dy = torch.ones(rows, D, device=DEV)
    _, _, ckpt = pal.palimpsa_selective_scan_checkpointed(*i.values(), **kw)
    want = [pal.palimpsa_selective_scan_backward(*i.values(), ckpt, dy, **kw)["dh0"],
            pal.palimpsa_causal_conv_backward(*c.values(), dy, **kw)["dstate0"]]
    busy = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-2
    got = [pal.palimpsa_selective_scan_backward(*i.values(), ckpt, dy, stream=side, **kw)["dh0"],
           pal.palimpsa_causal_conv_backward(*c.values(), dy, stream=side, **kw)["dstate0"]]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert a.any() and torch.equal(a, b)
    _status()


def test_fresh_outputs_on_another_stream_are_its_own():
    """Memory given back on the current stream, with work still queued there that writes it, is not taken for the
    outputs of a call on another one."""
    B, T, D, N = 2, 50, 64, 16
    i = _dev(_dense(_scan_inputs(4, B * T, B, D, 1, N, F32), B))
    w = torch.randn(D, 4, device=DEV)

    def chain(stream):
        y, st = pal.palimpsa_causal_conv(i["x"], w, stream=stream)
        o, h, ck = pal.palimpsa_selective_scan_checkpointed(*i.values(), stream=stream)
        g = pal.palimpsa_selective_scan_backward(*i.values(), ck, i["x"], stream=stream)
        c = pal.palimpsa_causal_conv_backward(i["x"], w, None, None, i["x"], stream=stream)
        return [y, st, o, h, ck, *g.values(), *c.values()]

    want = chain(None)
    shapes = [t.shape for t in want]
    busy = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-2
    old = [torch.full(s, float("nan"), device=DEV) for s in shapes]
    places = {t.data_ptr() for t in old}
    del old
    got = chain(side)
    assert not places & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    _status()


@pytest.mark.parametrize("what", ["A", "dt", "bias"])
def test_domain_violations_are_latched(what):
    i = _dev(_dense(_scan_inputs(3, 40, 2, 16, 1, 16, F32), 2))
    if what == "A":
        i["A"][3, 5] = 0.0
    elif what == "dt":
        i["dt"][1, 7, 4] = float("nan")
    else:
        i["dt_bias"][2] = float("inf")
    _, _, ckpt = pal.palimpsa_selective_scan_checkpointed(*i.values())
    assert pal.palimpsa_get_device_status() == 5
    pal.palimpsa_selective_scan_backward(*i.values(), ckpt, i["x"])
    assert pal.palimpsa_get_device_status() == 5
    t = lambda k: i[k][:, 7 - 0]  # noqa: E731
    pal.palimpsa_selective_scan_step(t("x"), t("dt"), i["A"], t("B"), t("C"), i["h0"], i["D"], t("z"), i["dt_bias"])
    assert pal.palimpsa_get_device_status() == 5
    _status()


def test_negative_step_size_without_softplus():
    x = torch.ones(1, 4, 8, device=DEV)
    bc = torch.ones(1, 4, 1, 16, device=DEV)
    A = torch.ones(8, 16, device=DEV)
    pal.palimpsa_selective_scan(x, x, A, bc, bc, softplus=False)
    _status()
    pal.palimpsa_selective_scan(x, -x, A, bc, bc, softplus=False)
    assert pal.palimpsa_get_device_status() == 5


def test_extreme_step_sizes_stay_finite():
    """Raw step sizes from far below to far above: softplus 0 (the state stands) to 100 (it is replaced)."""
    raw = torch.tensor([-200.0, -90.0, -20.0, -10.0, 0.0, 20.0, 100.0], dtype=F32)
    T, D, N = raw.numel(), 8, 16
    i = _scan_inputs(8, T, 1, D, 1, N, F32)
    i["dt"], i["dt_bias"] = raw[:, None].expand(T, D).contiguous(), None
    y, last = ssm.scan(*_up(i).values(), [0, T])
    d = _dev(_dense(i, 1))
    gy, gh = pal.palimpsa_selective_scan(*d.values())
    _near(gy[0], y, 1e-4, "y")
    _near(gh, last, 1e-4, "h")
    # each token's own increment: softplus is accurate relative to itself down to e^-90
    one = dict(i, h0=None, D=None, z=None)
    for t in range(1, T):
        step = {k: v[t:t + 1] if k in ("x", "dt", "B", "C") else v for k, v in one.items()}
        _, want = ssm.scan(*_up(step).values(), [0, 1])
        _, got = pal.palimpsa_selective_scan(*_dev(_dense(step, 1)).values())
        # expf of 90 is off by 90 x 2^-23 relative; four more roundings
        _near(got, want, 2e-5, f"softplus({raw[t]})")


def test_a_step_of_size_zero_leaves_the_state_as_it_is():
    """softplus(-200) is 0 in fp32: the decay is exactly 1, for the largest A too."""
    T, D, N = 37, 40, 16
    i = _scan_inputs(12, T, 1, D, 1, N, F32)
    i["dt"], i["dt_bias"] = torch.full((T, D), -200.0), None
    i["A"][0], i["A"][1] = 3e38, 1e-38
    d = _dev(_dense(i, 1))
    _, h = pal.palimpsa_selective_scan(*d.values())
    assert torch.equal(h, d["h0"])
    tok = {k: (v[:, 0] if k in ("x", "dt", "z", "B", "C") else v) for k, v in d.items()}
    h = d["h0"].clone()
    pal.palimpsa_selective_scan_step(tok["x"], tok["dt"], d["A"], tok["B"], tok["C"], h, d["D"], tok["z"])
    assert torch.equal(h, d["h0"])
    _status()


def test_channels_past_a_tile_add_nothing_to_the_shared_gradients():
    """40 channels fill a tile and a quarter: infinite reads of a silent token must not turn into NaN there."""
    T, D, N = 20, 40, 16
    i = _dev(_dense(_scan_inputs(13, T, 1, D, 1, N, F32, gate=False), 1))
    i["B"][0, 7, 0, 3] = float("inf")
    _, _, ck = pal.palimpsa_selective_scan_checkpointed(*i.values())
    dy = torch.ones(1, T, D, device=DEV)
    g = pal.palimpsa_selective_scan_backward(*i.values(), ck, dy)
    want = (ck[:, :1, :, 3] * 0).sum()                     # (the states before it are finite)
    assert torch.isfinite(want) and torch.isfinite(g["dC"][0, :7]).all() and torch.isfinite(g["dB"]).all()


@pytest.mark.parametrize("side", [False, True])
def test_on_a_side_stream_and_in_a_graph(side):
    """Two graphs captured from the same calls replay side by side, and a call on another stream waits for its
    inputs; both equal the plain call."""
    i = _dev(_dense(_scan_inputs(11, 2 * 520, 2, 64, 1, 16, BF), 2))      # short of channels: time is split
    w, bias = torch.randn(64, 4, device=DEV), torch.randn(64, device=DEV)
    dy = torch.randn(2, 520, 64, device=DEV).to(BF)

    def chain(stream=None):
        x, st = pal.palimpsa_causal_conv(i["x"], w, bias, stream=stream)
        y, h, ck = pal.palimpsa_selective_scan_checkpointed(*dict(i, x=x).values(), stream=stream)
        g = pal.palimpsa_selective_scan_backward(*dict(i, x=x).values(), ck, dy, stream=stream)
        c = pal.palimpsa_causal_conv_backward(i["x"], w, bias, None, g["dx"], stream=stream)
        return [y, h, st, *g.values(), *c.values()]

    want = [t.clone() for t in chain()]
    torch.cuda.synchronize()
    if side:
        s = torch.cuda.Stream()
        got = chain(s)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        return
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = chain()
        graphs.append((gr, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (gr, out), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for t in out:
                    t.zero_()
                gr.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(p, q) for p, q in zip(out, want))
    _status()


def test_graph_of_a_packed_batch_takes_new_offsets():
    """A captured run of the packed operators replays on offsets, and rows, that were written after its capture."""
    D, N, count = 136, 16, 700
    batches = [_cu(_one_long(count, 900, at)) for at in (4, 640)]
    rows = max(cu[-1] for cu in batches) + 2
    w = torch.randn(D, 4, device=DEV)
    ins = [_dev(_scan_inputs(k, rows, count, D, 1, N, F32)) for k in (1, 2)]
    cud = torch.tensor(batches[0], dtype=torch.int32, device=DEV)
    i = {k: v.clone() for k, v in ins[0].items()}
    kw = dict(cu_seqlens=cud, max_seqlen=900)

    def chain():
        u, st = pal.palimpsa_causal_conv(i["x"], w, **kw)
        y, h, ck = pal.palimpsa_selective_scan_checkpointed(*dict(i, x=u).values(), **kw)
        g = pal.palimpsa_selective_scan_backward(*dict(i, x=u).values(), ck, i["x"], **kw)
        c = pal.palimpsa_causal_conv_backward(i["x"], w, None, None, g["dx"], **kw)
        return [u, st, y, h, *g.values(), *c.values()]

    chain()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = chain()
    for cu, src in zip(batches[::-1], ins[::-1]):
        cud.copy_(torch.tensor(cu, dtype=torch.int32))
        for k, v in i.items():
            v.copy_(src[k])
        gr.replay()
        got = [t.clone() for t in out]
        assert all(torch.equal(p, q) for p, q in zip(got, chain()))
    _status()


def test_layer_prompt_then_tokens_and_training():
    """A state-space layer's middle as it is used: projection slices -> convolution -> scan over a packed prompt,
    then tokens from the states it left, against one dense pass of the oracle; and its gradients chained."""
    lens, more, D, N, W = [7, 40], 3, 48, 16, 4
    g = _gen(21)
    cu = _cu(lens)
    total = [n + more for n in lens]
    full = [_scan_inputs(30 + k, n, 1, D, 1, N, F32, state=False) for k, n in enumerate(total)]
    A, skip, bias = full[0]["A"], full[0]["D"], full[0]["dt_bias"]
    w, wb = _r(g, D, W, scale=0.5), _r(g, D)
    rows = lambda k: torch.cat([f[k][:n] for f, n in zip(full, lens)]).to(DEV)  # noqa: E731
    P = {k: v.to(DEV) for k, v in dict(A=A, skip=skip, bias=bias, w=w, wb=wb).items()}
    cud = torch.tensor(cu, dtype=torch.int32)                                    # host offsets are copied
    u, st = pal.palimpsa_causal_conv(rows("x"), P["w"], P["wb"], cu_seqlens=cud)
    y, h = pal.palimpsa_selective_scan(u, rows("dt"), P["A"], rows("B"), rows("C"), P["skip"], rows("z"), P["bias"], cu_seqlens=cud)
    out = [list(y[a:b].cpu()) for a, b in zip(cu, cu[1:])]
    for t in range(more):
        tok = lambda k: torch.stack([f[k][n + t] for f, n in zip(full, lens)]).to(DEV)  # noqa: E731,B023
        ut = pal.palimpsa_causal_conv_step(tok("x"), P["w"], P["wb"], st)
        yt = pal.palimpsa_selective_scan_step(ut, tok("dt"), P["A"], tok("B"), tok("C"), h, P["skip"], tok("z"), P["bias"])
        for k in range(2):
            out[k].append(yt[k].cpu())
    for k, f in enumerate(full):
        f = _up(f)
        u64, _ = ssm.conv(f["x"], w.to(F64), wb.to(F64), None, [0, total[k]])
        y64, h64 = ssm.scan(u64, f["dt"], A.to(F64), f["B"], f["C"], skip.to(F64), f["z"], bias.to(F64), None, [0, total[k]])
        _near(torch.stack(out[k]), y64, 1e-4, "y")
        _near(h[k], h64[0], 1e-4, "h")
    # training on the first prompt: gradients through both operators
    f, n = full[1], lens[1]
    leaf = {k: f[k][:n].to(F64).requires_grad_() for k in ("x", "dt", "B", "C", "z")}
    w64 = w.to(F64).requires_grad_()
    u64, _ = ssm.conv(leaf["x"], w64, wb.to(F64), None, [0, n])
    y64, _ = ssm.scan(u64, leaf["dt"], A.to(F64), leaf["B"], leaf["C"], skip.to(F64), leaf["z"], bias.to(F64), None, [0, n])
    dy = _r(g, n, D)
    want = torch.autograd.grad((y64 * dy.to(F64)).sum(), [leaf["x"], w64])
    d = {k: f[k][None, :n].to(DEV) for k in leaf}
    u, _ = pal.palimpsa_causal_conv(d["x"], P["w"], P["wb"])
    args = (u, d["dt"], P["A"], d["B"], d["C"], P["skip"], d["z"], P["bias"], None)
    _, _, ck = pal.palimpsa_selective_scan_checkpointed(*args)
    gs = pal.palimpsa_selective_scan_backward(*args, ck, dy[None].to(DEV))
    gc = pal.palimpsa_causal_conv_backward(d["x"], P["w"], P["wb"], None, gs["dx"])
    _near(gc["dx"][0], want[0], 1e-4, "dx")
    _near(gc["dweight"], want[1], 1e-4, "dweight")
    _status()
