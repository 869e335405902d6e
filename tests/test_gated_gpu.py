"""The gated scan on the GPU against the fp64 oracle on the same (rounded) inputs.

Bars, relative L2 per output. A value that is rounded once to the input type is off by at most half a step, 2^-8
relative in bf16. In fp32: a gate is off by at most the SFU's 2 ulp of 2^x, an ulp of the reciprocal and three
roundings, with the exponent's rounding (|u| 2^-24, |u| < 6) below 1.2e-6 relative. So is a rate w; a decay
a = e^-w by w times that and one rounding, 6e-8; an input's factor by half of that and two more. The rates here are at least
0.05 sigmoid(-5) = 3e-4 and mostly above 0.01, so that a state remembers a hundred tokens, at most a few
thousand, each adding 6e-8 + 1.2e-6 w: 1.2e-6 + 6e-8 / w, 6e-6 for w = 0.01, and 2e-4 at the very worst token of the
slowest channel. 2e-5 over all channels and tokens. Gradients go through the same decays in the other
direction and multiply both: twice that. Sums over tokens add their terms' errors, of either sign, as they
add the terms."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from oracle import ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FINE, FINE_G = 2e-5, 4e-5
TOKENS = ("x", "r", "i", "z")


def _rel(got, want):
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    d, n = float((got - want).norm()), float(want.norm())
    return d / n if n else d


def _near(got, want, bar, what=""):
    r = _rel(got, want)
    assert r <= bar, f"{what}: relative L2 {r:.3g} over {bar:.3g}"


def _r(g, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _inputs(seed, rows, n, D, dtype, gates="iz", bias=True, state=True):
    g = _gen(seed)
    return dict(x=_r(g, rows, D, dtype=dtype), r=_r(g, rows, D, dtype=dtype), A=0.05 + 1.5 * torch.rand((D,), generator=g) ** 2,
                i=_r(g, rows, D, dtype=dtype) if "i" in gates else None, z=_r(g, rows, D, dtype=dtype) if "z" in gates else None,
                r_bias=_r(g, D, scale=0.5) if bias else None, i_bias=_r(g, D, scale=0.5) if bias and "i" in gates else None,
                h0=_r(g, n, D) if state else None)


def _up(d):
    return {k: None if v is None else v.to(F64) for k, v in d.items()}


def _dev(d):
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}


def _dense(i, B):
    return {k: v.reshape(B, -1, v.shape[-1]) if v is not None and k in TOKENS else v for k, v in i.items()}


def _status():
    assert pal.palimpsa_get_device_status() == 0


NAMES = (("dx", "x"), ("dr", "r"), ("di", "i"), ("dz", "z"))
PARAMS = (("dA", "A"), ("dr_bias", "r_bias"), ("di_bias", "i_bias"), ("dh0", "h0"))


def _case(dtype, lens, dense, D, gates="iz", bias=True, state=True, tail=0, inputs=None, scale=1.0):
    n, cu = len(lens), _cu(lens)
    rows = cu[-1] + tail
    i = inputs or _inputs(rows + D, rows, n, D, dtype, gates, bias, state)
    g = _gen(7)
    dy, dl = _r(g, rows, D, dtype=dtype), _r(g, n, D)
    y, last, grads = ssm.gradients(ssm.gate, _up(i), dy.to(F64), dl.to(F64), cu)
    kw = {} if dense else dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=max(lens))
    d = _dev(_dense(i, n) if dense else i)
    gdy = (dy.reshape(n, -1, D) if dense else dy).to(DEV)
    gy, gh = pal.palimpsa_gated_scan(*d.values(), **kw)
    cy, ch, ckpt = pal.palimpsa_gated_scan_checkpointed(*d.values(), **kw)
    assert torch.equal(gy, cy) and torch.equal(gh, ch)
    _near(gy.reshape(-1, D), y, HALF[dtype] + scale * FINE, "y")
    _near(gh, last, scale * FINE, "h_T")
    args = list(d.values())[:-1]
    got = pal.palimpsa_gated_scan_backward(*args, ckpt, gdy, dl.to(DEV), **kw)
    again = pal.palimpsa_gated_scan_backward(*args, ckpt, gdy, dl.to(DEV), **kw)
    for k, v in got.items():
        assert torch.equal(v, again[k]), f"{k} differs from run to run"
    assert ("di" in got) == ("di_bias" in got) == ("i" in gates) and ("dz" in got) == ("z" in gates)
    for k, name in NAMES:
        if k in got:
            _near(got[k].reshape(-1, D), grads[name], HALF[dtype] + scale * FINE_G, k)
    for k, name in PARAMS:
        if k in got and name in grads:
            _near(got[k], grads[name], scale * FINE_G, k)
    _status()
    return got, grads


# From one token on, around the pieces of 8 tokens and the tiles of 64 (32 in fp32) and 64 channels, and lengths that
# clusters of every size share.
SHAPES = [(1, 1, 8), (2, 7, 64), (3, 8, 72), (1, 9, 128), (2, 31, 136), (1, 33, 64), (2, 63, 8), (1, 65, 200), (2, 130, 64),
          (1, 200, 72), (1, 515, 64), (1, 1500, 40), (1, 2100, 64), (2, 3500, 24), (64, 70, 512), (200, 33, 320), (3, 300, 1024)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("gates,bias,state", [("iz", True, True), ("", False, False)])
def test_dense(dtype, B, T, D, gates, bias, state):
    _case(dtype, [T] * B, True, D, gates, bias, state)


# Short sequences, many of them: a thread (backward: a warp) walks each.
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", [(700, 1, 72), (300, 3, 8), (300, 8, 264), (200, 9, 520), (500, 20, 136)])
@pytest.mark.parametrize("gates,bias,state", [("iz", True, True), ("", False, False), ("z", True, True), ("i", False, False)])
def test_many_short(dtype, B, T, D, gates, bias, state):
    _case(dtype, [T] * B, True, D, gates, bias, state)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_short_packed(dtype):
    _case(dtype, [(5, 0, 1, 8, 17, 2)[k % 6] for k in range(900)], False, 200, tail=3)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_short_with_bad_offsets(dtype):
    """One sequence among hundreds is longer than max_seqlen, the last ends past the rows: both are skipped."""
    lens = [(4, 1, 7, 2)[k % 4] for k in range(600)]
    lens[300] = 9
    D, cu = 136, _cu(lens)
    rows, ok = cu[-1] - 1, [k not in (300, 599) for k in range(600)]
    i = _inputs(3, rows, 600, D, dtype)
    dy = _r(_gen(5), rows, D, dtype=dtype)
    keep = torch.zeros(rows, dtype=torch.bool)
    for n in range(600):
        if ok[n]:
            keep[cu[n]:cu[n + 1]] = True
    okt = torch.tensor(ok)
    pick = lambda v: (v[keep] if v.shape[0] == rows else v[okt] if v.shape[0] == 600 else v).to(F64)  # noqa: E731
    cug = _cu([n for n, fine in zip(lens, ok) if fine])
    y, last, want = ssm.gradients(ssm.gate, {k: pick(v) for k, v in i.items()}, pick(dy), torch.zeros(598, D, dtype=F64), cug)
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=8)
    h = torch.full((600, D), 7.0, device=DEV)
    gy, _, ckpt = pal.palimpsa_gated_scan_checkpointed(*_dev(i).values(), h_T=h, **kw)
    assert pal.palimpsa_get_device_status() == 5
    g = pal.palimpsa_gated_scan_backward(*list(_dev(i).values())[:-1], ckpt, dy.to(DEV), **kw)
    assert pal.palimpsa_get_device_status() == 5
    _near(gy[keep], y, HALF[dtype] + FINE, "y")
    _near(h[okt], last, FINE, "h_T")
    assert (h[~okt] == 7).all() and not gy[~keep].any()
    for k, name in NAMES:
        _near(g[k][keep], want[name], HALF[dtype] + FINE_G, k)
        assert not g[k][~keep].any()
    for k, name in PARAMS[:3]:
        _near(g[k], want[name], FINE_G, k)
    _near(g["dh0"][okt], want["h0"], FINE_G, "dh0")
    assert not g["dh0"][~okt].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gates,bias,state", [("i", True, False), ("z", False, True), ("i", False, True), ("z", True, False)])
@pytest.mark.parametrize("B,T,D", [(2, 75, 72), (1, 300, 64), (80, 70, 512)])
def test_options(dtype, gates, bias, state, B, T, D):
    _case(dtype, [T] * B, True, D, gates, bias, state)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[5, 0, 1, 130, 16, 3], [0], [0, 0, 7], [400, 3, 1, 129], [32, 16, 48], [8] * 50 + [700],
                                  [1] * 300])
@pytest.mark.parametrize("D", [8, 136])
def test_packed(dtype, lens, D):
    _case(dtype, lens, False, D, tail=2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_many_channels(dtype):
    """CTAs enough that no sequence is shared by several."""
    _case(dtype, [70, 0, 130, 1, 33] * 12, False, 1024, tail=3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("at", [0, 333, 599])
def test_packed_one_long(dtype, at):
    _case(dtype, [900 if k == at else (0, 1, 3, 2)[k % 4] for k in range(600)], False, 40, tail=2)


def test_rows_outside_the_sequences():
    """Rows behind the last sequence stay as they were in outputs that are given, and are zero in fresh ones."""
    lens, D, tail = [5, 40], 72, 4
    i = _dev(_inputs(3, 45 + tail, 2, D, BF))
    kw = dict(cu_seqlens=torch.tensor(_cu(lens), dtype=torch.int32, device=DEV), max_seqlen=40)
    mine = torch.full((45 + tail, D), 7.0, dtype=BF, device=DEV)
    y, _, ckpt = pal.palimpsa_gated_scan_checkpointed(*i.values(), y=mine, **kw)
    fresh, _ = pal.palimpsa_gated_scan(*i.values(), **kw)
    assert (mine[45:] == 7).all() and not fresh[45:].any() and torch.equal(fresh[:45], y[:45])
    g = pal.palimpsa_gated_scan_backward(*list(i.values())[:-1], ckpt, mine, **kw)
    for k in ("dx", "dr", "di", "dz"):
        assert not g[k][45:].any()
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_offsets(dtype):
    """A sequence that ends past the rows is skipped, and one that is longer than max_seqlen; the others are right."""
    lens = [20, 300, 41, 9, 50]
    D, cu = 72, _cu(lens)
    rows = cu[-1] - 5
    i = _inputs(3, rows, 5, D, dtype)
    dy = _r(_gen(5), rows, D, dtype=dtype)
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=300)
    keep = torch.zeros(rows, dtype=torch.bool)
    for n in (0, 1, 2, 3):
        keep[cu[n]:cu[n + 1]] = True
    pick = lambda v, s: (v[keep] if v.shape[0] == rows else v[s] if v.shape[0] == 5 else v).to(F64)  # noqa: E731
    live = torch.tensor([True, True, True, True, False])
    sub = {k: pick(v, live) for k, v in i.items()}
    y, last, want = ssm.gradients(ssm.gate, sub, dy[keep].to(F64), torch.zeros(4, D, dtype=F64), cu[:5])
    h = torch.full((5, D), 7.0, device=DEV)
    gy, _, ckpt = pal.palimpsa_gated_scan_checkpointed(*_dev(i).values(), h_T=h, **kw)
    assert pal.palimpsa_get_device_status() == 5
    g = pal.palimpsa_gated_scan_backward(*list(_dev(i).values())[:-1], ckpt, dy.to(DEV), **kw)
    assert pal.palimpsa_get_device_status() == 5
    _near(gy[keep], y, HALF[dtype] + FINE, "y")
    _near(h[live], last, FINE, "h_T")
    assert (h[4] == 7).all() and not gy[~keep].any()
    for k, name in NAMES:
        _near(g[k][keep], want[name], HALF[dtype] + FINE_G, k)
        assert not g[k][~keep].any()
    for k, name in PARAMS[:3]:
        _near(g[k], want[name], FINE_G, k)
    _near(g["dh0"][live], want["h0"], FINE_G, "dh0")
    assert not g["dh0"][4].any()
    # Too long for max_seqlen: the second sequence alone is skipped.
    kw["max_seqlen"] = 299
    y2, h2 = pal.palimpsa_gated_scan(*_dev(i).values(), **kw)
    assert pal.palimpsa_get_device_status() == 5
    assert not y2[20:320].any() and not h2[1].any() and torch.equal(y2[320:361], gy[320:361])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,cut", [(21, 9), (300, 64), (70, 69)])
def test_steps_continue_a_prompt(dtype, T, cut):
    """A prompt, then tokens one by one, in place, against the whole sequence (two orders of the same sums)."""
    B, D = 3, 72
    i = _dev(_dense(_inputs(3, B * T, B, D, dtype), B))
    y, last = pal.palimpsa_gated_scan(*i.values())
    h = i["h0"].clone()
    part = {k: v[:, :cut].contiguous() if k in TOKENS else v for k, v in i.items()}
    y1, h1 = pal.palimpsa_gated_scan(*dict(part, h0=h).values(), h_T=h)
    assert h1 is h
    ys = [y1]
    for t in range(cut, T):
        a = [i[k][:, t] for k in ("x", "r")]
        ys.append(pal.palimpsa_gated_scan_step(*a, i["A"], h, i["i"][:, t], i["z"][:, t], i["r_bias"], i["i_bias"])[:, None])
    _near(torch.cat(ys, 1), y.cpu(), 2 * HALF[dtype] + 2 * FINE)
    _near(h, last.cpu(), 2 * FINE)
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,D", [(1, 8), (3, 72), (256, 2048), (1, 4096)])
@pytest.mark.parametrize("gates", ["iz", "i", "z", ""])
def test_step(dtype, B, D, gates):
    i = _inputs(B + D, B, B, D, dtype, gates)
    y, last = ssm.gate(*_up(i).values(), list(range(B + 1)))
    d = _dev(i)
    got = pal.palimpsa_gated_scan_step(d["x"], d["r"], d["A"], d["h0"], d["i"], d["z"], d["r_bias"], d["i_bias"])
    _near(got, y, HALF[dtype] + 3e-6)     # one token: a gate's 1.2e-6, the root's half of it, four roundings
    _near(d["h0"], last, 3e-6)
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_wider_projections(dtype):
    """x, r, i, z and dy as slices of one projection give the bits of dense copies."""
    B, T, D = 2, 77, 72
    wide = _r(_gen(4), B, T, 5 * D, dtype=dtype).to(DEV)
    x, r, i, z, dy = (wide[..., k * D:(k + 1) * D] for k in range(5))
    g = _gen(5)
    A, rb, ib, h0 = (0.1 + torch.rand(D, generator=g)).to(DEV), _r(g, D).to(DEV), _r(g, D).to(DEV), _r(g, B, D).to(DEV)
    res = []
    for f in (lambda t: t, lambda t: t.contiguous()):
        y, h, ckpt = pal.palimpsa_gated_scan_checkpointed(f(x), f(r), A, f(i), f(z), rb, ib, h0)
        gr = pal.palimpsa_gated_scan_backward(f(x), f(r), A, f(i), f(z), rb, ib, ckpt, f(dy))
        hs = h0.clone()
        ys = pal.palimpsa_gated_scan_step(f(x[:, 3]), f(r[:, 3]), A, hs, f(i[:, 3]), f(z[:, 3]), rb, ib)
        res.append([y, h, *gr.values(), ys, hs])
    for a, b in zip(*res):
        assert torch.equal(a, b)
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates_far_out(dtype):
    """Gates wide open and shut (raw values to +-200), slow and fast channels: nothing overflows, and outputs and
    gradients agree with 64 bits relative to their channel."""
    T, D = 150, 64
    i = _inputs(11, T, 1, D, dtype)
    g = _gen(12)
    for k in ("r", "i", "z"):
        far = torch.tensor([-200.0, -90.0, -30.0, 0.0, 30.0, 90.0, 200.0])
        i[k] = (far[torch.randint(0, 7, (T, D), generator=g)] + _r(g, T, D)).to(dtype)
    i["A"] = torch.logspace(-6, 3, D)
    dy = _r(g, T, D, dtype=dtype)
    y, last, grads = ssm.gradients(ssm.gate, _up(i), dy.to(F64), None, [0, T])
    d = _dev(_dense(i, 1))
    gy, gh, ckpt = pal.palimpsa_gated_scan_checkpointed(*d.values())
    got = pal.palimpsa_gated_scan_backward(*list(d.values())[:-1], ckpt, dy[None].to(DEV))
    # Gates that are shut to within 1e-30 are worth nothing beside those that are open, in every channel.
    _near(gy[0], y, HALF[dtype] + FINE, "y")
    _near(gh, last, FINE, "h_T")
    for k, name in NAMES:
        _near(got[k][0], grads[name], HALF[dtype] + FINE_G, k)
    for k, name in PARAMS:
        _near(got[k], grads[name], FINE_G, k)
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_channels_that_hardly_forget(dtype):
    """Rates down to 1e-12: 1 - a^2 is 2 w to the last digit, though a is 1 in fp32. A state's own rounding, 6e-8 a token over 300
    tokens, stays below 300 x 6e-8 = 1.8e-5 of it."""
    T, D = 300, 64
    i = _inputs(61, T, 1, D, dtype, state=False)
    i["A"] = torch.logspace(-12, -3, D)
    _case(dtype, [T], True, D, state=False, inputs=i)


@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf")])
def test_rates_out_of_range_are_latched(bad):
    i = _dev(_dense(_inputs(1, 20, 2, 72, F32), 2))
    i["A"][50] = bad
    pal.palimpsa_gated_scan(*i.values())
    assert pal.palimpsa_get_device_status() == 5
    pal.palimpsa_gated_scan_step(i["x"][:, 0], i["r"][:, 0], i["A"], i["h0"], i["i"][:, 0], i["z"][:, 0])
    assert pal.palimpsa_get_device_status() == 5
    ckpt = torch.zeros(pal.palimpsa_gated_scan_checkpoint_shape(2, 10, 72), device=DEV)
    pal.palimpsa_gated_scan_backward(*list(i.values())[:-1], ckpt, i["x"])
    assert pal.palimpsa_get_device_status() == 5


def test_a_nan_stays_in_its_sequence_and_channel():
    i = _dev(_dense(_inputs(2, 3 * 200, 3, 72, F32), 3))
    clean, _ = pal.palimpsa_gated_scan(*i.values())
    i["x"][1, 70, 5] = float("nan")
    y, h = pal.palimpsa_gated_scan(*i.values())
    assert torch.isnan(y[1, 70:, 5]).all() and torch.isnan(h[1, 5])
    y[1, 70:, 5] = clean[1, 70:, 5]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("T", [0, 5])
def test_empty_batches(T):
    """No tokens: the state and its gradient pass through, the parameters' gradients are 0."""
    D, B = 72, 2
    e = torch.empty(B, 0, D, device=DEV)
    if T:   # packed: rows, but none in a sequence
        e = torch.ones(T, D, device=DEV)
    kw = dict(cu_seqlens=torch.zeros(B + 1, dtype=torch.int32, device=DEV), max_seqlen=0) if T else {}
    A, h0, dl = torch.ones(D, device=DEV), torch.randn(B, D, device=DEV), torch.randn(B, D, device=DEV)
    y, h, ckpt = pal.palimpsa_gated_scan_checkpointed(e, e, A, e, e, A, A, h0, **kw)
    assert torch.equal(h, h0) and not y.any()
    g = pal.palimpsa_gated_scan_backward(e, e, A, e, e, A, A, ckpt, e, dl, **kw)
    assert torch.equal(g["dh0"], dl) and not any(g[k].any() for k in g if k != "dh0")
    _status()


def test_gradients_against_differences_of_the_kernels():
    """The kernels' own fp32 forward, differenced along random directions: the step 2e-3 leaves 1e-6 of third
    derivatives, and outputs of 1 that are 1e-6 off leave 1e-6 / 4e-3 = 3e-4 an element, their random sum over
    B T D = 4000 elements 60 times that, 0.02, on derivatives of about sqrt(4000) = 60."""
    B, T, D = 2, 50, 40
    i = _dev(_dense(_inputs(21, B * T, B, D, F32), B))
    g = torch.Generator(device=DEV).manual_seed(22)
    dy, dl = torch.randn(B, T, D, generator=g, device=DEV), torch.randn(B, D, generator=g, device=DEV)
    _, _, ckpt = pal.palimpsa_gated_scan_checkpointed(*i.values())
    got = pal.palimpsa_gated_scan_backward(*list(i.values())[:-1], ckpt, dy, dl)

    def loss(d):
        y, h = pal.palimpsa_gated_scan(*d.values())
        return float((y.double() * dy).sum() + (h.double() * dl).sum())

    for k, name in NAMES + PARAMS:
        way = torch.randn(i[name].shape, generator=g, device=DEV)
        e = 2e-3 * (0.02 if name == "A" else 1.0)
        hi, lo = dict(i, **{name: i[name] + e * way}), dict(i, **{name: i[name] - e * way})
        d = (loss(hi) - loss(lo)) / (2 * e)
        want = float((got[k].double() * way).sum())
        assert abs(d - want) <= 0.05 * (50 if name == "A" else 1) + 1e-3 * abs(want), k


def test_long_memory_beyond_32_bits():
    """More than 2^31 elements of a token array: the last channels of the last sequence are right."""
    B, T, D = 3, 131072, 8192      # 3.2e9 elements, 6.4 GB of bf16 an array
    x = torch.empty(B, T, D, dtype=BF, device=DEV)
    r = torch.empty(B, T, D, dtype=BF, device=DEV)
    x.zero_()
    r.zero_()
    last = slice(D - 64, D)
    g = _gen(1)
    xs, rs = _r(g, 300, 64, dtype=BF), _r(g, 300, 64, dtype=BF)
    x[-1, -300:, last], r[-1, -300:, last] = xs.to(DEV), rs.to(DEV)
    A = torch.full((D,), 0.5, device=DEV)
    y, h = pal.palimpsa_gated_scan(x, r, A)
    wy, wh = ssm.gate(xs.to(F64), rs.to(F64), torch.full((64,), 0.5, dtype=F64), None, None, None, None, None, [0, 300])
    _near(y[-1, -300:, last], wy, HALF[BF] + FINE)
    _near(h[-1:, last], wh, FINE)
    assert not y[:-1].any() and not y[-1, :-300].any()
    _status()


def test_gradients_beyond_32_bits():
    """The same, backward: rows, checkpoints and gradients past 2^31 elements of an array."""
    B, T, D = 3, 131072, 8192
    x, r, dy = (torch.zeros(B, T, D, dtype=BF, device=DEV) for _ in range(3))
    last = slice(D - 64, D)
    g = _gen(2)
    xs, rs, ds = (_r(g, 300, 64, dtype=BF) for _ in range(3))
    for t, v in ((x, xs), (r, rs), (dy, ds)):
        t[-1, -300:, last] = v.to(DEV)
    A = torch.full((D,), 0.5, device=DEV)
    ckpt = pal.palimpsa_gated_scan_checkpointed(x, r, A)[2]
    got = pal.palimpsa_gated_scan_backward(x, r, A, None, None, None, None, ckpt, dy)
    i = dict(x=xs, r=rs, A=torch.full((64,), 0.5), i=None, z=None, r_bias=None, i_bias=None, h0=None)
    want = ssm.gradients(ssm.gate, _up(i), ds.to(F64), torch.zeros(1, 64, dtype=F64), [0, 300])[2]
    for k in ("dx", "dr"):
        _near(got[k][-1, -300:, last], want[k[1:]], HALF[BF] + FINE_G, k)
        assert not got[k][:-1].any() and not got[k][-1, :, :D - 64].any()
    _near(got["dA"][last], want["A"], FINE_G, "dA")     # (x and h are 0 in front of the last 300 tokens)
    assert not got["dA"][:D - 64].any()
    _status()


def test_captured_and_replayed():
    """A training pass in a CUDA graph, replayed on new inputs and new offsets."""
    D, rows = 72, 500
    i = _dev(_inputs(31, rows, 4, D, BF))
    cu = torch.tensor([0, 100, 101, 300, 500], dtype=torch.int32, device=DEV)
    dy, dl = torch.randn(rows, D, device=DEV).bfloat16(), torch.randn(4, D, device=DEV)
    kw = dict(cu_seqlens=cu, max_seqlen=400)

    def both():
        y, h, ckpt = pal.palimpsa_gated_scan_checkpointed(*i.values(), **kw)
        return [y, h, *pal.palimpsa_gated_scan_backward(*list(i.values())[:-1], ckpt, dy, dl, **kw).values()]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    new = _dev(_inputs(32, rows, 4, D, BF))
    for k, v in new.items():
        i[k].copy_(v)
    cu.copy_(torch.tensor([0, 7, 400, 400, 499], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, both()):
        assert torch.equal(a, b)
    _status()


def test_two_streams_at_once():
    side = torch.cuda.Stream()
    a, b = (_dev(_dense(_inputs(s, 4 * 700, 4, 520, BF), 4)) for s in (41, 42))
    dy = a["z"].clone()

    def run(i, **kw):
        y, h, ckpt = pal.palimpsa_gated_scan_checkpointed(*i.values(), **kw)
        return [y, h, *pal.palimpsa_gated_scan_backward(*list(i.values())[:-1], ckpt, dy, **kw).values()]

    want = run(a), run(b)
    for _ in range(5):
        got = run(a, stream=side), run(b)
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for p, q in zip(w, g):
                assert torch.equal(p, q)
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_state_that_is_not_handed_on_times_out(dtype):
    """One long sequence, shared by a cluster whose first CTA withholds its first state (gradient): the others' bounded
    waits run out, the kernels latch PALIMPSA_ERR_TIMEOUT and end, and later calls work."""
    i = _dev(_dense(_inputs(51, 1500, 1, 64, dtype), 1))
    want = pal.palimpsa_gated_scan_checkpointed(*i.values())
    args = list(i.values())[:-1]
    grads = pal.palimpsa_gated_scan_backward(*args, want[2], i["x"])
    _status()
    pal.palimpsa_set_wait_timeout_ns(2_000_000)
    pal.palimpsa_debug_withhold_first_copy(True)
    try:
        pal.palimpsa_gated_scan(*i.values())
        assert pal.palimpsa_get_device_status() == 8
        pal.palimpsa_gated_scan_backward(*args, want[2], i["x"])
        assert pal.palimpsa_get_device_status() == 8
    finally:
        pal.palimpsa_debug_withhold_first_copy(False)
        pal.palimpsa_set_wait_timeout_ns(2_000_000_000)
    for a, b in zip(want, pal.palimpsa_gated_scan_checkpointed(*i.values())):
        assert torch.equal(a, b)
    again = pal.palimpsa_gated_scan_backward(*args, want[2], i["x"])
    for k in grads:
        assert torch.equal(grads[k], again[k])
    _status()
