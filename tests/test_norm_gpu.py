"""The layer norm on the GPU against the fp64 oracle on the same (rounded) inputs.

Bars, relative L2 per output. An output of the input type is rounded once: half a step, 2^-8 relative in bf16. In
fp32: a mean is a sum of 8 values in turn, of 32 lanes in 5 steps and of at most 16 warps: 29 roundings of 2^-24, 1.7e-6 of
the mean absolute value, which here is at most 5 deviations: 9e-6 of a deviation; the squares likewise, relative to
themselves. Half of that remains in 1 / deviation, and y adds four roundings: 1.2e-5 with everything at its worst. The
gradient's two means are such sums of terms that are themselves 2e-6 off (and cancel nothing): 2.4e-5. Sums over rows: up to
2000 terms of either sign, each off by 1.2e-5: 3e-5 relative to their norm."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from oracle import ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FINE, FINE_G = 1.2e-5, 3e-5


def _near(got, want, bar, what=""):
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert got.shape == want.shape and torch.isfinite(got).all()
    d, n = float((got - want).norm()), float(want.norm())
    assert (d / n if n else d) <= bar, f"{what}: relative L2 {d / n if n else d:.3g} over {bar:.3g}"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _r(g, *shape, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def _inputs(seed, rows, D, dtype, residual=True, affine=True):
    g = _gen(seed)
    off = 2 * torch.randn((rows, 1), generator=g)          # rows off centre by up to some deviations
    return dict(x=(_r(g, rows, D) + off).to(dtype), weight=1 + _r(g, D, scale=0.3) if affine else None,
                bias=_r(g, D) if affine else None, residual=_r(g, rows, D, dtype=dtype, scale=2.0) if residual else None,
                dy=_r(g, rows, D, dtype=dtype), ds=_r(g, rows, D, dtype=dtype))


def _dev(d):
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}


def _up(v):
    return None if v is None else v.to(F64)


def _oracle(i, eps, with_ds):
    s = i["x"] if i["residual"] is None else (i["x"].float() + i["residual"].float()).to(i["x"].dtype)
    leaves = [None if v is None else v.to(F64).requires_grad_() for v in (s, i["weight"], i["bias"])]
    y = ssm.layer_norm(*leaves, eps)
    loss = (y * _up(i["dy"])).sum() + ((leaves[0] * _up(i["ds"])).sum() if with_ds else 0)
    some = [v for v in leaves if v is not None]
    got = iter(torch.autograd.grad(loss, some))
    return s, y.detach(), [None if v is None else next(got) for v in leaves]


def _case(rows, D, dtype, residual, affine, with_ds, eps=1e-5, shape=None):
    i = _inputs(rows + D, rows, D, dtype, residual, affine)
    s, y, (ds, dw, db) = _oracle(i, eps, with_ds)
    d = _dev(i)
    if shape:
        d = {k: v.reshape(*shape, D) if v is not None and v.dim() == 2 else v for k, v in d.items()}
    gy, gs, st = pal.palimpsa_layer_norm(d["x"], d["weight"], d["bias"], d["residual"], eps=eps, want_stats=True)
    assert torch.equal(gs.reshape(-1, D).cpu(), s) and (residual or gs is d["x"])
    plain, _, none = pal.palimpsa_layer_norm(d["x"], d["weight"], d["bias"], d["residual"], eps=eps)
    assert none is None and torch.equal(plain, gy)
    _near(gy.reshape(-1, D), y, HALF[dtype] + FINE, "y")
    su = s.to(F64)
    _near(st.reshape(-1, 2)[:, 0], su.mean(1), FINE, "mean")
    _near(st.reshape(-1, 2)[:, 1], (su.var(1, unbiased=False) + eps).rsqrt(), FINE, "1 / deviation")
    args = (gs, d["weight"], st, d["dy"], d["ds"] if with_ds else None)
    g = pal.palimpsa_layer_norm_backward(*args)
    again = pal.palimpsa_layer_norm_backward(*args)
    assert ("dweight" in g) == affine and "dbias" in g
    for k in g:
        assert torch.equal(g[k], again[k]), f"{k} differs from run to run"
    _near(g["dx"].reshape(-1, D), ds, HALF[dtype] + FINE_G, "dx")
    if affine:
        _near(g["dweight"], dw, FINE_G, "dweight")
        _near(g["dbias"], db, FINE_G, "dbias")
    else:
        _near(g["dbias"], i["dy"].to(F64).sum(0), FINE_G, "dbias")


# Widths around the teams' limits.
WIDTHS = [8, 16, 24, 32, 56, 64, 72, 96, 104, 128, 136, 192, 200, 248, 256, 264, 384, 392, 512, 520, 768, 776, 1024, 1032, 1536,
          1544, 2048, 2056, 4088, 4096, 4104, 6152, 8192]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("residual,affine,with_ds", [(True, True, True), (False, True, False)])
def test_widths(dtype, D, residual, affine, with_ds):
    if D == 8 and not affine:
        return
    _case(37, D, dtype, residual, affine, with_ds)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 2, 3, 31, 33, 129, 2000])
@pytest.mark.parametrize("D", [64, 200, 520])
@pytest.mark.parametrize("residual,affine,with_ds", [(True, False, False), (False, False, True), (True, True, True)])
def test_rows(dtype, rows, D, residual, affine, with_ds):
    _case(rows, D, dtype, residual, affine, with_ds)


@pytest.mark.parametrize("shape", [(1, 1), (2, 3, 4), (5, 7), (2, 3, 2, 5)])
def test_leading_dimensions(shape):
    _case(torch.Size(shape).numel(), 72, F32, True, True, True, shape=shape)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,D", [(60001, 72), (120001, 16), (60001, 64), (30001, 264), (20001, 520), (20001, 1024), (5001, 2056),
                                    (5001, 4104)])
def test_many_rows(dtype, rows, D):
    """More rows than the GPU's CTAs hold at once: every CTA walks several batches. Against torch in 64 bits on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x, dy = (torch.randn(rows, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    w, b = torch.rand(D, generator=g, device=DEV) + 0.5, torch.randn(D, generator=g, device=DEV)
    y, s, st = pal.palimpsa_layer_norm(x, w, b, want_stats=True)
    got = pal.palimpsa_layer_norm_backward(s, w, st, dy)
    lx, lw, lb = (t.double().requires_grad_() for t in (x, w, b))
    want = torch.nn.functional.layer_norm(lx, (D,), lw, lb, 1e-5)
    grads = torch.autograd.grad(want, (lx, lw, lb), dy.double())
    _near(y, want.detach().cpu(), HALF[dtype] + FINE, "y")
    for k, v, bar in zip(("dx", "dweight", "dbias"), grads, (HALF[dtype] + FINE_G, FINE_G, FINE_G)):
        _near(got[k], v.cpu(), bar, k)


@pytest.mark.parametrize("D", [64, 256, 1536, 8192])
def test_rows_far_off_centre(D):
    """Rows around 1000 with a deviation of 1: fp32 inputs are 1000 +- 2^-15 exact, so their deviations are; a mean's 29
    roundings at 1000, 2^-24 each, are 1.7e-3 of a deviation in the worst case, and its error e changes the squares about it
    only by e^2. Where squares and mean were subtracted, 1e6 2^-24 = 0.06 would be lost."""
    g = _gen(D)
    x = 1000 + _r(g, 33, D)
    y, _, st = pal.palimpsa_layer_norm(x.to(DEV), want_stats=True)
    _near(y, ssm.layer_norm(x.to(F64), None, None, 1e-5), 1.7e-3)
    _near(st[:, 1], (x.to(F64).var(1, unbiased=False) + 1e-5).rsqrt(), FINE)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 520])
def test_constant_rows(dtype, D):
    """A row without a deviation: y is the bias, and its gradient is that of eps alone."""
    x = torch.full((3, D), 1.5, dtype=dtype, device=DEV)
    b = torch.randn(D, device=DEV)
    y, _, st = pal.palimpsa_layer_norm(x, None, b, want_stats=True)
    assert torch.equal(y, b.to(dtype).expand(3, D))
    _near(st[:, 1], torch.full((3,), 1e-5, dtype=F64).rsqrt(), 2e-7)
    dy = torch.randn(3, D, device=DEV).to(dtype)
    g = pal.palimpsa_layer_norm_backward(x, None, st, dy)
    dyu = dy.double().cpu()
    _near(g["dx"], (dyu - dyu.mean(1, keepdim=True)) / 1e-5 ** 0.5, HALF[dtype] + FINE)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 200, 520])
def test_a_row_with_infinity_or_nan_spoils_no_other(dtype, D):
    i = _dev(_inputs(5, 40, D, dtype))
    want, _, _ = pal.palimpsa_layer_norm(i["x"], i["weight"], i["bias"])
    i["x"][7, 3], i["x"][20, 0] = float("inf"), float("nan")
    y, s, st = pal.palimpsa_layer_norm(i["x"], i["weight"], i["bias"], want_stats=True)
    ok = torch.ones(40, dtype=torch.bool)
    ok[7] = ok[20] = False
    assert torch.equal(y[ok], want[ok]) and not torch.isfinite(y[~ok]).all(1).any()
    g = pal.palimpsa_layer_norm_backward(s, i["weight"], st, i["dy"])
    assert torch.isfinite(g["dx"][ok]).all() and torch.isfinite(g["dbias"]).all()


@pytest.mark.parametrize("D", [64, 200, 1536, 4104])
def test_deviations_past_the_range_of_their_squares(D):
    """Deviations of 1e30: their squares overflow, and y is the bias; the rows beside it are as ever."""
    x = _r(_gen(D), 5, D).to(DEV)
    w, b = torch.rand(D, device=DEV), torch.randn(D, device=DEV)
    want, _, _ = pal.palimpsa_layer_norm(x, w, b)
    x[2] *= 1e30
    y, _, st = pal.palimpsa_layer_norm(x, w, b, want_stats=True)
    assert torch.equal(y[2], b) and st[2, 1] == 0
    y[2] = want[2]
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 520])
def test_rows_of_wider_rows_and_in_place(dtype, D):
    wide = _r(_gen(8), 3, 20, 4 * D, dtype=dtype).to(DEV)
    x, res, dy, ds = (wide[..., k * D:(k + 1) * D] for k in range(4))
    w, b = torch.rand(D, device=DEV), torch.rand(D, device=DEV)
    y, s, st = pal.palimpsa_layer_norm(x, w, b, res, want_stats=True)
    y2, s2, st2 = pal.palimpsa_layer_norm(x.contiguous(), w, b, res.contiguous(), want_stats=True)
    assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(st, st2)
    for given in ("x", "residual"):
        d = dict(x=x.contiguous(), residual=res.contiguous())
        y3, s3, _ = pal.palimpsa_layer_norm(d["x"], w, b, d["residual"], s=d[given])
        assert s3 is d[given] and torch.equal(s3, s) and torch.equal(y3, y)
    g = pal.palimpsa_layer_norm_backward(s, w, st, dy, ds)
    for given in range(2):
        a = [dy.contiguous(), ds.contiguous()]
        h = pal.palimpsa_layer_norm_backward(s, w, st, *a, dx=a[given])
        assert h["dx"] is a[given]
        for k in g:
            assert torch.equal(g[k], h[k])


def test_beyond_32_bits():
    """More than 2^31 elements of an array: the last rows are those of a small call."""
    D, some = 1024, 5
    rows = 2 ** 31 // D + some
    i = _dev(_inputs(7, some, D, BF))
    big = {}
    for k in ("x", "residual", "dy"):
        big[k] = torch.zeros(rows, D, dtype=BF, device=DEV)
        big[k][-some:] = i[k]
    y, s, stats = pal.palimpsa_layer_norm(big["x"], i["weight"], i["bias"], big["residual"], want_stats=True)
    wy, ws, wstats = pal.palimpsa_layer_norm(i["x"], i["weight"], i["bias"], i["residual"], want_stats=True)
    assert torch.equal(y[-some:], wy) and torch.equal(s[-some:], ws) and torch.equal(stats[-some:], wstats)
    assert torch.equal(y[0], i["bias"].bfloat16()) and torch.equal(y[-some - 1], y[0])
    g = pal.palimpsa_layer_norm_backward(s, i["weight"], stats, big["dy"])
    w = pal.palimpsa_layer_norm_backward(ws, i["weight"], wstats, i["dy"])
    assert torch.equal(g["dx"][-some:], w["dx"]) and not g["dx"][:-some].any()
    for k in ("dweight", "dbias"):
        _near(g[k], w[k].cpu(), FINE_G, k)


def test_no_rows():
    x, w = torch.empty(0, 72, device=DEV), torch.ones(72, device=DEV)
    y, s, st = pal.palimpsa_layer_norm(x, w, w, x, want_stats=True)
    assert y.shape == s.shape == (0, 72) and st.shape == (0, 2)
    g = pal.palimpsa_layer_norm_backward(s, w, st, x)
    assert not g["dweight"].any() and not g["dbias"].any()


def test_only_the_gradients_that_are_wanted():
    i = _dev(_inputs(9, 20, 72, F32))
    y, s, st = pal.palimpsa_layer_norm(i["x"], i["weight"], None, want_stats=True)
    full = pal.palimpsa_layer_norm_backward(s, i["weight"], st, i["dy"])
    for kw, keys in ((dict(want_bias_grad=False), {"dx", "dweight"}), (dict(want_weight_grad=False), {"dx", "dbias"}),
                     (dict(want_weight_grad=False, want_bias_grad=False), {"dx"})):
        g = pal.palimpsa_layer_norm_backward(s, i["weight"], st, i["dy"], **kw)
        assert g.keys() == keys
        for k in keys:
            assert torch.equal(g[k], full[k])


def test_captured_and_replayed_and_on_two_streams():
    i = _dev(_inputs(10, 700, 1536, BF))
    side = torch.cuda.Stream()

    def both(**kw):
        y, s, st = pal.palimpsa_layer_norm(i["x"], i["weight"], i["bias"], i["residual"], want_stats=True, **kw)
        return [y, s, st, *pal.palimpsa_layer_norm_backward(s, i["weight"], st, i["dy"], i["ds"], **kw).values()]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for k, v in _dev(_inputs(11, 700, 1536, BF)).items():
        i[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    want = both()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    for _ in range(5):
        got = both(stream=side), both()
        torch.cuda.synchronize()
        for g in got:
            for a, b in zip(g, want):
                assert torch.equal(a, b)
