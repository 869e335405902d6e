"""Pins of the state-space oracle (CPU): closed forms, continuation, and gradients against
central differences of the plain forward."""
import pytest
import torch

from oracle import ssm

F64 = torch.float64


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _r(g, *shape):
    return torch.randn(shape, generator=g, dtype=F64)


def _conv_inputs(g, rows, D, W, n, state=True):
    return dict(x=_r(g, rows, D), weight=_r(g, D, W), bias=_r(g, D), state0=_r(g, n, W - 1, D) if state else None)


def _scan_inputs(g, rows, ch, G, N, n):
    return dict(x=_r(g, rows, ch), dt=_r(g, rows, ch) - 1, A=torch.rand((ch, N), generator=g, dtype=F64) + 0.3,
                B=_r(g, rows, G, N), C=_r(g, rows, G, N), D=_r(g, ch), z=_r(g, rows, ch), dt_bias=_r(g, ch),
                h0=_r(g, n, ch, N))


def test_conv_equals_a_sum_over_taps():
    g = _gen(0)
    i = _conv_inputs(g, 7, 3, 4, 1)
    y, last = ssm.conv(*i.values(), [0, 7], silu=False)
    full = torch.cat([i["state0"][0], i["x"]])
    for t in range(7):
        assert torch.allclose(y[t], (full[t:t + 4] * i["weight"].t()).sum(0) + i["bias"], rtol=0, atol=1e-14)
    assert torch.equal(last[0], full[-3:])


def test_scan_of_constant_input_reaches_the_geometric_sum():
    """x = B = 1, step s, decay a = exp(-A s): h_t = s (1 - a^t) / (1 - a)."""
    T, s, A = 40, 0.3, torch.tensor([[0.5, 2.0]], dtype=F64)
    one = torch.ones(T, 1, dtype=F64)
    _, h = ssm.scan(one, s * one, A, torch.ones(T, 1, 2, dtype=F64), torch.ones(T, 1, 2, dtype=F64), None, None, None,
                    None, [0, T], softplus=False)
    a = torch.exp(-A * s)
    assert torch.allclose(h[0], s * (1 - a ** T) / (1 - a), rtol=1e-13, atol=0)


@pytest.mark.parametrize("cut", [0, 1, 5, 11])
def test_a_cut_sequence_continues_from_its_state(cut):
    g = _gen(1)
    i = _scan_inputs(g, 11, 4, 2, 3, 1)
    y, h = ssm.scan(*i.values(), [0, 11])
    y1, h1 = ssm.scan(*i.values(), [0, cut])
    y2, h2 = ssm.scan(*(dict(i, h0=h1)).values(), [cut, 11])
    assert torch.allclose(y, y1 + y2, rtol=0, atol=1e-13) and torch.allclose(h, h2, rtol=0, atol=1e-13)
    c = _conv_inputs(g, 11, 4, 3, 1)
    y, s = ssm.conv(*c.values(), [0, 11])
    y1, s1 = ssm.conv(*c.values(), [0, cut])
    y2, s2 = ssm.conv(*(dict(c, state0=s1)).values(), [cut, 11])
    assert torch.allclose(y, y1 + y2, rtol=0, atol=1e-13) and torch.equal(s, s2)


def _check_differences(fn, inputs, cu, seed, **kw):
    g = _gen(seed)
    y, last = fn(*inputs.values(), cu, **kw)
    dy, dl = _r(g, *y.shape), _r(g, *last.shape)
    _, _, grads = ssm.gradients(fn, inputs, dy, dl, cu, **kw)

    def loss(v):
        y, last = fn(*v.values(), cu, **kw)
        return float((y * dy).sum() + (last * dl).sum())

    eps = 1e-6
    for name, gr in grads.items():
        move = _r(g, *inputs[name].shape)
        up, down = (dict(inputs, **{name: inputs[name] + s * eps * move}) for s in (1, -1))
        diff = (loss(up) - loss(down)) / (2 * eps)
        want = float((gr * move).sum())
        # central differences: eps^2 of the third derivative, and 1e-16 / eps of cancellation
        assert abs(diff - want) < 1e-7 * (1 + abs(want)), name


@pytest.mark.parametrize("cu", [[0, 6], [1, 1, 4, 9]])
def test_gradients_equal_central_differences(cu):
    g = _gen(2)
    _check_differences(ssm.conv, _conv_inputs(g, cu[-1] + 1, 3, 4, len(cu) - 1), cu, 3)
    _check_differences(ssm.scan, _scan_inputs(g, cu[-1] + 1, 4, 2, 3, len(cu) - 1), cu, 4)
