"""The fp64 statements of the gated scan and the layer norm, pinned (CPU)."""
import math

import torch

from oracle import ssm

F64 = torch.float64


def _r(g, *shape):
    return torch.randn(shape, generator=g, dtype=F64)


def test_gate_by_hand():
    x, r, i, z = (torch.tensor([[a], [b]], dtype=F64) for a, b in ((1.0, -2.0), (0.3, 1.1), (-0.4, 0.2), (0.7, -1.5)))
    A, rb, ib, h0 = (torch.tensor([v], dtype=F64) for v in (0.8, 0.1, -0.2, 0.5))
    y, last = ssm.gate(x, r, A, i, z, rb, ib, h0[None], [0, 2])
    h = 0.5
    sig = lambda u: 1 / (1 + math.exp(-u))  # noqa: E731
    for t in range(2):
        a = math.exp(-0.8 * sig(float(r[t]) + 0.1))
        h = a * h + math.sqrt(1 - a * a) * sig(float(i[t]) - 0.2) * float(x[t])
        assert abs(float(y[t]) - h * float(z[t]) * sig(float(z[t]))) < 1e-14
    assert abs(float(last[0]) - h) < 1e-14


def test_gate_keeps_the_variance_of_white_inputs():
    """With the input gate open, h is of the input's variance, whatever the decay."""
    g = torch.Generator().manual_seed(0)
    x = _r(g, 400, 256)
    A = torch.logspace(-1, 0.5, 256, dtype=F64)
    y, _ = ssm.gate(x, _r(g, 400, 256), A, None, None, None, None, _r(g, 1, 256), [0, 400])
    assert abs(float(y.var()) - 1) < 0.05   # 400 x 256 values, correlated over up to 20 tokens: 1.4 / sqrt(5000) = 0.02


def test_gate_sequences_are_apart_and_continue():
    g = torch.Generator().manual_seed(1)
    x, r, i, z = (_r(g, 9, 4) for _ in range(4))
    A, h0 = torch.rand(4, generator=g, dtype=F64) + 0.1, _r(g, 3, 4)
    y, last = ssm.gate(x, r, A, i, z, None, None, h0, [0, 4, 4, 8])
    y0, l0 = ssm.gate(x[:4], r[:4], A, i[:4], z[:4], None, None, h0[:1], [0, 4])
    assert torch.equal(y[:4], y0) and torch.equal(last[0], l0[0]) and torch.equal(last[1], h0[1]) and not y[8].any()
    ya, la = ssm.gate(x[:2], r[:2], A, i[:2], z[:2], None, None, h0[:1], [0, 2])
    yb, lb = ssm.gate(x[2:4], r[2:4], A, i[2:4], z[2:4], None, None, la, [0, 2])
    assert torch.equal(torch.cat([ya, yb]), y0) and torch.equal(lb, l0)


def test_gate_gradients_against_differences():
    g = torch.Generator().manual_seed(2)
    D = 3
    inputs = dict(x=_r(g, 5, D), r=_r(g, 5, D), A=torch.rand(D, generator=g, dtype=F64) + 0.2, i=_r(g, 5, D), z=_r(g, 5, D),
                  r_bias=_r(g, D), i_bias=_r(g, D), h0=_r(g, 2, D))
    dy, dl, cu = _r(g, 5, D), _r(g, 2, D), [0, 3, 5]
    _, _, grads = ssm.gradients(ssm.gate, inputs, dy, dl, cu)

    def loss(d):
        y, last = ssm.gate(*d.values(), cu)
        return float((y * dy).sum() + (last * dl).sum())

    e = 1e-6
    for k, v in inputs.items():
        for at in range(v.numel()):
            hi, lo = v.clone(), v.clone()
            hi.view(-1)[at] += e
            lo.view(-1)[at] -= e
            d = (loss({**inputs, k: hi}) - loss({**inputs, k: lo})) / (2 * e)
            assert abs(d - float(grads[k].view(-1)[at])) < 1e-7   # e^2 / 6 third derivatives, 1e-16 / e rounding


def test_layer_norm_pins():
    g = torch.Generator().manual_seed(3)
    s, w, b = _r(g, 6, 16) * 3 + 5, _r(g, 16), _r(g, 16)
    y = ssm.layer_norm(s, None, None, 1e-30)
    assert (y.mean(1).abs() < 1e-14).all() and ((y ** 2).mean(1) - 1).abs().max() < 1e-13
    assert torch.allclose(ssm.layer_norm(2 * s + 7, None, None, 1e-30), y, atol=1e-13)
    assert torch.allclose(ssm.layer_norm(s, w, b, 1e-30), y * w + b, atol=1e-13)
    assert torch.allclose(ssm.layer_norm(s, w, b, 1e-5), torch.nn.functional.layer_norm(s, (16,), w, b, 1e-5), atol=1e-13)
