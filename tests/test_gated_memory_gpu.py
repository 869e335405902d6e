"""The gated scan over long memories with gates that hardly change: rates w from 1e-6 to 1e-4 a token over up to 32768
tokens, where the decay a = e^-w in fp32 is off by up to half its last place, 3e-8, the same way at every token: over
all of them 1e-3 of a state, where its memory goes on, and 3 % of the rate it forgets at. Against the recurrence in 64 bits on the GPU,
from a state that is not empty.

Bars, relative L2 over all tokens. The gates as in test_gated_gpu.py: a rate is off by 1.2e-6, a memory of w T = 3.3
at the most by 4e-6, an input's factor by 1e-6. A state is rounded to fp32 where it is handed on, at every token or every 8th:
2^-24 / sqrt(3) each in root mean square, either way since the inputs differ: 3.1e-6 over 8192 tokens one by one, and over 32768 / 8 of
them less. Together 1e-5; 2e-5 as there, 4e-5 for gradients, and half a step of the type where outputs have it."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FINE, FINE_G = 2e-5, 4e-5


def _near(got, want, bar, what):
    d = float((got.to(F64) - want).norm() / want.norm())
    assert d <= bar, f"{what}: relative L2 {d:.3g} over {bar:.3g}"


def _inputs(B, T, D, dtype):
    g = torch.Generator(device=DEV).manual_seed(B + T + D)
    r = lambda *s, dtype=F32: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    raw = r(D, dtype=dtype)
    A = torch.logspace(-6, -4, D, device=DEV) * (1 + torch.exp(-raw.float()))       # a rate A sigmoid(raw) of 1e-6 to 1e-4
    return r(B, T, D, dtype=dtype), raw.expand(B, T, D).contiguous(), A, 1 + r(B, D), r(B, T, D, dtype=dtype), 1 + r(B, D)


def _exact(x, raw, A, h0, dy, dl):
    """y, h_T and the gradients of x, of the raw gate (by token), of A and of h0, in 64 bits."""
    B, T, D = x.shape
    s, A = torch.sigmoid(raw[0, 0].to(F64)), A.to(F64)
    w = A * s
    a, n = torch.exp(-w), torch.sqrt(-torch.expm1(-2 * w))
    h, x, dy = h0.to(F64), x.to(F64), dy.to(F64)
    y = torch.empty_like(x)
    for t in range(T):
        h = a * h + n * x[:, t]
        y[:, t] = h
    before = torch.cat([h0.to(F64)[:, None], y[:, :-1]], 1)
    g, c = torch.empty_like(x), dl.to(F64)
    for t in range(T - 1, -1, -1):
        g[:, t] = dy[:, t] + c
        c = a * g[:, t]
    dw = g * (x * (a * a / n) - a * before)
    return y, h, g * n, dw * (w * (1 - s)), (dw * s).sum((0, 1)), c


# A cluster; few CTAs of a cluster; one CTA a sequence; many short sequences.
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", [(1, 32768, 64), (4, 16384, 1024), (64, 8192, 1024), (1024, 64, 512)])
def test_long_memories(dtype, B, T, D):
    x, raw, A, h0, dy, dl = _inputs(B, T, D, dtype)
    y, last, dx, dr, dA, dh0 = _exact(x, raw, A, h0, dy, dl)
    gy, gh, ckpt = pal.palimpsa_gated_scan_checkpointed(x, raw, A, h0=h0)
    _near(gy, y, HALF[dtype] + FINE, "y")
    _near(gh, last, FINE, "h_T")
    _near(gy[:, -1], y[:, -1], HALF[dtype] + FINE, "y of the last token")
    g = pal.palimpsa_gated_scan_backward(x, raw, A, None, None, None, None, ckpt, dy, dl)
    for k, want, bar in (("dx", dx, HALF[dtype] + FINE_G), ("dr", dr, HALF[dtype] + FINE_G), ("dA", dA, FINE_G), ("dh0", dh0, FINE_G)):
        _near(g[k], want, bar, k)
    assert pal.palimpsa_get_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_memories_token_by_token(dtype):
    B, T, D = 2, 8192, 64
    x, raw, A, h0, _, _ = _inputs(B, T, D, dtype)
    s = A.to(F64) * torch.sigmoid(raw[0, 0].to(F64))
    a, n = torch.exp(-s), torch.sqrt(-torch.expm1(-2 * s))
    want, h = h0.to(F64), h0.clone()
    for t in range(T):
        pal.palimpsa_gated_scan_step(x[:, t], raw[:, t], A, h)
        want = a * want + n * x[:, t].to(F64)
    _near(h, want, FINE, "h")
    assert pal.palimpsa_get_device_status() == 0
