"""How exact a step size is, by itself. From an empty state with x = B = 1, one token leaves h = s, the step size
softplus(u), with no other rounding; the gradient of x is s and that of dt is sigmoid(u) where dh_T picks one state.

Bar, root mean square of the relative error over many u of [-10, 2]: e^-|u| = (2^(x/2))^2 with x = -|u| log2 e. The
product's rounding gives |u| 2^-24 / sqrt(3) and log2 e's own |u| 1.4e-8: at |u| = 10, 3.5e-7 and 1.4e-7 (less where |u| is
less: 2.0e-7 and 0.8e-7 root mean square over [0, 10]). 2^x with a largest error of 2^-22, taken as uniform, squared: 2.8e-7. Six
more roundings of 2^-24 / sqrt(3): 0.8e-7. Together 4.5e-7 at most; the reciprocal (1 ulp) is among the six."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BAR = 5e-7


def _rms(got, want):
    return float(((got.cpu().to(F64) - want) / want).square().mean().sqrt())


@pytest.mark.parametrize("lo,hi", [(-10.0, -2.0), (-7.0, -2.0), (-2.0, 2.0)])
def test_step_sizes_are_accurate_relative_to_themselves(lo, hi):
    D, N = 4096, 8
    u = lo + (hi - lo) * torch.rand((D,), generator=torch.Generator().manual_seed(1))
    s = torch.logaddexp(u.to(F64), torch.zeros(D, dtype=F64))
    one = lambda *shape: torch.ones(shape, device=DEV)  # noqa: E731
    raw, A, bc = u.to(DEV), one(D, N), one(1, 1, 1, N)
    _, h, ckpt = pal.palimpsa_selective_scan_checkpointed(one(1, 1, D), raw.reshape(1, 1, D), A, bc, bc)
    assert _rms(h[0, :, 3], s) <= BAR                     # of a prompt
    state = torch.zeros(1, D, N, device=DEV)
    pal.palimpsa_selective_scan_step(one(1, D), raw.reshape(1, D), A, bc[0], bc[0], state)
    assert _rms(state[0, :, 5], s) <= BAR                 # of a single token
    dh = torch.zeros(1, D, N, device=DEV)
    dh[..., 2] = 1
    g = pal.palimpsa_selective_scan_backward(one(1, 1, D), raw.reshape(1, 1, D), A, bc, bc, None, None, None, None, ckpt,
                                             torch.zeros(1, 1, D, device=DEV), dh)
    assert _rms(g["dx"][0, 0], s) <= BAR                  # of the backward
    assert _rms(g["ddt"][0, 0], torch.sigmoid(u.to(F64))) <= BAR
    assert pal.palimpsa_get_device_status() == 0
