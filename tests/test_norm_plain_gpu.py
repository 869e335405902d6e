"""The layer norm without weight and bias at every width's kernel, against torch in 64 bits. Bars as in test_norm_gpu.py."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _near(got, want, bar, what):
    d = float((got.to(F64) - want).norm() / want.norm())
    assert d <= bar, f"{what}: relative L2 {d:.3g} over {bar:.3g}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [8, 16, 24, 64, 72, 104, 136, 200, 264, 392, 520, 768, 776, 1032, 1544, 2056, 4104, 8192])
@pytest.mark.parametrize("residual", [False, True])
def test_widths_without_parameters(dtype, D, residual):
    g = torch.Generator(device=DEV).manual_seed(D)
    x, res, dy, ds = (torch.randn(41, D, generator=g, device=DEV).to(dtype) for _ in range(4))
    y, s, st = pal.palimpsa_layer_norm(x, residual=res if residual else None, want_stats=True)
    got = pal.palimpsa_layer_norm_backward(s, None, st, dy, ds if residual else None)
    u, p = s.to(F64), dy.to(F64)
    rstd = (u.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    t = (u - u.mean(1, keepdim=True)) * rstd
    _near(y, t, HALF[dtype] + 1.2e-5, "y")
    dx = rstd * (p - p.mean(1, keepdim=True) - t * (p * t).mean(1, keepdim=True))
    _near(got["dx"], dx + ds.to(F64) if residual else dx, HALF[dtype] + 3e-5, "dx")
    _near(got["dbias"], p.sum(0), 3e-5, "dbias")
    assert "dweight" not in got
