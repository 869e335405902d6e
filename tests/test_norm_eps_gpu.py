"""The layer norm with an eps below fp32's normal numbers: rows without a deviation have 1 / sqrt(eps)."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
F32 = torch.float32


@pytest.mark.parametrize("D", [64, 520])
@pytest.mark.parametrize("eps", [1e-38, 1e-40, 1e-43, 2e-45])
def test_a_tiny_eps(D, eps):
    """Rows without a deviation: 1 / sqrt(eps) as fp32 has eps, to the reciprocal root's 2 ulp and one step of Newton's method."""
    x = torch.full((3, D), 1.5, device=DEV)
    y, _, st = pal.palimpsa_layer_norm(x, eps=eps, want_stats=True)
    want = torch.tensor(eps, dtype=F32).to(F64).rsqrt()
    assert not y.any()
    assert float((st[:, 1].cpu().to(F64) / want - 1).abs().max()) <= 5e-7
