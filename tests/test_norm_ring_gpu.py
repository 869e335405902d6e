"""The layer norm with a residual and its backward with ds, over rows enough that every team walks its ring of batches several
times round, against torch in 64 bits on the GPU. Bars as in test_norm_gpu.py; sums over up to 4e5 rows: 1.2e-5 a term, of
either sign, and a fixed tree of fp32 additions, some 300 in turn: 300^0.5 2^-24 = 1e-6 of the sum's size in the middle."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FINE, FINE_G = 1.2e-5, 3e-5


def _near(got, want, bar, what):
    d = float((got.to(F64) - want).norm() / want.norm())
    assert d <= bar, f"{what}: relative L2 {d:.3g} over {bar:.3g}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,D", [(400001, 16), (300001, 32), (200001, 64), (200001, 72), (150001, 128), (90001, 136), (90001, 256),
                                    (60001, 264), (40001, 512), (30001, 520), (20001, 1024), (12001, 1536), (9001, 2048), (4001, 2056),
                                    (2501, 4104), (1501, 8192)])
def test_many_batches_with_a_residual_and_its_gradient(dtype, rows, D):
    g = torch.Generator(device=DEV).manual_seed(D)
    r = lambda *s, dtype=F32: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    x, res, dy, ds = (r(rows, D, dtype=dtype) for _ in range(4))
    w, b = 1 + 0.3 * r(D), r(D)
    y, s, st = pal.palimpsa_layer_norm(x, w, b, res, want_stats=True)
    assert torch.equal(s, (x.float() + res.float()).to(dtype))
    got = pal.palimpsa_layer_norm_backward(s, w, st, dy, ds)
    u, p = s.to(F64), dy.to(F64)
    mean, rstd = u.mean(1, keepdim=True), (u.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    t = (u - mean) * rstd
    _near(y, t * w.to(F64) + b.to(F64), HALF[dtype] + FINE, "y")
    _near(st[:, 0:1], mean, FINE, "mean")
    _near(st[:, 1:], rstd, FINE, "1 / deviation")
    _near(got["dweight"], (p * t).sum(0), FINE_G, "dweight")
    _near(got["dbias"], p.sum(0), FINE_G, "dbias")
    p = p * w.to(F64)
    _near(got["dx"], rstd * (p - p.mean(1, keepdim=True) - t * (p * t).mean(1, keepdim=True)) + ds.to(F64), HALF[dtype] + FINE_G, "dx")
