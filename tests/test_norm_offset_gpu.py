"""The layer norm of rows whose groups of columns lie at different means, far from 0, in fp32, against 64 bits: the parts that a row
is summed in have means of their own, and the error of each part's mean must not reach the deviation.

Bars, of a row's deviation (about 1.4, of 64 columns at least 0.75) or relative. What a sum leaves out of a mean is added up again
from the deviations, so the deviation is a sum of up to 64 squares a thread, 5 steps of lanes and 16 warps of terms that are 2e-7
off: below 1.2e-5, as for rows around 0. The mean itself is rounded to fp32, half a step: 2^-15 = 3.05e-5 below 1024, 4.1e-5 of 0.75,
and 2^-10 = 9.8e-4 below 32768, 1.31e-3; a normalised value keeps that and 1.2e-5 of its own. Rows of up to 64 columns have their
mean as it is summed, a thread's 8 values by 4 additions of pairs and one, its team's by 3: 8 such roundings, each of a part of
the mean."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
F32 = torch.float32


@pytest.mark.parametrize("D", [64, 264, 512, 1024, 1536, 2048, 2056, 4096, 6152, 8192])
@pytest.mark.parametrize("centre,step", [(1000.0, 4.1e-5), (30000.0, 1.31e-3)])
@pytest.mark.parametrize("residual", [False, True])
def test_groups_of_columns_with_means_of_their_own(D, centre, step, residual):
    g = torch.Generator(device=DEV).manual_seed(D)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    rows = 37
    step *= 8 if D <= 64 else 1
    group = torch.arange(D, device=DEV) // 128
    x = centre + r(rows, D) + r(rows, (D + 127) // 128)[:, group]
    res = r(rows, D) if residual else None
    w, b = 1 + 0.1 * r(D), r(D)
    y, s, st = pal.palimpsa_layer_norm(x, w, b, res, want_stats=True)
    assert torch.equal(s, x if res is None else x + res)
    u = s.to(F64)
    mean, dev = u.mean(1), (u.var(1, unbiased=False) + 1e-5).sqrt()
    assert float((st[:, 1].to(F64) * dev - 1).abs().max()) <= 1.2e-5
    assert float(((st[:, 0].to(F64) - mean) / dev).abs().max()) <= step + 1.2e-5
    t = (u - mean[:, None]) / dev[:, None]
    got = (y.to(F64) - b.to(F64)) / w.to(F64)
    assert float((got - t).norm() / t.norm()) <= step + 1.2e-5
