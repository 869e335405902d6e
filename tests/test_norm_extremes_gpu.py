"""The layer norm at the end of fp32's range: rows whose sum passes it though none of their values does."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [8, 64, 264, 520, 1536, 2056, 4104, 8192])
@pytest.mark.parametrize("size", [1e37, 1.5e38])
def test_rows_whose_sum_passes_the_range(dtype, D, size):
    """A constant row, rows off centre and a row of either sign: their deviations pass the range of their squares or are
    those of eps, so y is the bias and no gradient passes; the rows beside them are as ever. A mean is the mean to 30 roundings of 2^-24, 2e-6 of the largest value."""
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.randn(6, D, generator=g, device=DEV)
    w, b = torch.rand(D, generator=g, device=DEV) + 0.5, torch.randn(D, generator=g, device=DEV)
    dy = torch.randn(6, D, generator=g, device=DEV).to(dtype)
    clean = x.to(dtype)
    want, _, wst = pal.palimpsa_layer_norm(clean, w, b, want_stats=True)
    wg = pal.palimpsa_layer_norm_backward(clean, w, wst, dy)
    x[1] = size
    x[2] = size * (0.5 + 0.5 * torch.rand(D, generator=g, device=DEV))
    x[3] = -x[2]
    x[4] = size * (2 * torch.rand(D, generator=g, device=DEV) - 1)
    x = x.to(dtype)
    y, s, st = pal.palimpsa_layer_norm(x, w, b, want_stats=True)
    for k in (2, 3, 4):
        assert torch.equal(y[k], b.to(dtype)) and st[k, 1] == 0
    assert torch.equal(y[1], b.to(dtype))
    assert float((st[:, 0].to(F64) - x.to(F64).mean(1))[1:5].abs().max()) <= 2e-6 * 2 * size
    assert torch.equal(y[0], want[0]) and torch.equal(y[5], want[5])
    got = pal.palimpsa_layer_norm_backward(s, w, st, dy)
    assert not got["dx"][2:5].any() and torch.isfinite(got["dx"]).all()
    assert torch.equal(got["dx"][0], wg["dx"][0]) and torch.equal(got["dx"][5], wg["dx"][5])
    assert torch.isfinite(got["dweight"]).all() and torch.isfinite(got["dbias"]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [16, 1536, 2056, 4096, 8192])
@pytest.mark.parametrize("col", [0, -1])
def test_infinities_and_nan_spoil_their_own_row_alone(dtype, D, col):
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.randn(40, D, generator=g, device=DEV).to(dtype)
    w, b = torch.rand(D, generator=g, device=DEV) + 0.5, torch.randn(D, generator=g, device=DEV)
    want, _, _ = pal.palimpsa_layer_norm(x, w, b)
    x[3, col], x[17, col], x[30, col] = float("inf"), float("-inf"), float("nan")
    y, _, st = pal.palimpsa_layer_norm(x, w, b, want_stats=True)
    for k in (3, 17, 30):
        assert torch.isnan(y[k]).all() and torch.isnan(st[k, 1])
        y[k] = want[k]
    assert torch.equal(y, want)
