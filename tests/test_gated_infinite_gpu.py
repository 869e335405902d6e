"""An infinite input of the gated scan makes its channel's state infinite from there on, as a h of an infinite h is, and touches no
other; an infinite gradient of the last state reaches the first one's."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


# Tiles of one CTA, of a cluster, many short sequences.
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", [(64, 300, 512), (1, 3000, 64), (300, 20, 264)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinite_states_stay_infinite(dtype, B, T, D, value):
    g = torch.Generator(device=DEV).manual_seed(T)
    x, r = (torch.randn(B, T, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    A = torch.logspace(-4, 0, D, device=DEV)
    clean, last = pal.palimpsa_gated_scan(x, r, A)
    at, n, ch = T // 3, B - 1, [3, D - 1]
    x[n, at, ch] = value
    y, h = pal.palimpsa_gated_scan(x, r, A)
    assert (y[n, at:, ch] == value).all() and (h[n, ch] == value).all()
    y[n, at:, ch], h[n, ch] = clean[n, at:, ch], last[n, ch]
    assert torch.equal(y, clean) and torch.equal(h, last)
    state = torch.randn(B, D, generator=g, device=DEV)
    state[n, ch] = value
    pal.palimpsa_gated_scan_step(x[:, 0], r[:, 0], A, state)
    assert (state[n, ch] == value).all() and torch.isfinite(state[:n]).all()
    x[n, at, ch] = 1
    ckpt = pal.palimpsa_gated_scan_checkpointed(x, r, A)[2]
    dl = torch.randn(B, D, generator=g, device=DEV)
    want = pal.palimpsa_gated_scan_backward(x, r, A, None, None, None, None, ckpt, x, dl)["dh0"]
    dl[n, ch] = value
    got = pal.palimpsa_gated_scan_backward(x, r, A, None, None, None, None, ckpt, x, dl)["dh0"]
    slow = [3]      # (the product of all the others' decays may be 0)
    assert (got[n, slow] == value).all()
    got[n, ch] = want[n, ch]
    assert torch.equal(got, want)
    assert pal.palimpsa_get_device_status() == 0
