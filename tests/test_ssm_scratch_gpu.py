"""A call whose scratch the device cannot give is refused, and the calls after it do not hear of it."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_calls_after_a_refusal_for_memory_are_not_affected():
    """4 million empty sequences: the sums of dA alone want 4 N bytes a channel and sequence, over a terabyte."""
    B, D, N = 1 << 22, 512, 128
    e = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    A = torch.ones(D, N, device=DEV)
    x, bc, ckpt = e(B, 0, D), e(B, 0, 1, N), e(B, 0, D, N)
    with pytest.raises(pal.PalimpsaError, match="PALIMPSA_ERR_CUDA"):
        pal.palimpsa_selective_scan_backward(x, x, A, bc, bc, None, None, None, None, ckpt, x, want_state_grad=False)
    one = torch.ones(1, 4, 8, device=DEV)                    # a launch of torch's, which looks at the last error
    u, _ = pal.palimpsa_causal_conv(one, torch.ones(8, 4, device=DEV), silu=False)
    assert u[0, :, 0].tolist() == [1, 2, 3, 4]
    assert pal.palimpsa_get_device_status() == 0
