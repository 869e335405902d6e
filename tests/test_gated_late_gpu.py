"""A cluster's state (gradient) that comes when the waits for it have run out: every CTA stays until what was sent to it has
landed, the kernels latch PALIMPSA_ERR_TIMEOUT and end, and later calls have the bits of earlier ones. With one round a
CTA (few tokens) the late state is the last thing that its sender does; with more, rounds follow."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", [(1, 130, 64), (1, 400, 8), (1, 1500, 64), (1, 9000, 520), (4, 2048, 1024)])
def test_states_that_come_late(dtype, B, T, D):
    g = torch.Generator(device=DEV).manual_seed(T)
    x, r, z, dy = (torch.randn(B, T, D, generator=g, device=DEV).to(dtype) for _ in range(4))
    A = 0.1 + torch.rand(D, generator=g, device=DEV)

    def forward():
        return pal.palimpsa_gated_scan_checkpointed(x, r, A, None, z)

    def backward(ckpt):
        return list(pal.palimpsa_gated_scan_backward(x, r, A, None, z, None, None, ckpt, dy).values())

    want = forward()
    grads = backward(want[2])
    assert pal.palimpsa_get_device_status() == 0
    pal.palimpsa_set_wait_timeout_ns(1_000_000)
    pal.palimpsa_debug_withhold_first_copy(2)
    try:
        for _ in range(3):
            forward()
            assert pal.palimpsa_get_device_status() == 8
            backward(want[2])
            assert pal.palimpsa_get_device_status() == 8
    finally:
        pal.palimpsa_debug_withhold_first_copy(False)
        pal.palimpsa_set_wait_timeout_ns(2_000_000_000)
    for a, b in zip([*want, *grads], [*forward(), *backward(want[2])]):
        assert torch.equal(a, b)
    assert pal.palimpsa_get_device_status() == 0
