"""The gated scan on slices of a wider projection, in tiles of clusters of every kind, of single CTAs and by threads: the bits of
dense copies."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", [(1, 9000, 64), (2, 3000, 520), (4, 2048, 1024), (8, 1000, 1536), (64, 300, 512), (300, 8, 264)])
@pytest.mark.parametrize("packed", [False, True])
def test_slices_of_a_projection(dtype, B, T, D, packed):
    g = torch.Generator(device=DEV).manual_seed(T + D)
    lead = (B * T,) if packed else (B, T)
    wide = torch.randn(*lead, 5 * D + 16, generator=g, device=DEV).to(dtype)
    x, r, i, z, dy = (wide[..., 16 + k * D:16 + (k + 1) * D] for k in range(5))
    A = 0.1 + torch.rand(D, generator=g, device=DEV)
    rb, ib, h0 = (torch.randn(*s, generator=g, device=DEV) for s in ((D,), (D,), (B, D)))
    kw = {}
    if packed:   # sequences of different lengths, the last one ending before the rows do
        cu = [k * T + (k % 3) * (T // 4) for k in range(B)] + [B * T - 3]
        cu[0] = 2
        kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=max(b - a for a, b in zip(cu, cu[1:])))
    res = []
    for f in (lambda t: t, lambda t: t.contiguous()):
        y, h, ckpt = pal.palimpsa_gated_scan_checkpointed(f(x), f(r), A, f(i), f(z), rb, ib, h0, **kw)
        grads = pal.palimpsa_gated_scan_backward(f(x), f(r), A, f(i), f(z), rb, ib, ckpt, f(dy), h0, **kw)
        res.append([y, h, *grads.values()])
    for a, b in zip(*res):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    assert pal.palimpsa_get_device_status() == 0
