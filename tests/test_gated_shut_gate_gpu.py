"""The gated scan where every input gate of a channel is nearly shut (sigmoid(i) from 8e-20 down to 2e-35, fp32 numbers
all the same), channel by channel against the fp64 oracle on the same (rounded) inputs, from an empty state: nothing
larger stands beside the gates' outputs.

Bars, relative L2 of a channel. The exponent -i log2(e), at most 116, is off by its rounding and by that of log2(e),
(2^-24 + 2^-25) 116 = 1.0e-5, of which a 2^x makes 7.2e-6; 2^x, the reciprocal and three products add 5e-7. Decays and states as in
test_gated_gpu.py, 2e-5 (twice that for gradients), so 3e-5 and 6e-5, and half a step of the type, bf16 2^-8. Values stay
above 1e-38, with x of 0.5 and more beside a root of 0.05 and more. So, too, for a shut gate with large x (1e25), which
leaves an input of ordinary size; and for a hardly forgetting channel with small x, whose product with 1 - a^2 lies below
fp32's normal numbers though the input does not."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from oracle import ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FINE, FINE_G = 3e-5, 6e-5
NAMES = ("x", "r", "A", "i", "z", "r_bias", "i_bias", "h0")
# Tiles, a cluster, many short sequences, many tiles.
SHAPES = [(2, 200, 72), (1, 1500, 40), (300, 8, 264), (64, 70, 512)]


def _near(got, want, bar, what):
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert got.shape == want.shape
    d, n = (got - want).flatten(0, -2).norm(dim=0), want.flatten(0, -2).norm(dim=0)
    worst = float((d / n).max())
    assert worst <= bar, f"{what}: relative L2 {worst:.3g} of a channel, over {bar:.3g}"


def _inputs(seed, B, T, D, dtype, raw, A, size):
    g = torch.Generator().manual_seed(seed)
    sign = torch.randint(0, 2, (B * T, D), generator=g) * 2 - 1
    r = lambda *s, dtype=F32: torch.randn(s, generator=g).to(dtype)  # noqa: E731
    x = (size * sign * (0.5 + torch.rand((B * T, D), generator=g))).to(dtype)
    return dict(x=x, r=r(B * T, D, dtype=dtype), A=A, i=None if raw is None else raw.expand(B * T, D).to(dtype),
                z=None, r_bias=None, i_bias=None, h0=None), r(B * T, D, dtype=dtype), r(B, D)


def _check(B, T, D, dtype, i, dy, dl):
    cu = list(range(0, B * T + 1, T))
    up = {k: None if v is None else v.to(F64) for k, v in i.items()}
    y, last, want = ssm.gradients(ssm.gate, up, dy.to(F64), dl.to(F64), cu)
    d = {k: v.to(DEV).reshape(B, T, D) if k in "xri" and v is not None else None if v is None else v.to(DEV) for k, v in i.items()}
    gy, gh, ckpt = pal.palimpsa_gated_scan_checkpointed(*d.values())
    _near(gy.reshape(-1, D), y, HALF[dtype] + FINE, "y")
    _near(gh, last, FINE, "h_T")
    got = pal.palimpsa_gated_scan_backward(*list(d.values())[:-1], ckpt, dy.reshape(B, T, D).to(DEV), dl.to(DEV))
    for k, name in (("dx", "x"), ("dr", "r"), ("di", "i")):
        if k in got:
            _near(got[k].reshape(-1, D), want[name], HALF[dtype] + FINE_G, k)
    h = torch.zeros(B, D, device=DEV)
    s = pal.palimpsa_gated_scan_step(d["x"][:, 0], d["r"][:, 0], d["A"], h, None if d["i"] is None else d["i"][:, 0])
    first = ssm.gate(*({**up, **{k: up[k].reshape(B, T, D)[:, 0] for k in "xri" if up[k] is not None}}[k] for k in NAMES),
                     list(range(B + 1)))
    _near(s, first[0], HALF[dtype] + FINE, "y of a token")
    _near(h, first[1], FINE, "h of a token")
    assert pal.palimpsa_get_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("size", [1.0, 1e25])
def test_nearly_shut_input_gates(dtype, B, T, D, size):
    A = 0.2 + torch.rand(D, generator=torch.Generator().manual_seed(4))
    _check(B, T, D, dtype, *_inputs(T + D, B, T, D, dtype, torch.linspace(-80, -40, D), A, size))


@pytest.mark.parametrize("B,T,D", SHAPES)
def test_small_inputs_of_channels_that_hardly_forget(B, T, D):
    _check(B, T, D, F32, *_inputs(T + D, B, T, D, F32, None, torch.logspace(-31, -29, D), 1e-10))
