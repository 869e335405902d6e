"""The selective scan's paths that no other test holds to the oracle: step sizes taken as they are (no softplus), and a
dense batch cut into so many segments that a kernel of its own folds their summaries, forward and in reverse.
Bars as in test_ssm_gpu: step sizes here are at least 0.02 and A at least 0.3."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from oracle import ssm
from tests.test_ssm_gpu import BF, DEV, F32, F64, HALF, _cu, _dense, _dev, _gen, _near, _r, _scan_inputs, _status, _up

pytestmark = pytest.mark.gpu


def _steps(i, seed):
    """The inputs with raw step sizes of at least 0.02, dt_bias (if there) among them."""
    g = _gen(seed)
    dt = 0.02 + 0.3 * torch.rand(i["dt"].shape, generator=g)
    bias = None if i["dt_bias"] is None else 0.2 * torch.rand(i["dt_bias"].shape, generator=g)
    return dict(i, dt=dt.to(i["dt"].dtype), dt_bias=bias)


def _check(dtype, lens, dense, D, G, N, gate, state, extras, softplus):
    n, cu = len(lens), _cu(lens)
    rows = cu[-1] if dense else cu[-1] + 2
    i = _scan_inputs(rows + D + N, rows, n, D, G, N, dtype, gate, state, extras)
    if not softplus:
        i = _steps(i, rows)
    g = _gen(7)
    dy, dl = _r(g, rows, D, dtype=dtype), _r(g, n, D, N)
    y, last, grads = ssm.gradients(ssm.scan, _up(i), dy.to(F64), dl.to(F64), cu, softplus=softplus)
    kw = dict(softplus=softplus)
    if not dense:
        kw.update(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=max(lens))
    d = _dev(_dense(i, n) if dense else i)
    gdy = dy.reshape(n, -1, D).to(DEV) if dense else dy.to(DEV)
    gy, gh = pal.palimpsa_selective_scan(*d.values(), **kw)
    cy, ch, ckpt = pal.palimpsa_selective_scan_checkpointed(*d.values(), **kw)
    assert torch.equal(gy, cy) and torch.equal(gh, ch)
    got = pal.palimpsa_selective_scan_backward(*d.values(), ckpt, gdy, dl.to(DEV), **kw)
    fine, bar = 1e-4, HALF[dtype] + 1e-4
    _near(gy.reshape(-1, D), y, bar, "y")
    _near(gh, last, fine, "h_T")
    for k, name in (("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dz", "z")):
        if k in got:
            _near(got[k].reshape(grads[name].shape), grads[name], bar, k)
    for k, name in (("dA", "A"), ("dD", "D"), ("ddt_bias", "dt_bias"), ("dh0", "h0")):
        if name in grads:
            _near(got[k], grads[name], fine, k)
    _status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,dense,D,G,N", [
    ([17, 17], True, 64, 1, 16), ([300], True, 40, 1, 8), ([50, 50], True, 48, 2, 64), ([5, 0, 1, 130, 16, 3], False, 48, 2, 32),
    ([400, 3], False, 24, 1, 128)])
@pytest.mark.parametrize("gate,state,extras", [(True, True, True), (False, False, False)])
def test_scan_without_softplus(dtype, lens, dense, D, G, N, gate, state, extras):
    _check(dtype, lens, dense, D, G, N, gate, state, extras, False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D,G,N", [(1, 1000, 32, 1, 16), (2, 1500, 24, 1, 8), (1, 1000, 16, 2, 128)])
@pytest.mark.parametrize("gate,state,extras", [(True, True, True), (False, False, False)])
def test_dense_scan_of_many_segments(dtype, B, T, D, G, N, gate, state, extras):
    _check(dtype, [T] * B, True, D, G, N, gate, state, extras, True)


def test_dense_scan_of_many_segments_without_softplus():
    _check(F32, [1000], True, 32, 1, 16, True, True, True, False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,G,N,gate,extras", [(64, 1, 16, True, True), (40, 1, 8, False, False), (48, 3, 32, True, False),
                                               (24, 1, 128, False, True)])
def test_step_without_softplus(dtype, D, G, N, gate, extras):
    B = 5
    i = _steps(_scan_inputs(6, B, B, D, G, N, dtype, gate, True, extras), 3)
    y, last = ssm.scan(*_up(i).values(), _cu([1] * B), softplus=False)
    d = _dev(i)
    h = d.pop("h0")
    got = pal.palimpsa_selective_scan_step(d["x"], d["dt"], d["A"], d["B"], d["C"], h, d["D"], d["z"], d["dt_bias"], softplus=False)
    _near(got, y, HALF[dtype] + 1e-4, "y")
    _near(h, last, 1e-4, "h")
    _status()
