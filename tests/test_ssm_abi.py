"""Refusals of the state-space entry points (CPU): status codes before any device is touched, and the
binding's checks of arguments."""
import ctypes

import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from metaplastic_linear_attention_gb300 import build_lib, ssm

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE, ERR_DOMAIN, ERR_UNSUPPORTED = range(7)
P = 1 << 20     # a well-aligned address that no check below gets as far as using


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    pal.load_library()
    return ssm._library()


CONV = dict(x=P, x_stride=0, weight=P, bias=None, state0=None, y=P, state_T=None, cu=None, B=2, T=16, max_seqlen=16, D=64,
            W=4, flags=1, dtype=1)
CONV_STEP = dict(x=P, x_stride=0, weight=P, bias=None, state=P, y=P, B=2, D=64, W=4, flags=1, dtype=1)
CONV_BWD = dict(x=P, x_stride=0, weight=P, bias=None, state0=None, dy=P, dy_stride=0, dstate_T=None, dx=P, dweight=P,
                dbias=None, dstate0=None, cu=None, B=2, T=16, max_seqlen=16, D=64, W=4, flags=1, dtype=1)
SCAN = dict(x=P, dt=P, A=P, B_t=P, C_t=P, skip=None, z=None, dt_bias=None, h0=None, y=P, h_T=P, ckpt=None, strides=None,
            cu=None, B=2, T=16, max_seqlen=16, D=64, G=1, N=16, flags=1, dtype=1)
SCAN_STEP = dict(x=P, dt=P, A=P, B_t=P, C_t=P, skip=None, z=None, dt_bias=None, h=P, y=P, strides=None, B=2, D=64, G=1,
                 N=16, flags=1, dtype=1)
SCAN_BWD = dict(x=P, dt=P, A=P, B_t=P, C_t=P, skip=None, z=None, dt_bias=None, ckpt=P, dy=P, dh_T=None, dx=P, ddt=P, dA=P,
                dB=P, dC=P, dskip=None, dz=None, ddt_bias=None, dh0=None, strides=None, cu=None, B=2, T=16,
                max_seqlen=16, D=64, G=1, N=16, flags=1, dtype=1)
CALLS = dict(palimpsa_causal_conv=CONV, palimpsa_causal_conv_step=CONV_STEP, palimpsa_causal_conv_backward=CONV_BWD,
             palimpsa_selective_scan=SCAN, palimpsa_selective_scan_step=SCAN_STEP,
             palimpsa_selective_scan_backward=SCAN_BWD)
PACKED = [n for n in CALLS if not n.endswith("step")]
SCANS = [n for n in CALLS if "scan" in n]
CONVS = [n for n in CALLS if "conv" in n]


def _call(lib, name, **over):
    args = dict(CALLS[name], **over)
    assert args.keys() == CALLS[name].keys()
    return getattr(lib, name)(*args.values(), None)


@pytest.mark.parametrize("name", CALLS)
def test_required_pointers(lib, name):
    for field, v in CALLS[name].items():
        if v == P:
            assert _call(lib, name, **{field: None}) == ERR_NULL, field


def test_gate_needs_its_gradient(lib):
    assert _call(lib, "palimpsa_selective_scan_backward", z=P) == ERR_NULL


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), ERR_DTYPE), (dict(dtype=-1), ERR_DTYPE), (dict(flags=2), ERR_UNSUPPORTED), (dict(B=0), ERR_SHAPE),
    (dict(B=-1), ERR_SHAPE), (dict(D=0), ERR_SHAPE), (dict(D=-8), ERR_SHAPE), (dict(D=12), ERR_UNSUPPORTED),
    (dict(x=P + 8), ERR_ALIGN), (dict(B=1 << 30, D=1 << 20), ERR_SHAPE),
    (dict(D=(1 << 24) + 8), ERR_SHAPE),
])
def test_common_refusals(lib, name, over, code):
    assert _call(lib, name, **over) == code


@pytest.mark.parametrize("name", PACKED)
@pytest.mark.parametrize("over,code", [
    (dict(T=-1), ERR_SHAPE), (dict(T=0x7fffffff, B=1, D=8), ERR_SHAPE), (dict(cu=P, max_seqlen=17), ERR_SHAPE), (dict(cu=P, max_seqlen=-1), ERR_SHAPE),
    (dict(cu=P + 2), ERR_ALIGN),
])
def test_batch_refusals(lib, name, over, code):
    assert _call(lib, name, **over) == code


@pytest.mark.parametrize("name", CONVS)
@pytest.mark.parametrize("over,code", [
    (dict(W=1), ERR_UNSUPPORTED), (dict(W=5), ERR_UNSUPPORTED), (dict(x_stride=56), ERR_SHAPE),
    (dict(x_stride=-64), ERR_SHAPE), (dict(x_stride=68), ERR_ALIGN), (dict(weight=P + 2), ERR_ALIGN),
])
def test_conv_refusals(lib, name, over, code):
    assert _call(lib, name, **over) == code


@pytest.mark.parametrize("name", SCANS)
@pytest.mark.parametrize("over,code", [
    (dict(N=12), ERR_UNSUPPORTED), (dict(N=256), ERR_UNSUPPORTED), (dict(N=4), ERR_UNSUPPORTED), (dict(N=0), ERR_SHAPE),
    (dict(G=0), ERR_SHAPE), (dict(G=3), ERR_UNSUPPORTED), (dict(G=16), ERR_UNSUPPORTED), (dict(A=P + 4), ERR_ALIGN),
    (dict(dt=P + 2), ERR_ALIGN), (dict(skip=P + 1), ERR_ALIGN),
])
def test_scan_refusals(lib, name, over, code):
    assert _call(lib, name, **over) == code


@pytest.mark.parametrize("name", SCANS)
@pytest.mark.parametrize("field,given,code", [
    ("x", 56, ERR_SHAPE), ("dt", 68, ERR_ALIGN), ("B", 8, ERR_SHAPE), ("C", 20, ERR_ALIGN), ("z", -1, ERR_SHAPE),
])
def test_scan_stride_refusals(lib, name, field, given, code):
    st = ssm._Strides(**{field: given})
    assert _call(lib, name, strides=ctypes.byref(st)) == code


@pytest.mark.parametrize("over,code", [
    (dict(cu=None), ERR_NULL), (dict(arrays=None), ERR_NULL), (dict(p=[P, 0]), ERR_NULL), (dict(n=9), ERR_SHAPE),
    (dict(n=-1), ERR_SHAPE), (dict(B=0), ERR_SHAPE), (dict(T=-1), ERR_SHAPE), (dict(p=[P, P + 8]), ERR_ALIGN),
    (dict(w=[16, 24]), ERR_ALIGN), (dict(w=[16, -16]), ERR_SHAPE), (dict(cu=P + 1), ERR_ALIGN), (dict(longest=-1), ERR_SHAPE),
    (dict(longest=101), ERR_SHAPE),
])
def test_zero_rows_outside_refusals(lib, over, code):
    a = dict(p=[P, P], w=[16, 32], n=2, cu=P, B=3, T=100, longest=50, arrays=True) | over
    p = (ctypes.c_void_p * 2)(*a["p"]) if a["arrays"] else None
    w = (ctypes.c_longlong * 2)(*a["w"])
    assert lib.palimpsa_zero_rows_outside(p, w, a["n"], a["cu"], a["B"], a["T"], a["longest"], None) == code


def test_checkpoint_bytes(lib):
    f = lib.palimpsa_selective_scan_checkpoint_bytes
    assert f(3, 33, 0, 64, 16) == 3 * 3 * 64 * 16 * 4
    assert f(3, 33, 1, 64, 16) == (33 // 16 + 3) * 64 * 16 * 4
    assert f(0, 33, 0, 64, 16) == 0 and f(3, 0, 0, 64, 16) == 0
    for packed in (False, True):
        shape = pal.palimpsa_selective_scan_checkpoint_shape(3, 33, 64, 16, packed)
        assert torch.Size(shape).numel() * 4 == f(3, 33, int(packed), 64, 16)


def test_packed_checkpoint_slots_never_overlap():
    """Sequence n from row s0 owns ceil(len / 16) slots from s0 / 16 + n."""
    g = torch.Generator().manual_seed(0)
    for _ in range(200):
        lens = torch.randint(0, 40, (9,), generator=g).tolist()
        s0, end = 0, 0
        for n, ln in enumerate(lens):
            first = s0 // 16 + n
            assert first >= end
            end = max(end, first + -(-ln // 16))
            s0 += ln
        assert end <= s0 // 16 + len(lens)


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="device tensors"):
        pal.palimpsa_causal_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="device tensors"):
        pal.palimpsa_selective_scan(x, x, torch.ones(8, 16), torch.zeros(2, 3, 1, 16), torch.zeros(2, 3, 1, 16))


@pytest.mark.parametrize("make,lead,ld", [
    (lambda: torch.zeros(2, 3, 8), 2, 0), (lambda: torch.zeros(2, 3, 24)[..., 8:16], 2, 24),
    (lambda: torch.zeros(2, 1, 24)[..., :8], 2, 24), (lambda: torch.zeros(1, 3, 24)[..., :8], 2, 24),
    (lambda: torch.zeros(5, 16)[:, :8], 1, 16), (lambda: torch.zeros(2, 3, 64)[..., :32].unflatten(-1, (4, 8)), 2, 64),
])
def test_row_strides(make, lead, ld):
    t = make()
    assert ssm._rows(t, "t", tuple(t.shape), t.dtype, t.get_device(), lead) == ld


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(2, 8, 3).transpose(1, 2), lambda: torch.zeros(2, 3, 16)[..., ::2],
    lambda: torch.zeros(2, 4, 8)[:, :3], lambda: torch.zeros(1, 1, 8).expand(2, 3, 8),
    lambda: torch.zeros(3, 2, 8).transpose(0, 1),
])
def test_rows_that_no_stride_describes_are_refused(make):
    t = make()
    with pytest.raises(ValueError):
        ssm._rows(t, "t", tuple(t.shape), t.dtype, t.get_device(), 2)


def test_rows_check_shape_dtype_and_device():
    t = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError):
        ssm._rows(t, "t", (2, 3, 16), t.dtype, t.get_device(), 2)
    with pytest.raises(TypeError):
        ssm._rows(t, "t", (2, 3, 8), torch.bfloat16, t.get_device(), 2)
    with pytest.raises(ValueError):
        ssm._rows(t, "t", (2, 3, 8), t.dtype, 3, 2)
