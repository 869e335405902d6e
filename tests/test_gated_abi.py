"""Refusals of the gated scan and the layer norm (CPU): status codes before any device is touched, and the binding's
checks of arguments."""
import ctypes

import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from metaplastic_linear_attention_gb300 import build_lib, gated, norm, ssm

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE, ERR_DOMAIN, ERR_UNSUPPORTED = range(7)
P = 1 << 20     # a well-aligned address that no check below gets as far as using


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    pal.load_library()
    return ssm._library()


SCAN = dict(x=P, r=P, A=P, i=None, z=None, r_bias=None, i_bias=None, h0=None, y=P, h_T=P, ckpt=None, strides=None, cu=None,
            B=2, T=16, max_seqlen=16, D=64, flags=0, dtype=1)
STEP = dict(x=P, r=P, A=P, i=None, z=None, r_bias=None, i_bias=None, h=P, y=P, strides=None, B=2, D=64, dtype=1)
BWD = dict(x=P, r=P, A=P, i=None, z=None, r_bias=None, i_bias=None, ckpt=P, dy=P, dh_T=None, dx=P, dr=P, dA=P, di=None, dz=None,
           dr_bias=None, di_bias=None, dh0=None, strides=None, cu=None, B=2, T=16, max_seqlen=16, D=64, flags=0, dtype=1)
NORM = dict(x=P, x_stride=0, residual=None, residual_stride=0, weight=None, bias=None, y=P, sum=None, stats=None, rows=16, D=64,
            eps=1e-5, dtype=1)
NORM_BWD = dict(s=P, s_stride=0, weight=None, stats=P, dy=P, dy_stride=0, ds=None, ds_stride=0, dx=P, dweight=None, dbias=None,
                rows=16, D=64, dtype=1)
CALLS = dict(palimpsa_gated_scan=SCAN, palimpsa_gated_scan_step=STEP, palimpsa_gated_scan_backward=BWD,
             palimpsa_layer_norm=NORM, palimpsa_layer_norm_backward=NORM_BWD)
SCANS = [n for n in CALLS if "scan" in n]
PACKED = [n for n in SCANS if not n.endswith("step")]
NORMS = [n for n in CALLS if "norm" in n]


def _call(lib, name, **over):
    args = dict(CALLS[name], **over)
    assert args.keys() == CALLS[name].keys()
    return getattr(lib, name)(*args.values(), None)


@pytest.mark.parametrize("name", CALLS)
def test_required_pointers(lib, name):
    for field, v in CALLS[name].items():
        if v == P:
            assert _call(lib, name, **{field: None}) == ERR_NULL, field


@pytest.mark.parametrize("name,over", [
    ("palimpsa_gated_scan", dict(i_bias=P)), ("palimpsa_gated_scan_step", dict(i_bias=P)),
    ("palimpsa_gated_scan_backward", dict(i_bias=P)), ("palimpsa_gated_scan_backward", dict(i=P)),
    ("palimpsa_gated_scan_backward", dict(z=P)), ("palimpsa_layer_norm", dict(residual=P)),
])
def test_what_an_option_needs(lib, name, over):
    assert _call(lib, name, **over) == ERR_NULL


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), ERR_DTYPE), (dict(dtype=-1), ERR_DTYPE), (dict(D=0), ERR_SHAPE), (dict(D=-8), ERR_SHAPE),
    (dict(D=12), ERR_UNSUPPORTED),
])
def test_common_refusals(lib, name, over, code):
    assert _call(lib, name, **over) == code


@pytest.mark.parametrize("name", SCANS)
@pytest.mark.parametrize("over,code", [
    (dict(B=0), ERR_SHAPE), (dict(B=-1), ERR_SHAPE), (dict(B=1 << 30, D=1 << 20), ERR_SHAPE), (dict(D=(1 << 24) + 8), ERR_SHAPE),
    (dict(x=P + 8), ERR_ALIGN), (dict(r=P + 2), ERR_ALIGN), (dict(A=P + 2), ERR_ALIGN), (dict(r_bias=P + 1), ERR_ALIGN),
])
def test_scan_refusals(lib, name, over, code):
    assert _call(lib, name, **over) == code


@pytest.mark.parametrize("name", PACKED)
@pytest.mark.parametrize("over,code", [
    (dict(T=-1), ERR_SHAPE), (dict(T=0x7fffffff, B=1, D=8), ERR_SHAPE), (dict(cu=P, max_seqlen=17), ERR_SHAPE),
    (dict(cu=P, max_seqlen=-1), ERR_SHAPE), (dict(cu=P + 2), ERR_ALIGN), (dict(ckpt=P + 4), ERR_ALIGN), (dict(flags=4), ERR_UNSUPPORTED),
])
def test_batch_refusals(lib, name, over, code):
    assert _call(lib, name, **over) == code


@pytest.mark.parametrize("name", SCANS)
@pytest.mark.parametrize("field,given,code", [
    ("x", 56, ERR_SHAPE), ("r", 68, ERR_ALIGN), ("i", 8, ERR_SHAPE), ("z", -1, ERR_SHAPE), ("dy", 68, ERR_ALIGN),
])
def test_scan_stride_refusals(lib, name, field, given, code):
    st = gated._Strides(**{field: given})
    assert _call(lib, name, strides=ctypes.byref(st)) == code


@pytest.mark.parametrize("name,over,code", [(n, o, c) for n in NORMS for o, c in (
    (dict(rows=-1), ERR_SHAPE), (dict(rows=1 << 36), ERR_SHAPE), (dict(D=8200), ERR_UNSUPPORTED), (dict(stats=P + 4), ERR_ALIGN),
    (dict(weight=P + 2), ERR_ALIGN))] + [
    ("palimpsa_layer_norm", dict(x=P + 8), ERR_ALIGN), ("palimpsa_layer_norm", dict(x_stride=56), ERR_SHAPE),
    ("palimpsa_layer_norm", dict(residual_stride=68), ERR_ALIGN), ("palimpsa_layer_norm", dict(eps=0.0), ERR_UNSUPPORTED),
    ("palimpsa_layer_norm", dict(eps=-1e-5), ERR_UNSUPPORTED), ("palimpsa_layer_norm", dict(eps=float("nan")), ERR_UNSUPPORTED),
    ("palimpsa_layer_norm", dict(eps=float("inf")), ERR_UNSUPPORTED), ("palimpsa_layer_norm_backward", dict(dy=P + 8), ERR_ALIGN),
    ("palimpsa_layer_norm_backward", dict(s_stride=-64), ERR_SHAPE), ("palimpsa_layer_norm_backward", dict(ds_stride=68), ERR_ALIGN),
    ("palimpsa_layer_norm_backward", dict(dy_stride=63), ERR_SHAPE),
])
def test_norm_refusals(lib, name, over, code):
    assert _call(lib, name, **over) == code


def test_checkpoint_bytes(lib):
    f = lib.palimpsa_gated_scan_checkpoint_bytes
    assert f(3, 33, 0, 64) == 3 * 5 * 64 * 4
    assert f(3, 33, 1, 64) == (33 // 8 + 3) * 64 * 4
    assert f(0, 33, 0, 64) == 0 and f(3, 0, 0, 64) == 0
    for packed in (False, True):
        shape = pal.palimpsa_gated_scan_checkpoint_shape(3, 33, 64, packed)
        assert torch.Size(shape).numel() * 4 == f(3, 33, int(packed), 64)


def test_packed_checkpoint_slots_never_overlap():
    """Sequence n from row s0 owns ceil(len / 8) slots from s0 / 8 + n."""
    g = torch.Generator().manual_seed(0)
    for _ in range(200):
        lens = torch.randint(0, 40, (9,), generator=g).tolist()
        s0, end = 0, 0
        for n, ln in enumerate(lens):
            first = s0 // 8 + n
            assert first >= end
            end = max(end, first + -(-ln // 8))
            s0 += ln
        assert end <= s0 // 8 + len(lens)


def test_binding_refuses_host_tensors():
    x, v = torch.zeros(2, 3, 8), torch.ones(8)
    for call in (lambda: pal.palimpsa_gated_scan(x, x, v), lambda: pal.palimpsa_gated_scan_step(x[0], x[0], v, x[0]),
                 lambda: pal.palimpsa_gated_scan_backward(x, x, v, None, None, None, None, x, x),
                 lambda: pal.palimpsa_layer_norm(x), lambda: pal.palimpsa_layer_norm_backward(x, None, x, x)):
        with pytest.raises(ValueError, match="device tensors"):
            call()


def test_binding_checks_rows():
    """The rows of the norm's arrays: any leading dimensions when contiguous, up to three when not."""
    f = lambda t: norm._token_rows(t, "t", t, t.get_device())  # noqa: E731
    assert f(torch.zeros(2, 3, 4, 8)) == 0 and f(torch.zeros(5, 16)[:, :8]) == 16 and f(torch.zeros(2, 3, 24)[..., 8:16]) == 24
    for t in (torch.zeros(2, 2, 3, 16)[..., :8], torch.zeros(2, 8, 3).transpose(1, 2), torch.zeros(2, 4, 8)[:, :3]):
        with pytest.raises(ValueError):
            f(t)
    x = torch.zeros(2, 3, 8)
    with pytest.raises(TypeError):
        norm._token_rows(x.bfloat16(), "residual", x, -1)
    with pytest.raises(ValueError):
        norm._token_rows(x[:1], "residual", x, -1)
    with pytest.raises(ValueError):
        norm._shape(torch.zeros(8), "palimpsa_layer_norm")


def test_binding_checks_the_gates():
    x, v = torch.zeros(2, 3, 8), torch.ones(8)
    call = lambda **kw: gated._inputs(**dict(dict(x=x, r=x, A=v, i=x, z=None, r_bias=None, i_bias=v, dev=-1, lead=2), **kw))  # noqa: E731
    with pytest.raises(ValueError, match="i_bias without i"):
        call(i=None)
    with pytest.raises(TypeError):
        call(r=x.bfloat16())
    with pytest.raises(ValueError):
        call(z=x[:, :2])
