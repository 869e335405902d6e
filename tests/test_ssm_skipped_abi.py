"""Refusals of palimpsa_zero_unwritten (CPU): status codes before any device is touched."""
import ctypes

import pytest

import metaplastic_linear_attention_gb300 as pal
from metaplastic_linear_attention_gb300 import build_lib, ssm

ERR_NULL, ERR_SHAPE, ERR_ALIGN = 1, 2, 3
P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    pal.load_library()
    return ssm._library()


@pytest.mark.parametrize("over,code", [
    (dict(cu=None), ERR_NULL), (dict(arrays=False), ERR_NULL), (dict(states=False), ERR_NULL), (dict(p=[P, 0]), ERR_NULL),
    (dict(q=[0, P]), ERR_NULL), (dict(T=0, longest=0, q=[0, P]), ERR_NULL), (dict(n=7), ERR_SHAPE), (dict(m=7), ERR_SHAPE),
    (dict(n=-1), ERR_SHAPE), (dict(m=-1), ERR_SHAPE), (dict(n=9, m=0), ERR_SHAPE), (dict(n=0, m=9), ERR_SHAPE), (dict(B=0), ERR_SHAPE),
    (dict(T=-1), ERR_SHAPE), (dict(p=[P, P + 8]), ERR_ALIGN), (dict(q=[P, P + 4]), ERR_ALIGN), (dict(w=[16, 24]), ERR_ALIGN),
    (dict(v=[8, 16]), ERR_ALIGN), (dict(w=[16, -16]), ERR_SHAPE), (dict(v=[16, -16]), ERR_SHAPE),
    (dict(v=[16, 1 << 40]), ERR_SHAPE), (dict(cu=P + 1), ERR_ALIGN), (dict(longest=-1), ERR_SHAPE), (dict(longest=101), ERR_SHAPE),
])
def test_zero_unwritten_refusals(lib, over, code):
    a = dict(p=[P, P], w=[16, 32], n=2, q=[P, P], v=[16, 32], m=2, cu=P, B=3, T=100, longest=50, arrays=True, states=True) | over
    arr = lambda t, v: (t * 2)(*v)  # noqa: E731
    p = arr(ctypes.c_void_p, a["p"]) if a["arrays"] else None
    q = arr(ctypes.c_void_p, a["q"]) if a["states"] else None
    assert lib.palimpsa_zero_unwritten(p, arr(ctypes.c_longlong, a["w"]), a["n"], q, arr(ctypes.c_longlong, a["v"]), a["m"],
                                       a["cu"], a["B"], a["T"], a["longest"], None) == code
