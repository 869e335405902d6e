"""A layer of the operators together, as a model runs them: the residual addition and norm, a joint projection (a plain
product), the convolution on its first part, the gated scan with gates from the others, and the next layer's norm. Forward and
backward in fp32 against the same layer in 64 bits, a packed batch against its sequences, and tokens after a prompt.

Bars: every operator's own is 2e-5 forward, 4e-5 backward; four of them in a row, each passing on its input's error with a
factor of about one (the norm divides by deviations of about one, the projections are orthogonal): 1e-4 and 2e-4."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal
from oracle import ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64, F32 = torch.float64, torch.float32
D, W, EPS = 64, 4, 1e-5


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _r(g, *shape, scale=1.0):
    return scale * torch.randn(shape, generator=g)


def _params(seed):
    g = _gen(seed)
    q, _ = torch.linalg.qr(_r(g, 4 * D, D).to(F64))          # orthonormal columns: joint.T joint = 1
    return dict(w1=1 + _r(g, D, scale=0.2), b1=_r(g, D, scale=0.2), joint=2 * q.to(F32), conv=_r(g, D, W, scale=0.5), cb=_r(g, D, scale=0.1),
                A=0.1 + torch.rand(D, generator=g), rb=_r(g, D, scale=0.5), ib=_r(g, D, scale=0.5), w2=1 + _r(g, D, scale=0.2),
                b2=_r(g, D, scale=0.2))


def _layer(p, x, res, **kw):
    """Forward with what the backward needs. x, res [..., D]."""
    k = {}
    k["n1"], k["s1"], k["st1"] = pal.palimpsa_layer_norm(x, p["w1"], p["b1"], res, eps=EPS, want_stats=True)
    k["proj"] = k["n1"] @ p["joint"].T                        # [..., 4 D]: the convolution's input, the gates r, i and z
    u, r, i, z = k["proj"].split(D, -1)
    k["c"], _ = pal.palimpsa_causal_conv(u, p["conv"], p["cb"], **kw)
    k["y"], k["h"], k["ckpt"] = pal.palimpsa_gated_scan_checkpointed(k["c"], r, p["A"], i, z, p["rb"], p["ib"], **kw)
    k["n2"], k["s2"], k["st2"] = pal.palimpsa_layer_norm(k["y"], p["w2"], p["b2"], k["s1"], eps=EPS, want_stats=True)
    return k


def _layer_backward(p, k, dn2, ds2, **kw):
    """Gradients of <dn2, n2> + <ds2, s2>: of the input x (and res) and of the parameters."""
    u, r, i, z = k["proj"].split(D, -1)
    g2 = pal.palimpsa_layer_norm_backward(k["s2"], p["w2"], k["st2"], dn2, ds2)
    gs = pal.palimpsa_gated_scan_backward(k["c"], r, p["A"], i, z, p["rb"], p["ib"], k["ckpt"], g2["dx"], want_state_grad=False, **kw)
    gc = pal.palimpsa_causal_conv_backward(u, p["conv"], p["cb"], None, gs["dx"], want_state_grad=False, **kw)
    dproj = torch.cat([gc["dx"], gs["dr"], gs["di"], gs["dz"]], -1)
    dn1 = dproj @ p["joint"]
    g1 = pal.palimpsa_layer_norm_backward(k["s1"], p["w1"], k["st1"], dn1, g2["dx"])
    return dict(x=g1["dx"], w1=g1["dweight"], b1=g1["dbias"], joint=dproj.reshape(-1, 4 * D).T @ k["n1"].reshape(-1, D), conv=gc["dweight"],
                cb=gc["dbias"], A=gs["dA"], rb=gs["dr_bias"], ib=gs["di_bias"], w2=g2["dweight"], b2=g2["dbias"])


def _oracle(p, x, res, cu, dn2, ds2):
    p = {k: v.to(F64).requires_grad_() for k, v in p.items()}
    x = x.to(F64).requires_grad_()
    s1 = x + res.to(F64)
    proj = ssm.layer_norm(s1, p["w1"], p["b1"], EPS) @ p["joint"].T
    u, r, i, z = proj.split(D, -1)
    c, _ = ssm.conv(u, p["conv"], p["cb"], None, cu)
    y, h = ssm.gate(c, r, p["A"], i, z, p["rb"], p["ib"], None, cu)
    s2 = y + s1
    n2 = ssm.layer_norm(s2, p["w2"], p["b2"], EPS)
    loss = (n2 * dn2.to(F64)).sum() + (s2 * ds2.to(F64)).sum()
    leaves = dict(x=x, **p)
    return n2.detach(), h.detach(), dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))


def _near(got, want, bar, what):
    got = got.detach().cpu().to(F64).reshape(want.shape)
    r = float((got - want).norm() / want.norm())
    assert r <= bar, f"{what}: relative L2 {r:.3g} over {bar:.3g}"


@pytest.mark.parametrize("lens,dense", [([130, 130, 130], True), ([77, 1, 200, 33], False)])
def test_layer_forward_and_backward(lens, dense):
    rows, g = sum(lens), _gen(2)
    cu = [sum(lens[:k]) for k in range(len(lens) + 1)]
    x, res, dn2, ds2 = (_r(g, rows, D) for _ in range(4))
    p = _params(1)
    want, wh, grads = _oracle(p, x, res, cu, dn2, ds2)
    shape = (len(lens), -1, D) if dense else (rows, D)
    dev = lambda t: t.reshape(shape).to(DEV)  # noqa: E731
    pd = {k: v.to(DEV) for k, v in p.items()}
    kw = {} if dense else dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_seqlen=max(lens))
    k = _layer(pd, dev(x), dev(res), **kw)
    _near(k["n2"], want, 1e-4, "n2")
    _near(k["h"], wh, 1e-4, "h")
    got = _layer_backward(pd, k, dev(dn2), dev(ds2), **kw)
    for name, v in grads.items():
        _near(got[name], v, 2e-4, name)
    assert pal.palimpsa_get_device_status() == 0


def test_tokens_after_a_prompt():
    """The layer on a prompt of 40 tokens, then one token at a time with its three states, against the whole sequence."""
    B, T, cut, g = 3, 50, 40, _gen(3)
    x, res = (_r(g, B, T, D).to(DEV) for _ in range(2))
    p = {k: v.to(DEV) for k, v in _params(4).items()}
    want = _layer(p, x, res)
    s1, n1 = want["s1"], want["n1"]
    u, r, i, z = (n1 @ p["joint"].T).split(D, -1)
    _, conv_state = pal.palimpsa_causal_conv(u[:, :cut].contiguous(), p["conv"], p["cb"])
    h = torch.zeros(B, D, device=DEV)
    part = lambda t: t[:, :cut].contiguous()  # noqa: E731
    pal.palimpsa_gated_scan(part(want["c"]), part(r), p["A"], part(i), part(z), p["rb"], p["ib"], h, h_T=h)
    for t in range(cut, T):
        n, s, _ = pal.palimpsa_layer_norm(x[:, t], p["w1"], p["b1"], res[:, t], eps=EPS)
        ut, rt, it, zt = (n @ p["joint"].T).split(D, -1)
        c = pal.palimpsa_causal_conv_step(ut, p["conv"], p["cb"], conv_state)
        y = pal.palimpsa_gated_scan_step(c, rt, p["A"], h, it, zt, p["rb"], p["ib"])
        n2, s2, _ = pal.palimpsa_layer_norm(y, p["w2"], p["b2"], s, eps=EPS, s=s)    # the stream, in place
        assert s2 is s
        _near(n2, want["n2"][:, t].cpu().to(F64), 1e-4, f"token {t}")
    _near(h, want["h"].cpu().to(F64), 1e-4, "h")
    assert pal.palimpsa_get_device_status() == 0
