"""The argument `stream` of the state-space operators on the GPU: a call on another stream comes after what the
current one has queued. Every buffer it reads or writes (inputs, offsets, states in place, given outputs) is written,
and read, behind long work on the current stream; nothing is synchronised before the call, and its results are
the plain call's bits. Before that work the buffers hold other valid values."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
B, T, D, N, W = 3, 40, 64, 16, 4
ROWS = B * T
CU = [[0, 1, 2, ROWS], [0, 50, 70, ROWS]]     # before and after; the longest sequences differ


def _inputs(seed, lead, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, dtype=F32: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    return dict(x=r(*lead, D, dtype=dtype), dt=r(*lead, D, dtype=dtype), A=0.3 + torch.rand((D, N), generator=g, device=DEV),
                B=r(*lead, 1, N, dtype=dtype), C=r(*lead, 1, N, dtype=dtype), D=r(D), z=r(*lead, D, dtype=dtype), bias=r(D) - 2,
                h=r(B, D, N), w=r(D, W), wb=r(D), st=r(B, W - 1, D, dtype=dtype), dy=r(*lead, D, dtype=dtype), dh=r(B, D, N),
                y=r(*lead, D, dtype=dtype),
                ckpt=r(*pal.palimpsa_selective_scan_checkpoint_shape(B, T, D, N) if len(lead) == 2
                       else pal.palimpsa_selective_scan_checkpoint_shape(B, ROWS, D, N, True)))


SCAN = ("x", "dt", "A", "B", "C", "D", "z", "bias")
CALLS = {  # operator: lambda of the buffers and keywords
    "conv": lambda i, kw: (*pal.palimpsa_causal_conv(i["x"], i["w"], i["wb"], i["st"], y=i["y"], state_T=i["st"], **kw),),
    "conv fresh": lambda i, kw: pal.palimpsa_causal_conv(i["x"], i["w"], i["wb"], i["st"], **kw),
    "conv_backward": lambda i, kw: tuple(pal.palimpsa_causal_conv_backward(i["x"], i["w"], i["wb"], i["st"], i["dy"], i["st"],
                                                                           **kw).values()),
    "scan": lambda i, kw: pal.palimpsa_selective_scan(*(i[k] for k in SCAN), i["h"], y=i["y"], h_T=i["h"], **kw),
    "scan fresh": lambda i, kw: pal.palimpsa_selective_scan(*(i[k] for k in SCAN), i["h"], **kw),
    "scan_checkpointed": lambda i, kw: pal.palimpsa_selective_scan_checkpointed(*(i[k] for k in SCAN), i["h"], ckpt=i["ckpt"], **kw),
    "scan_backward": lambda i, kw: tuple(pal.palimpsa_selective_scan_backward(*(i[k] for k in SCAN), i["h"], i["ckpt"], i["dy"],
                                                                              i["dh"], **kw).values()),
    "conv_step": lambda i, kw: (pal.palimpsa_causal_conv_step(i["x"], i["w"], i["wb"], i["st"], y=i["y"], **kw), i["st"]),
    "scan_step": lambda i, kw: (pal.palimpsa_selective_scan_step(*(i[k] for k in SCAN[:5]), i["h"], *(i[k] for k in SCAN[5:]),
                                                                 y=i["y"], **kw), i["h"]),
}
CASES = [(n, "token" if n.endswith("step") else form) for n in CALLS for form in
         (("dense",) if n.endswith("step") else ("dense", "packed", "offsets"))]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name,form", CASES)
def test_a_call_on_another_stream_comes_after_the_current_ones_work(name, form, dtype):
    lead = (B,) if form == "token" else (B, T) if form == "dense" else (ROWS,)
    old, new = (_inputs(seed, lead, dtype) for seed in (1, 2))
    i = {k: v.clone() for k, v in old.items()}
    kw = {}
    if form in ("packed", "offsets"):                 # with "offsets", the longest sequence is read from them
        cus = [torch.tensor(c, dtype=torch.int32, device=DEV) for c in CU]
        cu = cus[0].clone()
        kw = dict(cu_seqlens=cu) if form == "offsets" else dict(cu_seqlens=cu, max_seqlen=ROWS)
    call = CALLS[name]
    ref = {k: v.clone() for k, v in new.items()}
    want = [t.clone() for t in call(ref, dict(kw, cu_seqlens=cus[1]) if kw else {})]
    busy = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(15):
        busy = busy @ busy * 1e-2
    kept = i["y"].clone()                             # reads what the call may write
    for k in i:
        i[k].copy_(new[k])
    if kw:
        cu.copy_(cus[1])
    assert not torch.cuda.current_stream().query()    # the current stream is still at work
    got = call(i, dict(kw, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(kept, old["y"])
    assert pal.palimpsa_get_device_status() == 0
