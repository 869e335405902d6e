"""The argument `stream` of the gated scan and the layer norm on the GPU: a call on another stream comes after what
the current one has queued, and its results are the plain call's bits. Every buffer it reads or writes is written,
and read, behind long work on the current stream; before that work the buffers hold other valid values."""
import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
B, T, D = 3, 200, 64
ROWS = B * T
CU = [[0, 1, 2, ROWS], [0, 50, 250, ROWS]]     # before and after


def _inputs(seed, lead, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, dtype=F32: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    t = lambda: r(*lead, D, dtype=dtype)  # noqa: E731
    ckpt = pal.palimpsa_gated_scan_checkpoint_shape(B, T if len(lead) == 2 else ROWS, D, len(lead) == 1)
    return dict(x=t(), r=t(), A=0.1 + torch.rand(D, generator=g, device=DEV), i=t(), z=t(), rb=r(D), ib=r(D), h=r(B, D), dy=t(),
                dh=r(B, D), y=t(), ckpt=r(*ckpt), w=r(D), b=r(D), res=t(), ds=t(), s=t(),
                stats=torch.rand((*lead, 2), generator=g, device=DEV))


GATES = ("x", "r", "A", "i", "z", "rb", "ib")
CALLS = {  # operator: lambda of the buffers and keywords
    "scan": lambda i, kw: pal.palimpsa_gated_scan(*(i[k] for k in GATES), i["h"], y=i["y"], h_T=i["h"], **kw),
    "scan fresh": lambda i, kw: pal.palimpsa_gated_scan(*(i[k] for k in GATES), i["h"], **kw),
    # (the checkpoints of a packed batch have slots that no sequence owns, which stay as they were)
    "scan_checkpointed": lambda i, kw: pal.palimpsa_gated_scan_checkpointed(*(i[k] for k in GATES), i["h"], ckpt=i["ckpt"], **kw),
    "scan_backward": lambda i, kw: tuple(pal.palimpsa_gated_scan_backward(*(i[k] for k in GATES), i["ckpt"], i["dy"], i["dh"],
                                                                          **kw).values()),
    "scan_step": lambda i, kw: (pal.palimpsa_gated_scan_step(*(i[k] for k in GATES[:3]), i["h"], *(i[k] for k in GATES[3:]),
                                                             y=i["y"], **kw), i["h"]),
    "norm": lambda i, kw: pal.palimpsa_layer_norm(i["x"], i["w"], i["b"], i["res"], y=i["y"], s=i["s"], stats=i["stats"],
                                                  want_stats=True, **kw),
    "norm fresh": lambda i, kw: pal.palimpsa_layer_norm(i["x"], i["w"], i["b"], i["res"], want_stats=True, **kw),
    "norm_backward": lambda i, kw: tuple(pal.palimpsa_layer_norm_backward(i["s"], i["w"], i["stats"], i["dy"], i["ds"],
                                                                          **kw).values()),
}
CASES = [(n, f) for n in CALLS for f in (("token",) if n.endswith("step") else ("dense",) if "norm" in n else
                                         ("dense", "packed", "offsets"))]


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
