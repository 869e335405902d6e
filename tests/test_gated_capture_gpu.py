"""Calls whose first run in a process comes while a CUDA graph is captured: the library's scratch pool is created then. Each
in a process of its own, against plain calls after it."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = """
import sys, torch
import metaplastic_linear_attention_gb300 as pal
x, A = torch.randn(2, 300, 72, device="cuda"), torch.rand(72, device="cuda") + 0.1
w = torch.randn(72, 4, device="cuda")
ckpt, stats = torch.randn(2, 38, 72, device="cuda"), torch.rand(2, 300, 2, device="cuda") + 0.5
calls = dict(gate=lambda: pal.palimpsa_gated_scan_backward(x, x, A, x, x, None, None, ckpt, x),
             norm=lambda: pal.palimpsa_layer_norm_backward(x, A, stats, x, x),
             conv=lambda: pal.palimpsa_causal_conv_backward(x, w, None, None, x))
call = calls[sys.argv[1]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
want = call()
assert all(torch.equal(got[k], want[k]) for k in want)
assert pal.palimpsa_get_device_status() == 0
"""


@pytest.mark.parametrize("name", ["gate", "norm", "conv"])
def test_a_first_call_inside_a_capture(name):
    r = subprocess.run([sys.executable, "-c", SCRIPT, name], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
