"""The argument `stream` of the gated scan and the layer norm, on the host (CPU): a call waits for the current stream and
enters its own before it does anything else. The streams are stand-ins that write down what is asked of them."""
import contextlib

import pytest
import torch

import metaplastic_linear_attention_gb300 as pal

ARGS = dict(palimpsa_gated_scan=3, palimpsa_gated_scan_checkpointed=3, palimpsa_gated_scan_step=4,
            palimpsa_gated_scan_backward=9, palimpsa_layer_norm=1, palimpsa_layer_norm_backward=4)


class Stream:
    device, device_index = torch.device("cuda", 0), 0

    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_stream(self, other):
        self.log.append((self.cuda_stream, "waits for", other.cuda_stream))


@pytest.mark.parametrize("name", ARGS)
def test_every_operator_takes_its_stream_this_way(name, monkeypatch):
    """With no tensor on a device the call itself is refused, after the wait."""
    log = []
    home, side = Stream(1, log), Stream(2, log)

    @contextlib.contextmanager
    def enter(stream):
        log.append(("enter", stream.cuda_stream))
        yield

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: home)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="device tensors"):
        getattr(pal, name)(*[x] * ARGS[name], stream=side)
    assert log == [(2, "waits for", 1), ("enter", 2)]
