"""The argument `stream` of the state-space operators, on the host (CPU): the order in which a call waits for the
current stream, enters its own and runs. The streams are stand-ins that write down what is asked of them."""
import contextlib

import pytest
import torch

from metaplastic_linear_attention_gb300 import ssm

OPERATORS = ["palimpsa_causal_conv", "palimpsa_causal_conv_step", "palimpsa_causal_conv_backward",
             "palimpsa_selective_scan", "palimpsa_selective_scan_checkpointed", "palimpsa_selective_scan_step",
             "palimpsa_selective_scan_backward"]


class Stream:
    device, device_index = torch.device("cuda", 0), 0

    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_stream(self, other):
        self.log.append((self.cuda_stream, "waits for", other.cuda_stream))


@pytest.fixture
def streams(monkeypatch):
    log = []
    home, side = Stream(1, log), Stream(2, log)

    @contextlib.contextmanager
    def enter(stream):
        log.append(("enter", stream.cuda_stream))
        yield
        log.append(("leave", stream.cuda_stream))

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: home)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    return log, home, side


def test_a_call_on_another_stream_waits_for_the_current_one(streams):
    log, _, side = streams
    ssm._on_stream(lambda x: log.append("call"))(torch.zeros(1), stream=side)
    assert log == [(2, "waits for", 1), ("enter", 2), "call", ("leave", 2)]


def test_a_call_on_the_current_stream_waits_for_nothing(streams):
    log, home, _ = streams
    for kw in ({}, dict(stream=None), dict(stream=home)):
        ssm._on_stream(lambda x: log.append("call"))(torch.zeros(1), **kw)
    assert log == ["call"] * 3


@pytest.mark.parametrize("name", OPERATORS)
def test_every_operator_takes_its_stream_this_way(streams, name):
    """With no tensor on a device the call itself is refused, after the wait."""
    log, _, side = streams
    x = torch.zeros(2, 8)
    args = dict(palimpsa_causal_conv=4, palimpsa_causal_conv_step=4, palimpsa_causal_conv_backward=5,
                palimpsa_selective_scan=5, palimpsa_selective_scan_checkpointed=5, palimpsa_selective_scan_step=6,
                palimpsa_selective_scan_backward=11)[name]
    with pytest.raises(ValueError, match="device tensors"):
        getattr(ssm, name)(*[x] * args, stream=side)
    assert log[:2] == [(2, "waits for", 1), ("enter", 2)]
