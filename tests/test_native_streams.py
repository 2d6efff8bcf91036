"""Which stream the native calls make current for a stream argument, with the
torch streams replaced by recorders (no GPU)."""
import contextlib
import types

import pytest
import torch

import grad_row_online_gb300 as g

HERE, THERE = torch.device("cuda:0"), torch.device("cuda:1")


class Stream:
    """Stands in for torch.cuda.Stream; the current device is cuda:0."""

    def __init__(self, handle, device=None):
        self.cuda_stream, self.device = handle, HERE if device is None else torch.device(device)


@pytest.fixture
def log(monkeypatch):
    entered, calls = [], []

    @contextlib.contextmanager
    def stream(s):
        entered.append(s)
        yield

    def call(*args):
        calls.append(args)
        return {}

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(g, "_calls", types.SimpleNamespace(
        token_logps=call, token_logps_grad=call, clip_grad_norm=call))
    return types.SimpleNamespace(entered=entered, calls=calls)


CALLS = {
    "logps": lambda t, s: g.grpo_token_logps(t, None, stream=s),
    "grad": lambda t, s: g.grpo_token_logps_grad(t, None, None, None, stream=s),
    "clip": lambda t, s: g.grpo_clip_grad_norm([t], 1.0, stream=s),
    "clip of an iterator": lambda t, s: g.grpo_clip_grad_norm(iter([t]), 1.0, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [HERE, THERE])
def test_a_handle_is_a_stream_of_the_tensors_device(log, name, device):
    CALLS[name](types.SimpleNamespace(device=device), 77)
    assert [(s.cuda_stream, s.device) for s in log.entered] == [(77, device)]
    assert len(log.calls) == 1


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(log, name):
    tensor = types.SimpleNamespace(device=THERE)
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](tensor, Stream(5, HERE))
    assert not log.calls
    CALLS[name](tensor, Stream(5, THERE))
    assert len(log.calls) == 1 and log.entered[-1].device == THERE


def test_what_is_no_cuda_tensor_is_left_to_the_call(log):
    """(the native call refuses it)"""
    for t in (types.SimpleNamespace(device=torch.device("cpu")), None):
        for name in CALLS:
            CALLS[name](t, Stream(5, HERE))
            CALLS[name](t, 6)
    g.grpo_clip_grad_norm([], 1.0, stream=Stream(5, THERE))
    assert log.entered[-1].device == THERE
    g.grpo_clip_grad_norm([], 1.0, stream=7)
    assert log.entered[-1].device == HERE
