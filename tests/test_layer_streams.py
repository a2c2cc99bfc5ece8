"""Which stream a call of the layer operators runs on, with torch's streams replaced by
stand-ins (no GPU needed: a second device is only a name here)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import nvfp4_bit_block_gb300 as nv
from nvfp4_bit_block_gb300 import layer

DEV0, DEV1 = torch.device("cuda", 0), torch.device("cuda", 1)


class Stream:
    def __init__(self, handle, device=DEV0):  # torch attaches a handle without a device to the current one, here 0
        self.cuda_stream, self.device = handle, torch.device(device)


@pytest.fixture
def seen(monkeypatch):
    """The streams that were current while the binding was called, by device."""
    current, seen = {}, []

    @contextlib.contextmanager
    def entered(stream):
        before = current.get(stream.device)
        current[stream.device] = stream.cuda_stream
        yield
        current[stream.device] = before

    def call(x, *args):
        seen.append(current.get(x.device))
        return (None,) * 4

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=DEV0: Stream(0, device))
    monkeypatch.setattr(layer, "_ext", SimpleNamespace(
        layernorm=call, layernorm_backward=lambda dy, x, *a: call(x)[:3], linear=lambda qa, *a: call(qa)[:3],
        act_backward=lambda dy, *a: call(dy)[:2]))
    return seen


def calls(x):
    return (lambda s: nv.nvfp4_layernorm(x, stream=s), lambda s: nv.nvfp4_layernorm_backward(x, x, None, None, stream=s),
            lambda s: nv.nvfp4_linear(x, x, x, x, x, x, stream=s), lambda s: nv.nvfp4_act_backward(x, x, 0, stream=s))


@pytest.mark.parametrize("device", [DEV0, DEV1])
def test_a_raw_handle_is_a_stream_of_the_tensors_device(seen, device):
    for k, call in enumerate(calls(SimpleNamespace(device=device, is_cuda=True))):
        call(100 + k)
        call(0)
        call(Stream(200 + k, device))
        assert seen[-3:] == [100 + k, 0, 200 + k]


def test_a_stream_of_another_device_is_refused(seen):
    for call in calls(SimpleNamespace(device=DEV1, is_cuda=True)):
        with pytest.raises(ValueError, match="cuda:1"):
            call(Stream(300, DEV0))
    assert not seen


def test_what_is_no_cuda_tensor_is_left_to_the_call(seen):
    call = calls(SimpleNamespace(device=torch.device("cpu"), is_cuda=False))[0]
    call(400)
    assert seen == [None]
