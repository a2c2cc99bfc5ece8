"""Which stream a call of the attention operators runs on, with torch's streams replaced by
stand-ins (no GPU needed: a second device is only a name here)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import nvfp4_bit_block_gb300 as nv
from nvfp4_bit_block_gb300 import attention

DEV0, DEV1 = torch.device("cuda", 0), torch.device("cuda", 1)


class Stream:
    def __init__(self, handle, device=DEV0):
        self.cuda_stream, self.device = handle, torch.device(device)


@pytest.fixture
def seen(monkeypatch):
    current, seen = {}, []

    @contextlib.contextmanager
    def entered(stream):
        before = current.get(stream.device)
        current[stream.device] = stream.cuda_stream
        yield
        current[stream.device] = before

    def call(x, n):
        seen.append(current.get(x.device))
        return (None,) * n

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=DEV0: Stream(0, device))
    monkeypatch.setattr(attention, "_ext", SimpleNamespace(
        qk_rope=lambda q, *a: call(q, 2), qk_rope_backward=lambda dq, *a: call(dq, 4), cache_write=lambda k, *a: call(k, 0),
        cache_read=lambda kc, *a: call(kc, 2), cache_attention=lambda q, *a: call(q, 2)))
    return seen


def calls(x):
    c = nv.KVCache(x, x, x, x, x)
    return (lambda s: nv.nvfp4_qk_rope(x, x, x, x, stream=s), lambda s: nv.nvfp4_qk_rope_backward(x, x, x, x, x, x, stream=s),
            lambda s: nv.nvfp4_cache_write(x, x, c, x, x, x, stream=s),
            lambda s: nv.nvfp4_cache_read(c, x, x, x, tokens=1, stream=s),
            lambda s: nv.nvfp4_cache_attention(x, c, x, x, x, stream=s))


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
