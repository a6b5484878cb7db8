"""The attention layer at its edges, on a machine without a GPU: what the binding and the C entry points refuse, and
where a call's memory comes from."""
import contextlib

import pytest
import torch

from ssd_chunked_scan_02_amd import attention


class _Stream:
    def __init__(self, device):
        self.device, self.cuda_stream = torch.device(device), 0


def test_memory_of_a_call_comes_from_its_stream(monkeypatch):
    """A call's own outputs and workspace are allocated while its stream is the current one."""
    now, seen = [None], []

    @contextlib.contextmanager
    def use(s):
        now[0] = s
        yield
        now[0] = None

    def empty(shape, dtype, device):
        seen.append(now[0])
        return torch.zeros(shape, dtype=dtype)

    monkeypatch.setattr(attention.torch.cuda, "stream", use)
    monkeypatch.setattr(attention.torch, "empty", empty)
    s, dev = _Stream("cuda:0"), torch.device("cuda", 0)
    attention._empty((2, 3), torch.float32, dev, s)
    attention._workspace(None, 64, dev, s)
    attention._empty((2, 3), torch.float32, dev, None)
    assert seen == [s, s, None] and now == [None]


def test_a_stream_of_another_device_is_refused():
    with pytest.raises(ValueError, match="stream"):
        attention._empty((2,), torch.float32, torch.device("cuda", 0), _Stream("cuda:1"))
    with pytest.raises(ValueError, match="stream"):
        attention._call("ssd_attn_forward", torch.device("cuda", 0), _Stream("cuda:1"))
