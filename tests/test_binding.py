"""The binding as a whole: its names, and where its own tensors come from when a call is given a stream."""
import contextlib
import inspect

import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
import ssd_inputs


def test_a_given_stream_is_the_current_one_during_a_call(monkeypatch):
    """Given by name or by place; without one nothing changes."""
    now, seen = [None], []

    @contextlib.contextmanager
    def use(s):
        now[0] = s
        yield
        now[0] = None

    monkeypatch.setattr(ssd.torch.cuda, "stream", use)

    @ssd._in_stream
    def call(x, y=None, stream=None):
        seen.append((now[0], x, y, stream))

    call(1)
    call(1, stream="s")
    call(1, 2, "t")
    call(1, 2, stream=None)
    assert seen == [(None, 1, None, None), ("s", 1, None, "s"), ("t", 1, 2, "t"), (None, 1, 2, None)] and now == [None]


def test_every_function_with_a_stream_allocates_from_it():
    """The scan's functions by the decorator, the attention layer's by their own allocation."""
    for name in ssd.__all__:
        f = getattr(ssd, name)
        if callable(f) and not inspect.isclass(f) and "stream" in inspect.signature(f).parameters and "attn" not in name and name != "ssd_kv_append":
            assert hasattr(f, "__wrapped__"), name


def test_every_name_of_the_package_is_there():
    assert [n for n in ssd.__all__ if not hasattr(ssd, n)] == []


@pytest.mark.gpu
def test_outputs_of_a_scan_on_a_stream_are_that_streams_memory():
    """No block that was freed on the current stream, where work that uses it may still be queued."""
    cfg = ssd_inputs.config("mamba2_layer")
    g = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in ssd_inputs.make_inputs(cfg, 3).items()}
    s = torch.cuda.Stream()
    args = (g["x"], g["log_a"], g["B"], g["C"])
    want, state = ssd.ssd_forward(*args, chunk=cfg["chunk"], final_state=True)
    grads0 = ssd.ssd_backward(*args, want)
    torch.cuda.synchronize()
    freed = [torch.empty_like(t) for t in (want, state, *grads0.values()) if t is not None and t.numel() * t.element_size() >= 1 << 21 for _ in range(2)]
    places = {t.data_ptr() for t in freed}
    del freed
    y, final = ssd.ssd_forward(*args, chunk=cfg["chunk"], final_state=True, stream=s)
    grads = ssd.ssd_backward(*args, y, stream=s)
    torch.cuda.synchronize()
    assert not places & {t.data_ptr() for t in (y, final, *grads.values()) if t is not None}
    # (dB and dC are summed by atomics: equal up to the order of their sums)
    assert torch.equal(y, want) and torch.equal(final, state) and torch.equal(grads["dx"], grads0["dx"])
