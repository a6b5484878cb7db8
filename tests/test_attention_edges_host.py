"""The attention layer at its edges, on a machine without a GPU: what the binding and the C entry points refuse, and
where a call's memory comes from."""
import contextlib
import ctypes
import os

import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from ssd_chunked_scan_02_amd import attention
from ssd_chunked_scan_02_amd.attention import AttnCache, AttnDims

INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.library_path()):
        from ssd_chunked_scan_02_amd.build import build
        build()
    return ssd.load_library()


def _dims(**kw):
    d = dict(nseq=2, total_q=100, total_k=100, nheads=4, nkvheads=2, headdim=64, q_stride=0, k_stride=0, v_stride=0, scale=0.125,
             softcap=0.0, dtype=1, causal=1, num_buckets=32, max_distance=128, bidirectional=0)
    d.update(kw)
    return AttnDims(**d)


def _cache(**kw):
    d = dict(nseq=3, nheads=8, nkvheads=2, headdim=64, num_pages=10, page_size=16, max_pages=4, q_stride=0, k_stride=0, v_stride=0,
             scale=0.125, softcap=0.0, dtype=1, num_buckets=32, max_distance=128, bidirectional=0)
    d.update(kw)
    return AttnCache(**d)


# The four entry points: arguments in the call's order, those that are inputs, and those that are written.
ENTRIES = {
    "ssd_attn_forward": ("cu_q cu_k prefix q k v slopes table y lse", "y lse"),
    "ssd_attn_backward": ("cu_q cu_k prefix q k v slopes table y lse dy dq dk dv dtable ws", "dq dk dv dtable ws"),
    "ssd_attn_decode": ("q kc vc bt sl slopes table y ws", "y ws"),
    "ssd_kv_append": ("cu sl bt k v q inv kc vc qo", "kc vc qo"),
}


def _entry(lib, name, at, dims=None):
    """The entry point's status, its pointers taken from ``at`` by name."""
    a = [at.get(n) for n in ENTRIES[name][0].split()]
    if name == "ssd_attn_backward" or name == "ssd_attn_decode":
        a.append(1 << 40)
    if name == "ssd_kv_append":
        a = [3] + a[:7] + [8, 0] + a[7:]
    d = dims if dims is not None else _dims() if name in ("ssd_attn_forward", "ssd_attn_backward") else _cache()
    return getattr(lib, name)(ctypes.byref(d), *a, None)


@pytest.mark.parametrize("name", ENTRIES)
@pytest.mark.parametrize("bias", ["slopes", "table"])
def test_outputs_and_workspace_are_nobody_elses(lib, name, bias):
    """Every output and workspace that is the pointer of any input, or of another output, is refused.  (Addresses that
    nothing follows: no call of this test may pass its checks.)"""
    every, written = (x.split() for x in ENTRIES[name])
    at = {n: (1 << 20) + 4096 * i for i, n in enumerate(every)}
    at[{"slopes": "table", "table": "slopes"}[bias]] = None
    if bias == "slopes":
        at["dtable"] = None
    pairs = [(o, x) for o in written for x in every if x != o and at.get(o) and at.get(x)]
    assert len(pairs) >= len(written)
    for o, x in pairs:
        assert _entry(lib, name, dict(at, **{o: at[x]})) == INVALID, (o, x)


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


SENTENCES = dict(nseq=1 << 20, total_q=1 << 20, total_k=1 << 20, nheads=16, nkvheads=16)  # one token each: 2^24 workgroups and more


def test_more_workgroups_than_a_launch_holds(lib):
    """Refused before the first launch, the backward pass's second kernel included."""
    def at(name):
        a = {n: (1 << 20) + 4096 * i for i, n in enumerate(ENTRIES[name][0].split())}
        return dict(a, slopes=None, table=None, dtable=None, prefix=None)

    assert _entry(lib, "ssd_attn_forward", at("ssd_attn_forward"), _dims(**SENTENCES)) == UNSUPPORTED
    assert _entry(lib, "ssd_attn_backward", at("ssd_attn_backward"), _dims(**SENTENCES)) == UNSUPPORTED
    # eight waves a workgroup: half as many
    half = _dims(**dict(SENTENCES, nseq=1 << 19, headdim=128))
    assert _entry(lib, "ssd_attn_backward", at("ssd_attn_backward"), half) == UNSUPPORTED
    cache = _cache(nseq=1 << 20, nheads=16, nkvheads=16)
    assert _entry(lib, "ssd_attn_decode", at("ssd_attn_decode"), cache) == UNSUPPORTED


def test_a_table_without_rows_is_refused():
    """Its address is null, which the library takes for no table."""
    cpu = torch.device("cpu")
    for table in (torch.zeros(0, 4), torch.zeros(1, 4), torch.zeros(4)):
        with pytest.raises(ValueError, match="buckets"):
            attention._bias_args(None, table, 4, cpu)


def test_short_caches_are_split_where_eight_waves_fill_a_cu(lib):
    """Eight waves a workgroup need no workspace; in fp32 at 128 wide only where that is faster than splitting."""
    def need(**kw):
        return ssd.ssd_attn_decode_workspace_bytes(_cache(**dict(dict(nseq=16, nheads=32, nkvheads=8, headdim=128, page_size=64), **kw)))

    assert need(dtype=1, max_pages=16) == 0 and need(dtype=0, headdim=64, max_pages=16) == 0
    assert need(dtype=0, max_pages=16) > 0 and need(dtype=0, max_pages=4) == 0
    assert need(dtype=0, max_pages=16, nseq=32) == 0 and need(dtype=0, max_pages=17, nseq=32) > 0
