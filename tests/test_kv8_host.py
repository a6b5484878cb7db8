"""The 8-bit cache's and the rotation's C ABI and binding on a machine without a GPU: every declared function is exported,
workspaces are sized and bad arguments refused before any HIP call; the frequencies of long contexts."""
import ctypes
import math
import os
import re

import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from ssd_chunked_scan_02_amd.attention import AttnCache
from ssd_chunked_scan_02_amd.kv8 import Kv8Pages
from ssd_chunked_scan_02_amd.rotary import RotaryDims

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGN = 0, -1, -2, -3
P = 1 << 20  # an aligned address that no refused call follows


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.library_path()):
        from ssd_chunked_scan_02_amd.build import build
        build()
    return ssd.load_library()


@pytest.mark.parametrize("header,want", [
    ("ssd_kv8.h", ["ssd_kv8_append", "ssd_kv8_decode", "ssd_kv8_decode_workspace_bytes", "ssd_kv8_read"]),
    ("ssd_rotary.h", ["ssd_rotate"])])
def test_header_and_exports(lib, header, want):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(ssd_[a-z0-9_]+)\s*\(", text))) == want
    for n in want:
        assert hasattr(lib, n) and hasattr(ssd, n) and n in ssd.__all__


def _cache(**kw):
    d = dict(nseq=3, nheads=8, nkvheads=2, headdim=64, num_pages=10, page_size=16, max_pages=4, q_stride=0, k_stride=0, v_stride=0,
             scale=0.125, softcap=0.0, dtype=1, num_buckets=32, max_distance=128, bidirectional=0)
    d.update(kw)
    return AttnCache(**d)


def _pages(k=P + 64, v=P + 128, k_scale=P + 192, v_scale=P + 256, format=0):
    return Kv8Pages(k, v, k_scale, v_scale, format)


def _append(lib, d=None, pages=None, tokens=None, cu=None, sl=P, bt=P, k=P, v=P, q=None, inv=None, rot=0, inter=0, q_out=None):
    d = d or _cache()
    return lib.ssd_kv8_append(ctypes.byref(d), ctypes.byref(pages or _pages()), d.nseq if tokens is None else tokens, cu, sl, bt, k, v, q, inv,
                              rot, inter, q_out, None)


def _decode(lib, d=None, pages=None, q=P, bt=P, sl=P, slopes=None, table=None, y=P + 512, ws=P + 1024, n=1 << 30):
    return lib.ssd_kv8_decode(ctypes.byref(d or _cache()), ctypes.byref(pages or _pages()), q, bt, sl, slopes, table, y, ws, n, None)


def _read(lib, d=None, pages=None, tokens=30, cu=None, sl=P, bt=P, k=P + 512, v=P + 1024):
    return lib.ssd_kv8_read(ctypes.byref(d or _cache()), ctypes.byref(pages or _pages()), tokens, cu, sl, bt, k, v, None)


SHAPES = [(dict(page_size=8), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(num_pages=-1), INVALID), (dict(num_pages=1 << 31), INVALID),
          (dict(max_pages=-1), INVALID), (dict(max_pages=1 << 28), UNSUPPORTED), (dict(headdim=256), UNSUPPORTED), (dict(headdim=16), UNSUPPORTED),
          (dict(nheads=7), INVALID), (dict(dtype=3), INVALID), (dict(nseq=-1), INVALID)]


@pytest.mark.parametrize("change,want", SHAPES, ids=range(len(SHAPES)))
def test_shape_refusals(lib, change, want):
    c = _cache(**change)
    assert _append(lib, c) == want and _decode(lib, c) == want and _read(lib, c) == want


def test_page_refusals(lib):
    for call in (_append, _decode, _read):
        for bad in (dict(format=2), dict(format=-1), dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None)):
            assert call(lib, pages=_pages(**bad)) == INVALID, (call, bad)
        for bad in (dict(k=P + 72), dict(v=P + 130), dict(k_scale=P + 196), dict(v_scale=P + 264)):
            assert call(lib, pages=_pages(**bad)) == ALIGN, (call, bad)


def test_append_refusals(lib):
    for bad in (dict(k=None), dict(v=None), dict(sl=None), dict(bt=None), dict(q=P), dict(q_out=P + 512), dict(rot=16), dict(inv=P, rot=40),
                dict(inv=P, rot=-8), dict(inter=2), dict(tokens=-1), dict(tokens=4), dict(tokens=1 << 31, cu=P),
                dict(q=P, q_out=P), dict(q=P, q_out=P + 64), dict(pages=_pages(k=P)), dict(pages=_pages(k=P + 128)), dict(pages=_pages(v_scale=P))):
        assert _append(lib, **bad) == INVALID, bad
    assert _append(lib, inv=P, rot=4) == UNSUPPORTED
    for bad in (dict(k=P + 8), dict(v=P + 8), dict(q=P + 8, q_out=P + 512), dict(q=P, q_out=P + 520), dict(sl=P + 4), dict(bt=P + 2),
                dict(cu=P + 4), dict(inv=P + 4, rot=8), dict(d=_cache(k_stride=132))):
        assert _append(lib, **bad) == ALIGN, bad
    assert _append(lib, d=_cache(q_stride=100)) == INVALID
    assert _append(lib, d=_cache(nseq=0)) == OK and _append(lib, tokens=0, cu=P) == OK


def test_decode_refusals_and_workspace(lib):
    for bad in (dict(q=None), dict(y=None), dict(bt=None), dict(sl=None), dict(slopes=P, table=P), dict(d=_cache(scale=math.nan)),
                dict(d=_cache(softcap=-1.0)), dict(d=_cache(num_buckets=1), table=P), dict(y=P), dict(y=P + 64), dict(ws=P),
                dict(d=_cache(max_pages=1000), n=8), dict(d=_cache(max_pages=1000), ws=None), dict(d=_cache(max_pages=1000), ws=P + 512)):
        assert _decode(lib, **bad) == INVALID, bad
    for bad in (dict(q=P + 8), dict(y=P + 520), dict(ws=P + 1032), dict(sl=P + 4), dict(bt=P + 2), dict(slopes=P + 4)):
        assert _decode(lib, **bad) == ALIGN, bad
    assert _decode(lib, d=_cache(nseq=0)) == OK
    assert ssd.ssd_kv8_decode_workspace_bytes(_cache()) == 0
    assert ssd.ssd_kv8_decode_workspace_bytes(_cache(max_pages=1000)) == 3 * 8 * 64 * (64 * 4 + 8)
    assert ssd.ssd_kv8_decode_workspace_bytes(_cache(page_size=4)) == 0


def test_read_refusals(lib):
    for bad in (dict(k=None), dict(v=None), dict(sl=None), dict(bt=None), dict(tokens=-3), dict(tokens=31), dict(tokens=1 << 31, cu=P),
                dict(k=P), dict(v=P + 64), dict(k=P + 1024)):
        assert _read(lib, **bad) == INVALID, bad
    for bad in (dict(k=P + 520), dict(v=P + 1028), dict(sl=P + 4), dict(bt=P + 2), dict(cu=P + 4)):
        assert _read(lib, **bad) == ALIGN, bad
    assert _read(lib, tokens=0) == OK and _read(lib, d=_cache(nseq=0), tokens=31) == OK


def _rotary(**kw):
    d = dict(nseq=2, total=20, nheads=4, nkvheads=2, headdim=64, q_stride=0, k_stride=0, magnitude=1.0, dtype=1, rot_pairs=32, interleaved=0, inverse=0)
    d.update(kw)
    return RotaryDims(**d)


ROTATE = [
    (dict(nseq=-1), {}, INVALID), (dict(total=-2), {}, INVALID), (dict(total=1 << 31), {}, INVALID), (dict(total=21), {}, INVALID),
    (dict(nheads=0), {}, INVALID), (dict(nheads=1 << 17), {}, INVALID), (dict(nkvheads=0), {}, INVALID), (dict(headdim=0), {}, INVALID),
    (dict(headdim=48, rot_pairs=16), {}, UNSUPPORTED), (dict(headdim=256), {}, UNSUPPORTED), (dict(dtype=2), {}, INVALID), (dict(interleaved=2), {}, INVALID),
    (dict(inverse=-1), {}, INVALID), (dict(magnitude=math.inf), {}, INVALID), (dict(rot_pairs=40), {}, INVALID), (dict(rot_pairs=-8), {}, INVALID),
    (dict(rot_pairs=12), {}, UNSUPPORTED), (dict(q_stride=100), {}, INVALID), (dict(q_stride=260), {}, ALIGN), (dict(k_stride=1 << 24), {}, INVALID),
    ({}, dict(q=None), INVALID), ({}, dict(q_out=None), INVALID), ({}, dict(k=None), INVALID), ({}, dict(k_out=None), INVALID),
    ({}, dict(inv=None), INVALID), ({}, dict(q_out=P), INVALID), ({}, dict(k_out=P + 64), INVALID), ({}, dict(cu=P + 64), INVALID),
    ({}, dict(q=P + 8), ALIGN), ({}, dict(k=P + 8), ALIGN), ({}, dict(q_out=P + 72), ALIGN), ({}, dict(k_out=P + 136), ALIGN),
    ({}, dict(inv=P + 4), ALIGN), ({}, dict(cu=P + 4), ALIGN), ({}, dict(start=P + 4), ALIGN),
    (dict(nseq=0), {}, OK), (dict(total=0), dict(q=None, q_out=None, k=None, k_out=None), OK),
]


@pytest.mark.parametrize("dims,args,want", ROTATE, ids=range(len(ROTATE)))
def test_rotate_refusals(lib, dims, args, want):
    a = dict(cu=None, start=None, q=P, k=P, inv=P, q_out=P + 64, k_out=P + 128)
    a.update(args)
    assert lib.ssd_rotate(ctypes.byref(_rotary(**dims)), *[a[n] for n in ("cu", "start", "q", "k", "inv", "q_out", "k_out")], None) == want


def test_rotate_refuses_no_dims(lib):
    assert lib.ssd_rotate(None, None, None, P, None, P, P + 64, None, None) == INVALID


def test_frequencies():
    """Unscaled: base^(-2 r / dim).  Each way of scaling: its ends, and all of it at factor 1."""
    plain, m = ssd.ssd_rotary_frequencies(128)
    want = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    assert m == 1.0 and plain.dtype == torch.float32 and torch.equal(plain, want.float())
    for how in ("linear", "base", "parts"):
        f, m = ssd.ssd_rotary_frequencies(128, how=how)
        assert m == 1.0 and torch.equal(f, plain), how
    assert torch.equal(ssd.ssd_rotary_frequencies(128, factor=4.0, how="linear")[0], (want / 4).float())
    f, m = ssd.ssd_rotary_frequencies(128, factor=4.0, how="base")
    assert m == 1.0 and f[0] == 1.0 and math.isclose(f[-1], want[-1] / 4, rel_tol=1e-6) and torch.all(f[1:] < plain[1:])
    f, m = ssd.ssd_rotary_frequencies(128, factor=4.0, how="parts", trained=4096)
    turns = 4096 * want / (2 * math.pi)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1.0)
    assert torch.equal(f[turns >= 32], plain[turns >= 32]) and torch.equal(f[turns <= 1], (want / 4).float()[turns <= 1])
    mid = (turns < 32) & (turns > 1)
    assert torch.all(f[mid] < plain[mid]) and torch.all(f[mid] > plain[mid] / 4) and torch.all(f[1:] < f[:-1])
    for bad in (dict(dim=0), dict(dim=7), dict(dim=8, base=1.0), dict(dim=8, factor=0.5), dict(dim=8, how="other"),
                dict(dim=8, factor=2.0, fast=1.0, slow=1.0), dict(dim=8, factor=2.0, slow=0.0)):
        with pytest.raises(ValueError):
            ssd.ssd_rotary_frequencies(**bad)


def test_binding_refuses_cpu_tensors():
    kc, s = torch.zeros((2, 16, 2, 32), dtype=torch.int8), torch.zeros((2, 16, 2))
    bt, sl, x = torch.zeros((1, 2), dtype=torch.int32), torch.tensor([4]), torch.zeros((1, 2, 32))
    with pytest.raises(ValueError):
        ssd.ssd_kv8_append(x, x, kc, kc, s, s, bt, sl)
    with pytest.raises(ValueError):
        ssd.ssd_kv8_decode(x, kc, kc, s, s, bt, sl)
    with pytest.raises(ValueError):
        ssd.ssd_kv8_read(kc, kc, s, s, bt, sl, None, 4)
    with pytest.raises(ValueError):
        ssd.ssd_rotate(x, torch.ones(16), cu_seqlens=torch.tensor([0, 1]))
