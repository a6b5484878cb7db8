"""Python binding of the paged cache in 8 bits (``include/ssd_kv8.h``): argument marshalling only.

k_cache, v_cache [num_pages, page_size, Hk, D] of torch.int8 or torch.float8_e4m3fn stand, with k_scale, v_scale
[num_pages, page_size, Hk] fp32, for scale * value.  block_table int32 [nseq, max_pages], seq_lens int64 [nseq].
"""
from __future__ import annotations

import ctypes

import torch

from . import _DTYPE_CODE, _in_stream, _on_stream, load_library
from .attention import AttnCache, _addr, _bias_args, _call, _dense, _offsets, _stride, _workspace

SSD_KV8_INT8, SSD_KV8_E4M3 = 0, 1
_FORMAT = {torch.int8: SSD_KV8_INT8, torch.float8_e4m3fn: SSD_KV8_E4M3}


class Kv8Pages(ctypes.Structure):
    """Mirror of ``ssd_kv8_pages``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("format", ctypes.c_int32)]


def declare(lib):
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    cp, gp = ctypes.POINTER(AttnCache), ctypes.POINTER(Kv8Pages)
    lib.ssd_kv8_append.argtypes = [cp, gp, i64] + [vp] * 7 + [i32, i32, vp, vp]
    lib.ssd_kv8_append.restype = i32
    lib.ssd_kv8_decode_workspace_bytes.argtypes = [cp]
    lib.ssd_kv8_decode_workspace_bytes.restype = sz
    lib.ssd_kv8_decode.argtypes = [cp, gp] + [vp] * 7 + [sz, vp]
    lib.ssd_kv8_decode.restype = i32
    lib.ssd_kv8_read.argtypes = [cp, gp, i64] + [vp] * 6
    lib.ssd_kv8_read.restype = i32


def _pages(dtype, dev, heads, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, strides=(0, 0, 0), scale=None, softcap=0.0,
           buckets=0, max_distance=0, bidirectional=False):
    """ssd_attn_cache and ssd_kv8_pages of a call, the cache's arguments checked."""
    if dtype not in _DTYPE_CODE:
        raise TypeError("queries, keys and values must be float32 or bfloat16, got %s" % dtype)
    if k_cache.dtype not in _FORMAT:
        raise TypeError("k_cache must be int8 or float8_e4m3fn, got %s" % k_cache.dtype)
    if not k_cache.is_cuda:
        raise ValueError("k_cache must be a GPU tensor")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, page_size, Hk, D], got shape %s" % (tuple(k_cache.shape),))
    _dense(k_cache, "k_cache", k_cache.shape, k_cache.dtype, dev)
    _dense(v_cache, "v_cache", k_cache.shape, k_cache.dtype, dev)
    _dense(k_scale, "k_scale", k_cache.shape[:3], torch.float32, dev)
    _dense(v_scale, "v_scale", k_cache.shape[:3], torch.float32, dev)
    pages, size, Hk, D = k_cache.shape
    nseq = seq_lens.numel()
    _offsets(seq_lens, "seq_lens", dev, nseq)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [nseq, max_pages]")
    _dense(block_table, "block_table", (nseq, block_table.shape[1]), torch.int32, dev)
    dims = AttnCache(nseq, heads, Hk, D, pages, size, block_table.shape[1], *strides, D ** -0.5 if scale is None else float(scale),
                     float(softcap), _DTYPE_CODE[dtype], buckets, int(max_distance), int(bool(bidirectional)))
    return dims, Kv8Pages(_addr(k_cache), _addr(v_cache), _addr(k_scale), _addr(v_scale), _FORMAT[k_cache.dtype])


@_in_stream
def ssd_kv8_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens=None, inv_freq=None,
                   interleaved: bool = False, q=None, q_out=None, stream=None):
    """Run ``ssd_kv8_append``: ssd_kv_append into 8-bit pages, in place: the keys (rotated) and values of new tokens,
    k, v [tokens,Hk,D], quantised with a scale for each token and head.

    ``cu_seqlens``: int64 offsets of each sequence's new tokens (None: one token per sequence); ``seq_lens`` counts the
    sequences with them.  Returns the rotated q, or None without q."""
    dev = k.device
    strides = [0 if t is None else _stride(t, n, 3, k.dtype, dev) for n, t in (("q", q), ("k", k), ("v", v))]
    tokens, Hk, D = k.shape
    H = Hk if q is None else q.shape[1]
    dims, pages = _pages(k.dtype, dev, H, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, strides)
    if (dims.nkvheads, dims.headdim) != (Hk, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k %s and v %s do not fit the cache %s" % (tuple(k.shape), tuple(v.shape), tuple(k_cache.shape)))
    if q is not None and (q.shape[0], q.shape[2]) != (tokens, D):
        raise ValueError("q %s does not fit k %s" % (tuple(q.shape), tuple(k.shape)))
    if q is not None and H % Hk != 0:
        raise ValueError("q's %d heads are not a multiple of k's %d" % (H, Hk))
    _offsets(cu_seqlens, "cu_seqlens", dev, dims.nseq + 1)
    if cu_seqlens is None and tokens != dims.nseq:
        raise ValueError("%d tokens for %d sequences: give cu_seqlens" % (tokens, dims.nseq))
    if inv_freq is not None:
        _dense(inv_freq, "inv_freq", (inv_freq.numel(),), torch.float32, dev)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out needs q")
    else:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        _dense(q_out, "q_out", q.shape, q.dtype, dev)
    _on_stream(stream, k, v, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, inv_freq, q_out)
    _call("ssd_kv8_append", dev, stream, ctypes.byref(dims), ctypes.byref(pages), tokens, _addr(cu_seqlens), _addr(seq_lens),
          _addr(block_table), _addr(k), _addr(v), _addr(q), _addr(inv_freq), 0 if inv_freq is None else inv_freq.numel(),
          int(bool(interleaved)), _addr(q_out))
    return q_out


def ssd_kv8_decode_workspace_bytes(dims: AttnCache) -> int:
    return int(load_library().ssd_kv8_decode_workspace_bytes(ctypes.byref(dims)))


@_in_stream
def ssd_kv8_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale=None, softcap: float = 0.0, slopes=None,
                   table=None, max_distance: int = 128, bidirectional: bool = False, y=None, workspace=None, stream=None):
    """Run ``ssd_kv8_decode``: ssd_attn_decode over 8-bit pages, one query per sequence, q [nseq,H,D].

    Bias and cap as in ssd_attn_forward.  Returns y [nseq,H,D]."""
    dev = q.device
    stride = _stride(q, "q", 3, q.dtype, dev)
    nseq, H, D = q.shape
    dims, pages = _pages(q.dtype, dev, H, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, (stride, 0, 0), scale, softcap,
                         _bias_args(slopes, table, H, dev), max_distance, bidirectional)
    if dims.nseq != nseq or dims.headdim != D:
        raise ValueError("q %s does not fit %d sequences of head dim %d" % (tuple(q.shape), dims.nseq, dims.headdim))
    if y is None:
        y = torch.empty((nseq, H, D), dtype=q.dtype, device=dev)
    _dense(y, "y", (nseq, H, D), q.dtype, dev)
    workspace, ws_bytes = _workspace(workspace, ssd_kv8_decode_workspace_bytes(dims), dev)
    _on_stream(stream, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, slopes, table, y, workspace)
    _call("ssd_kv8_decode", dev, stream, ctypes.byref(dims), ctypes.byref(pages), _addr(q), _addr(block_table), _addr(seq_lens),
          _addr(slopes), _addr(table), _addr(y), _addr(workspace), ws_bytes)
    return y


@_in_stream
def ssd_kv8_read(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, tokens: int, dtype=torch.bfloat16, k=None,
                 v=None, stream=None):
    """Run ``ssd_kv8_read``: the keys and values that the pages stand for, packed, for ssd_attn_forward over what is cached.

    Row cu_seqlens[s] + i of k, v [tokens,Hk,D] is position i of sequence s; ``cu_seqlens`` int64 [nseq + 1] on the GPU, or
    None for tokens / nseq rows of each.  ``tokens`` is the host's count of rows.  Rows past a sequence's length are zeros,
    rows of no sequence are not written.  Returns (k, v)."""
    dev = k_cache.device
    dims, pages = _pages(dtype, dev, k_cache.shape[2] if k_cache.dim() == 4 else 1, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens)
    shape = (int(tokens), dims.nkvheads, dims.headdim)
    _offsets(cu_seqlens, "cu_seqlens", dev, dims.nseq + 1)
    out = []
    for n, t in (("k", k), ("v", v)):
        out.append(torch.empty(shape, dtype=dtype, device=dev) if t is None else t)
        _dense(out[-1], n, shape, dtype, dev)
    _on_stream(stream, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, *out)
    _call("ssd_kv8_read", dev, stream, ctypes.byref(dims), ctypes.byref(pages), shape[0], _addr(cu_seqlens), _addr(seq_lens),
          _addr(block_table), _addr(out[0]), _addr(out[1]))
    return tuple(out)
