"""Python binding of the attention layer (``include/ssd_attn.h``): argument marshalling only.

Tensors of a batched call are q [B,Lq,H,D], k, v [B,Lk,Hk,D]; of a packed call (``cu_seqlens`` given)
q [Tq,H,D], k, v [Tk,Hk,D].  One token's heads are dense; q, k and v may be views of wider rows, such as
a fused projection's output.
"""
from __future__ import annotations

import ctypes

import torch

from . import SSD_OK, SSDError, _DTYPE_CODE, _check, _on_stream, load_library


class AttnDims(ctypes.Structure):
    """Mirror of ``ssd_attn_dims``."""
    _fields_ = [("nseq", ctypes.c_int64), ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("nkvheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("num_buckets", ctypes.c_int32),
                ("max_distance", ctypes.c_int32), ("bidirectional", ctypes.c_int32)]


class AttnCache(ctypes.Structure):
    """Mirror of ``ssd_attn_cache``."""
    _fields_ = [("nseq", ctypes.c_int64), ("nheads", ctypes.c_int64), ("nkvheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("num_buckets", ctypes.c_int32), ("max_distance", ctypes.c_int32),
                ("bidirectional", ctypes.c_int32)]


def declare(lib):
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    dp = ctypes.POINTER(AttnDims)
    lib.ssd_attn_forward.argtypes = [dp] + [vp] * 11
    lib.ssd_attn_forward.restype = i32
    lib.ssd_attn_backward_workspace_bytes.argtypes = [dp, i32]
    lib.ssd_attn_backward_workspace_bytes.restype = sz
    lib.ssd_attn_backward.argtypes = [dp] + [vp] * 16 + [sz, vp]
    lib.ssd_attn_backward.restype = i32
    cp = ctypes.POINTER(AttnCache)
    lib.ssd_attn_decode_workspace_bytes.argtypes = [cp]
    lib.ssd_attn_decode_workspace_bytes.restype = sz
    lib.ssd_attn_decode.argtypes = [cp] + [vp] * 9 + [sz, vp]
    lib.ssd_attn_decode.restype = i32
    lib.ssd_kv_append.argtypes = [cp, ctypes.c_int64] + [vp] * 7 + [i32, i32] + [vp] * 4
    lib.ssd_kv_append.restype = i32


# The calls below are short (a decode step's kernels take some microseconds), so the checks first ask whether
# everything is as it should be, in as few steps as that takes, and only then what is not.

def _addr(t):
    return None if t is None else t.data_ptr()


def _dense(t, name, shape, dtype, device):
    """As _check."""
    if t is not None and not (t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous()):
        _check(t, name, shape, dtype, device)


def _call(name, device, stream, *args):
    """The library's function on the caller's stream of the tensors' device, which is made the current one for it
    where it is another's."""
    index = device.index
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        if stream.device != device:
            raise ValueError("stream is of %s, the tensors are on %s" % (stream.device, device))
        handle = stream.cuda_stream
    function = getattr(load_library(), name)
    if torch._C._cuda_getDevice() == index:
        rc = function(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = function(*args, handle)
    if rc != SSD_OK:
        raise SSDError(rc, name)


def _token_stride(t, name, dim, dtype, device):
    """Elements from one token to the next of a tensor [..., tokens, heads, D] whose tokens are dense."""
    if dim == 3 and t.dim() == 3 and t.dtype is dtype and t.device == device and device.type == "cuda":
        tokens, heads, D = t.shape
        step, s1, s0 = t.stride()
        if s0 == 1 and s1 == D and step >= heads * D and tokens > 1:
            return step
    if t.dim() != dim:
        raise ValueError("%s must have %d dimensions, got shape %s" % (name, dim, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.numel() == 0:
        return 0
    if (t.shape[-1] > 1 and t.stride(-1) != 1) or (t.shape[-2] > 1 and t.stride(-2) != t.shape[-1]):
        raise ValueError("%s must have dense heads (strides %s)" % (name, t.stride()))
    dense = t.shape[-2] * t.shape[-1]
    step = t.stride(-3) if t.shape[-3] > 1 else dense
    if dim == 4 and t.shape[0] > 1:
        if t.shape[1] == 1:
            step = t.stride(0)
        elif t.stride(0) != t.shape[1] * step:
            raise ValueError("%s must have its sequences one after another (strides %s)" % (name, t.stride()))
    if step < dense:
        raise ValueError("%s has overlapping tokens (strides %s)" % (name, t.stride()))
    return step


def _offsets(t, name, device, n=None):
    if t is None or (n is not None and t.dtype is torch.int64 and t.shape == (n,) and t.device == device and t.is_contiguous()):
        return
    if t.dtype != torch.int64 or t.dim() != 1 or t.device != device or not t.is_contiguous() or (n is None and t.numel() < 1):
        raise ValueError("%s must be a contiguous 1-D int64 tensor on q's device" % name)
    if n is not None and t.numel() != n:
        raise ValueError("%s has %d values, expected %d" % (name, t.numel(), n))


def _empty(shape, dtype, device, stream):
    """Memory for a call on ``stream`` (None: the current one), taken from that stream's own pool: a block that was
    just freed on another stream may still be in use by what is queued there, which the call would not wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if stream.device != device:
        raise ValueError("stream is of %s, the tensors are on %s" % (stream.device, device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(t, need, device, stream=None):
    """The caller's workspace, or one of ``need`` bytes, and its size."""
    if t is None:
        return (None, 0) if need == 0 else (_empty(need, torch.uint8, device, stream), need)
    if t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    return t, t.numel() * t.element_size()


def _bias_args(slopes, table, H, device):
    if slopes is None and table is None:
        return 0
    if slopes is not None and table is not None:
        raise ValueError("slopes and table are two forms of the bias: give at most one")
    _dense(slopes, "slopes", (H,), torch.float32, device)
    if table is not None:
        if table.dim() != 2 or table.shape[0] < 2:
            raise ValueError("table must be [num_buckets, H], of two buckets or more")
        _dense(table, "table", (table.shape[0], H), torch.float32, device)
    return 0 if table is None else table.shape[0]


def _dims(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale, softcap, slopes, table, max_distance, bidirectional, prefix):
    """ssd_attn_dims of a call, its arguments checked."""
    dev, dim = q.device, 4 if cu_seqlens is None else 3
    if q.dtype not in _DTYPE_CODE:
        raise TypeError("q must be float32 or bfloat16, got %s" % q.dtype)
    strides = [_token_stride(t, n, dim, q.dtype, dev) for n, t in (("q", q), ("k", k), ("v", v))]
    H, D = q.shape[-2:]
    Hk = k.shape[-2]
    if tuple(v.shape) != tuple(k.shape) or k.shape[-1] != D or (dim == 4 and k.shape[0] != q.shape[0]):
        raise ValueError("k and v must be alike and fit q: q %s, k %s, v %s" % (tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    if cu_seqlens is None:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        nseq, tq, tk = q.shape[0], q.shape[0] * q.shape[1], k.shape[0] * k.shape[1]
    else:
        _offsets(cu_seqlens, "cu_seqlens", dev)
        nseq, tq, tk = cu_seqlens.numel() - 1, q.shape[0], k.shape[0]
        _offsets(cu_seqlens_k, "cu_seqlens_k", dev, nseq + 1)
        if cu_seqlens_k is None and tq != tk:
            raise ValueError("q and k have different token counts: give cu_seqlens_k")
    _offsets(prefix, "prefix", dev, nseq)
    if prefix is not None and not causal:
        raise ValueError("a prefix needs causal=True")
    buckets = _bias_args(slopes, table, H, dev)
    return AttnDims(nseq, tq, tk, H, Hk, D, *strides, D ** -0.5 if scale is None else float(scale), float(softcap),
                    _DTYPE_CODE[q.dtype], int(bool(causal)), buckets, int(max_distance), int(bool(bidirectional)))


def ssd_attn_forward(q, k, v, cu_seqlens=None, cu_seqlens_k=None, causal: bool = True, scale=None,
                     softcap: float = 0.0, slopes=None, table=None, max_distance: int = 128,
                     bidirectional: bool = False, prefix=None, y=None, lse=None, stream=None):
    """Run ``ssd_attn_forward``: softmax attention of every query over the visible keys of its own
    sequence, with scores capped to ``softcap`` * tanh and a bias by distance (``slopes`` [H] or a learned
    ``table`` [num_buckets, H]).

    ``cu_seqlens``: int64 offsets [nseq + 1] on the GPU of a packed batch (``cu_seqlens_k`` where the keys
    have offsets of their own; a sequence's queries are then its last positions).  ``scale`` defaults to
    D ** -0.5.  ``prefix``: int64 [nseq], keys before it are visible to their whole sequence.  ``y`` is
    allocated when not given; ``lse`` may be a tensor [..., H] fp32 to write, True to allocate one, or
    None/False to skip it.  Tokens of no sequence are not written.  Returns (y, lse)."""
    dims = _dims(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale, softcap, slopes, table, max_distance, bidirectional,
                 prefix)
    dev = q.device
    if y is None:
        y = _empty(q.shape, q.dtype, dev, stream)
    _dense(y, "y", q.shape, q.dtype, dev)
    if lse is True:
        lse = _empty(q.shape[:-1], torch.float32, dev, stream)
    elif lse is False:
        lse = None
    _dense(lse, "lse", q.shape[:-1], torch.float32, dev)
    _on_stream(stream, q, k, v, cu_seqlens, cu_seqlens_k, prefix, slopes, table, y, lse)
    _call("ssd_attn_forward", dev, stream, ctypes.byref(dims), _addr(cu_seqlens), _addr(cu_seqlens_k), _addr(prefix),
          _addr(q), _addr(k), _addr(v), _addr(slopes), _addr(table), _addr(y), _addr(lse))
    return y, lse


def ssd_attn_backward_workspace_bytes(dims: AttnDims, want_dtable: bool = False) -> int:
    return int(load_library().ssd_attn_backward_workspace_bytes(ctypes.byref(dims), int(bool(want_dtable))))


def ssd_attn_backward(q, k, v, y, lse, dy, cu_seqlens=None, cu_seqlens_k=None, causal: bool = True, scale=None,
                      softcap: float = 0.0, slopes=None, table=None, max_distance: int = 128,
                      bidirectional: bool = False, prefix=None, want_dtable=None, workspace=None, stream=None):
    """Run ``ssd_attn_backward``: the gradients of <dy, y> for ssd_attn_forward, whose arguments these are
    with its results ``y`` and ``lse``.  Returns a dict: dq, dk, dv (dtype of q, dense), and dtable
    [num_buckets, H] fp32 where a table is given (want_dtable=False skips it).  Rows of no sequence are
    not written."""
    dims = _dims(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale, softcap, slopes, table, max_distance, bidirectional,
                 prefix)
    dev = q.device
    _dense(y, "y", q.shape, q.dtype, dev)
    _dense(dy, "dy", q.shape, q.dtype, dev)
    _dense(lse, "lse", q.shape[:-1], torch.float32, dev)
    if want_dtable is None:
        want_dtable = table is not None
    if want_dtable and table is None:
        raise ValueError("dtable needs a table")
    out = {"d" + n: _empty(t.shape, q.dtype, dev, stream) for n, t in (("q", q), ("k", k), ("v", v))}
    if want_dtable:
        out["dtable"] = _empty(table.shape, torch.float32, dev, stream)
        if dims.nseq == 0:  # (no launch writes it)
            with torch.cuda.stream(stream):
                out["dtable"].zero_()
    need = ssd_attn_backward_workspace_bytes(dims, want_dtable)
    workspace, ws_bytes = _workspace(workspace, need, dev, stream)
    _on_stream(stream, q, k, v, cu_seqlens, cu_seqlens_k, prefix, slopes, table, y, lse, dy, workspace, *out.values())
    _call("ssd_attn_backward", dev, stream, ctypes.byref(dims), _addr(cu_seqlens), _addr(cu_seqlens_k), _addr(prefix),
          _addr(q), _addr(k), _addr(v), _addr(slopes), _addr(table), _addr(y), _addr(lse), _addr(dy), _addr(out["dq"]),
          _addr(out["dk"]), _addr(out["dv"]), _addr(out.get("dtable")), _addr(workspace), ws_bytes)
    return out


def _cache_dims(q, heads, k_cache, v_cache, block_table, seq_lens, strides, scale, softcap, buckets, max_distance,
                bidirectional):
    """ssd_attn_cache of a call, the cache's arguments checked; q: any tensor of its dtype and device."""
    dev = q.device
    if q.dtype not in _DTYPE_CODE:
        raise TypeError("the cache's tensors must be float32 or bfloat16, got %s" % q.dtype)
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, page_size, Hk, D], got shape %s" % (tuple(k_cache.shape),))
    _dense(k_cache, "k_cache", k_cache.shape, q.dtype, dev)
    _dense(v_cache, "v_cache", k_cache.shape, q.dtype, dev)
    pages, size, Hk, D = k_cache.shape
    nseq = seq_lens.numel()
    _offsets(seq_lens, "seq_lens", dev, nseq)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [nseq, max_pages]")
    _dense(block_table, "block_table", (nseq, block_table.shape[1]), torch.int32, dev)
    return AttnCache(nseq, heads, Hk, D, pages, size, block_table.shape[1], *strides,
                     D ** -0.5 if scale is None else float(scale), float(softcap), _DTYPE_CODE[q.dtype], buckets,
                     int(max_distance), int(bool(bidirectional)))


def ssd_attn_decode_workspace_bytes(dims: AttnCache) -> int:
    return int(load_library().ssd_attn_decode_workspace_bytes(ctypes.byref(dims)))


def ssd_attn_decode(q, k_cache, v_cache, block_table, seq_lens, scale=None, softcap: float = 0.0, slopes=None, table=None,
                    max_distance: int = 128, bidirectional: bool = False, y=None, workspace=None, stream=None):
    """Run ``ssd_attn_decode``: one query per sequence, q [nseq,H,D], over a paged cache.

    k_cache, v_cache [num_pages, page_size, Hk, D] (page_size a multiple of 16), block_table int32
    [nseq, max_pages], seq_lens int64 [nseq] with the present token, all on the GPU.  Bias and cap as in
    ssd_attn_forward.  Returns y [nseq,H,D]."""
    dev = q.device
    stride = _token_stride(q, "q", 3, q.dtype, dev)
    nseq, H, D = q.shape
    buckets = _bias_args(slopes, table, H, dev)
    dims = _cache_dims(q, H, k_cache, v_cache, block_table, seq_lens, (stride, 0, 0), scale, softcap, buckets,
                       max_distance, bidirectional)
    if dims.nseq != nseq or dims.headdim != D:
        raise ValueError("q %s does not fit %d sequences of head dim %d" % (tuple(q.shape), dims.nseq, dims.headdim))
    if y is None:
        y = _empty((nseq, H, D), q.dtype, dev, stream)
    _dense(y, "y", (nseq, H, D), q.dtype, dev)
    need = ssd_attn_decode_workspace_bytes(dims)
    workspace, ws_bytes = _workspace(workspace, need, dev, stream)
    _on_stream(stream, q, k_cache, v_cache, block_table, seq_lens, slopes, table, y, workspace)
    _call("ssd_attn_decode", dev, stream, ctypes.byref(dims), _addr(q), _addr(k_cache), _addr(v_cache), _addr(block_table),
          _addr(seq_lens), _addr(slopes), _addr(table), _addr(y), _addr(workspace), ws_bytes)
    return y


def ssd_kv_append(k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, inv_freq=None,
                  interleaved: bool = False, q=None, q_out=None, stream=None):
    """Run ``ssd_kv_append``: the keys and values of new tokens, k, v [tokens,Hk,D], into the cache's pages in
    place, the keys (and q [tokens,H,D], if given) rotated by their positions with ``inv_freq`` [pairs].

    ``cu_seqlens``: int64 offsets of each sequence's new tokens (None: one token per sequence);
    ``seq_lens`` counts the sequences with them.  Returns the rotated q, or None without q."""
    dev = k.device
    strides = [0 if t is None else _token_stride(t, n, 3, k.dtype, dev) for n, t in (("q", q), ("k", k), ("v", v))]
    tokens, Hk, D = k.shape
    H = Hk if q is None else q.shape[1]
    dims = _cache_dims(k, H, k_cache, v_cache, block_table, seq_lens, strides, None, 0.0, 0, 0, False)
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
            q_out = _empty(q.shape, q.dtype, dev, stream)
        _dense(q_out, "q_out", q.shape, q.dtype, dev)
    _on_stream(stream, k, v, q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, inv_freq, q_out)
    _call("ssd_kv_append", dev, stream, ctypes.byref(dims), tokens, _addr(cu_seqlens), _addr(seq_lens), _addr(block_table),
          _addr(k), _addr(v), _addr(q), _addr(inv_freq), 0 if inv_freq is None else inv_freq.numel(), int(bool(interleaved)),
          _addr(k_cache), _addr(v_cache), _addr(q_out))
    return q_out
