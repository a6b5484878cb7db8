"""Python binding of the rotation by positions (``include/ssd_rotary.h``): argument marshalling, and the frequencies.

Tensors of a batched call are q [B,L,H,D], k [B,L,Hk,D]; of a packed call (``cu_seqlens`` given) q [T,H,D], k [T,Hk,D].  One
token's heads are dense; q and k may be views of wider rows, such as a fused projection's output.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _DTYPE_CODE, _in_stream, _on_stream
from .attention import _addr, _call, _dense, _offsets, _stride


class RotaryDims(ctypes.Structure):
    """Mirror of ``ssd_rotary_dims``."""
    _fields_ = [("nseq", ctypes.c_int64), ("total", ctypes.c_int64), ("nheads", ctypes.c_int64), ("nkvheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("magnitude", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("rot_pairs", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32)]


def declare(lib):
    lib.ssd_rotate.argtypes = [ctypes.POINTER(RotaryDims)] + [ctypes.c_void_p] * 8
    lib.ssd_rotate.restype = ctypes.c_int


@_in_stream
def ssd_rotate(q, inv_freq, cu_seqlens=None, start=None, k=None, interleaved: bool = False, magnitude: float = 1.0,
               inverse: bool = False, q_out=None, k_out=None, stream=None):
    """Run ``ssd_rotate``: the first 2 * len(inv_freq) elements of every head of q (and k) turned by their token's position
    times ``inv_freq`` fp32 [pairs], and multiplied by ``magnitude``; the rest is copied.

    ``cu_seqlens``: int64 offsets [nseq + 1] on the GPU of a packed batch.  ``start``: int64 [nseq], the positions of the
    sequences' first tokens (None: zero).  Pairs are (r, r + pairs), or ``interleaved`` (2 r, 2 r + 1).  ``inverse`` turns
    back: the gradient with respect to q (k) is the same call with ``inverse`` on the gradient of its output.  Tokens of
    no sequence are not written.  Returns (q_out, k_out), dense; k_out is None without k."""
    dev, dim = q.device, 4 if cu_seqlens is None else 3
    if q.dtype not in _DTYPE_CODE:
        raise TypeError("q must be float32 or bfloat16, got %s" % q.dtype)
    strides = [0 if t is None else _stride(t, n, dim, q.dtype, dev) for n, t in (("q", q), ("k", k))]
    if k is not None and (k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]):
        raise ValueError("q %s and k %s must have the same tokens and head dim" % (tuple(q.shape), tuple(k.shape)))
    if k is None and k_out is not None:
        raise ValueError("k_out needs k")
    if cu_seqlens is None:
        nseq, total = q.shape[0], q.shape[0] * q.shape[1]
    else:
        _offsets(cu_seqlens, "cu_seqlens", dev)
        nseq, total = cu_seqlens.numel() - 1, q.shape[0]
    _offsets(start, "start", dev, nseq)
    _dense(inv_freq, "inv_freq", (inv_freq.numel(),), torch.float32, dev)
    out = []
    for n, t, given in (("q_out", q, q_out), ("k_out", k, k_out)):
        out.append(torch.empty(t.shape, dtype=q.dtype, device=dev) if given is None and t is not None else given)
        if t is not None:
            _dense(out[-1], n, t.shape, q.dtype, dev)
    dims = RotaryDims(nseq, total, q.shape[-2], 0 if k is None else k.shape[-2], q.shape[-1], *strides, float(magnitude),
                      _DTYPE_CODE[q.dtype], inv_freq.numel(), int(bool(interleaved)), int(bool(inverse)))
    _on_stream(stream, q, k, inv_freq, cu_seqlens, start, *out)
    _call("ssd_rotate", dev, stream, ctypes.byref(dims), _addr(cu_seqlens), _addr(start), _addr(q), _addr(k), _addr(inv_freq),
          _addr(out[0]), _addr(out[1]))
    return tuple(out)


def ssd_rotary_frequencies(dim: int, base: float = 10000.0, factor: float = 1.0, how: str = "parts", trained: int = 4096,
                           fast: float = 32.0, slow: float = 1.0):
    """Frequencies of ``dim`` rotated elements, base^(-2 r / dim) for pair r, for a context ``factor`` times the one
    trained on, and the magnitude that goes with them.  Returns (inv_freq fp32 [dim / 2] on the CPU, magnitude).

    how="linear": every frequency over ``factor`` (positions interpolated).  "base": a larger base, so that the
    slowest pair's frequency is over ``factor`` and the fastest's unchanged.  "parts": by how often a pair turns in
    ``trained`` positions: ``fast`` times and more unchanged, ``slow`` times and less over ``factor``, in between a
    mixture of the two that is straight in the pair's turns; the magnitude is then 0.1 ln(factor) + 1.  (Models trained with a
    mixture straight in the pair's index, or with borders rounded to whole pairs, have other angles: give `ssd_rotate` theirs.)"""
    if dim < 2 or dim % 2 != 0:
        raise ValueError("dim must be even and at least 2, got %d" % dim)
    if not (base > 1.0 and factor >= 1.0):
        raise ValueError("base must be above 1 and factor at least 1, got %g and %g" % (base, factor))
    if how not in ("linear", "base", "parts"):
        raise ValueError("how must be 'linear', 'base' or 'parts', got %r" % (how,))
    if how == "base" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    r = torch.arange(0, dim, 2, dtype=torch.float64)
    freq, magnitude = base ** (-r / dim), 1.0
    if how == "linear":
        freq = freq / factor
    if how == "parts" and factor > 1.0:
        if not fast > slow > 0.0:
            raise ValueError("fast must be above slow, and slow above 0, got %g and %g" % (fast, slow))
        keep = ((trained * freq / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        freq = freq * (keep + (1.0 - keep) / factor)
        magnitude = 0.1 * math.log(factor) + 1.0
    return freq.float(), magnitude
