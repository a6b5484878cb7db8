"""fp64 model of the attention layer (include/ssd_attn.h): softmax attention over one packed batch, its
gradients, and the append to a paged cache.  Test infrastructure: plain loops over sequences and heads.

Beside each result stand the sums of magnitudes that bound what rounding can do to it (``*_abs``).
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


def bucket(rel: int, num_buckets: int, max_distance: int, bidirectional: bool) -> int:
    """Bucket of key position minus query position, in exact fractions."""
    n = num_buckets // 2 if bidirectional else num_buckets
    d = abs(rel) if bidirectional else max(-rel, 0)
    e = n // 2
    b = d
    if d >= e:
        f = n - e
        b = e + max(k for k in range(f) if Fraction(max_distance, e) ** k <= Fraction(d, e) ** f)
    return b + (n if bidirectional and rel > 0 else 0)


def bias_of(rel, h, slopes, table, max_distance, bidirectional):
    """Bias [*rel.shape] of head h, and the bucket of every cell (None without a table)."""
    if slopes is not None:
        return -slopes[h] * np.abs(rel), None
    if table is None:
        return np.zeros(rel.shape), None
    lo, hi = int(rel.min()), int(rel.max())
    lut = np.array([bucket(r, table.shape[0], max_distance, bidirectional) for r in range(lo, hi + 1)])
    cells = lut[rel - lo]
    return table[cells, h], cells


def _spans(offsets, total, nseq):
    if offsets is None:
        each = total // nseq if nseq else 0
        return [(s * each, each) for s in range(nseq)]
    return [(int(a), int(b) - int(a)) for a, b in zip(offsets[:-1], offsets[1:])]


def attention(q, k, v, nseq=None, cu=None, cu_k=None, causal=True, scale=None, cap=0.0, slopes=None, table=None,
              max_distance=128, bidirectional=False, prefix=None, dy=None, y_err=None):
    """q [Tq,H,D], k, v [Tk,Hk,D] in fp64.  With dy also the gradients; y_err [Tq,H,D] is how far the y
    that the backward pass is given may be off (it enters the bounds only)."""
    Tq, H, D = q.shape
    Hk = k.shape[1]
    nseq = len(cu) - 1 if cu is not None else nseq
    scale = D ** -0.5 if scale is None else scale
    out = dict(y=np.zeros_like(q), lse=np.full((Tq, H), -np.inf), y_abs=np.zeros_like(q), s_abs=np.zeros((Tq, H)),
               seen=np.zeros(Tq, dtype=bool))
    if dy is not None:
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            out[n], out[n + "_abs"], out[n + "_y"] = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
        if table is not None:
            out["dtable"], out["dtable_abs"] = np.zeros_like(table), np.zeros_like(table)
    for s, ((q0, lq), (k0, lk)) in enumerate(zip(_spans(cu, Tq, nseq), _spans(cu if cu_k is None else cu_k, len(k), nseq))):
        out["seen"][q0:q0 + lq] = True
        if lq == 0 or lk == 0:
            continue
        pq, pk = np.arange(lq)[:, None] + lk - lq, np.arange(lk)[None, :]
        see = np.ones((lq, lk), dtype=bool)
        if causal:
            see = (pk <= pq) | (pk < (prefix[s] if prefix is not None else 0))
        for h in range(H):
            g = h // (H // Hk)
            qs, ks, vs = q[q0:q0 + lq, h], k[k0:k0 + lk, g], v[k0:k0 + lk, g]
            z = scale * (qs @ ks.T)
            c1 = np.ones_like(z)
            if cap:
                t = np.tanh(z / cap)
                z, c1 = cap * t, 1 - t * t
            b, cells = bias_of(pk - pq, h, slopes, table, max_distance, bidirectional)
            z = np.where(see, z + b, -np.inf)
            top = np.where(see.any(1), z.max(1, initial=-np.inf), 0.0)
            e = np.where(see, np.exp(z - top[:, None]), 0.0)
            tot = e.sum(1)
            p = e / np.where(tot > 0, tot, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                out["lse"][q0:q0 + lq, h] = np.where(tot > 0, top + np.log(tot), -np.inf)
            out["y"][q0:q0 + lq, h] = p @ vs
            out["y_abs"][q0:q0 + lq, h] = p @ np.abs(vs)
            out["s_abs"][q0:q0 + lq, h] = np.where(see, abs(scale) * (np.abs(qs) @ np.abs(ks).T) + np.abs(b), 0).max(1)
            if dy is None:
                continue
            gs = dy[q0:q0 + lq, h]
            dp = gs @ vs.T
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            off = np.zeros(lq) if y_err is None else (np.abs(gs) * y_err[q0:q0 + lq, h]).sum(1)
            dsy = p * off[:, None]                   # what an inexact y can add to dS
            dsa = p * (np.abs(gs) @ np.abs(vs).T + (p * np.abs(dp)).sum(1, keepdims=True))
            out["dv"][k0:k0 + lk, g] += p.T @ gs
            out["dv_abs"][k0:k0 + lk, g] += p.T @ np.abs(gs)
            if cells is not None:
                for n, x in (("dtable", ds), ("dtable_abs", dsa)):
                    out[n][:, h] += np.bincount(cells.ravel(), x.ravel(), table.shape[0])
            w = c1 * abs(scale)
            for n, a, x, rows, hd in (("dq", lambda m: m, ks, slice(q0, q0 + lq), h), ("dk", np.transpose, qs, slice(k0, k0 + lk), g)):
                out[n][rows, hd] += a(ds * c1 * scale) @ x
                out[n + "_abs"][rows, hd] += a(np.abs(ds) * w) @ np.abs(x)
                out[n + "_y"][rows, hd] += a(dsy * w) @ np.abs(x)
                out.setdefault(n + "_all", np.zeros_like(out[n]))[rows, hd] += a(dsa * w) @ np.abs(x)
                out.setdefault(n + "_uncapped", np.zeros_like(out[n]))[rows, hd] += a(np.abs(ds) * abs(scale)) @ np.abs(x)
    return out


def append(k, v, k_cache, v_cache, block_table, seq_lens, cu=None, inv_freq=None, interleaved=False, q=None):
    """Copies of the caches with the tokens appended, and q rotated.  Bad pages and places are passed over."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    q = None if q is None else q.copy()
    pages, size = k_cache.shape[:2]
    n = len(seq_lens)
    for s in range(n):
        a, b = (s, s + 1) if cu is None else (int(cu[s]), int(cu[s + 1]))
        for i in range(a, b):
            pos = int(seq_lens[s]) - (b - i)

            def turned(x):
                x = x.copy()
                if inv_freq is None:
                    return x
                r = len(inv_freq)
                ang = [math.remainder(float(pos) * float(w), 2 * math.pi) for w in inv_freq]
                c, si = np.cos(ang), np.sin(ang)
                lo, hi = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
                u, w = x[:, lo].copy(), x[:, hi].copy()
                x[:, lo], x[:, hi] = u * c - w * si, w * c + u * si
                return x

            if q is not None:
                q[i] = turned(q[i])
            if pos < 0 or pos >= block_table.shape[1] * size:
                continue
            page = int(block_table[s, pos // size])
            if 0 <= page < pages:
                k_cache[page, pos % size], v_cache[page, pos % size] = turned(k[i]), v[i]
    return k_cache, v_cache, q
