"""Inputs and error bounds of the attention tests.

A rounding is off by at most U = half a step of its type, relative to the value.  bf16 kernels round the
weights p (and in the backward pass dS) to bf16 once for the matrix unit and the output once; the rest is
fp32.  With every term's magnitude in sum_j |p_ij v_j| =: A, an output is off by at most
    U (A + |y|) + fp32 part,
and the fp32 part is the score's error e_s times A on numerator and denominator, plus the sums' own:
    (2 e_s + (n + 16) u) A,   u = 2^-24,   e_s = (D + 16) u (sum_d |q_d k_d| scale + |bias|) + 4 u cap-or-1,
a sum of n products in any order being off by at most n u times the sum of their magnitudes.  Second-order
terms stay under a tenth of these, which the factor 1.1 covers.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle.attention as oa

U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(seed, tq, tk, H, Hk, D, dtype, spread=1.0, bias="none", buckets=32, grads=False):
    """Random inputs on the CPU, rounded to the dtype."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(DTYPE[dtype])

    d = dict(q=normal(tq, H, D, scale=spread), k=normal(tk, Hk, D, scale=spread), v=normal(tk, Hk, D))
    if grads:
        d["dy"] = normal(tq, H, D)
    d["slopes"] = torch.rand(H, generator=g) + 0.05 if bias == "slopes" else None
    d["table"] = torch.randn((buckets, H), generator=g) if bias == "buckets" else None
    return d


def score_error(ref, D, cap):
    return ((D + 16) * ref["s_abs"] + 4 * max(cap, 1.0)) * 2.0 ** -24


def y_bound(ref, dtype, D, n, cap):
    es = score_error(ref, D, cap)[..., None]
    soft = U[dtype] * (ref["y_abs"] + np.abs(ref["y"])) if dtype == "bf16" else U[dtype] * np.abs(ref["y"])
    return 1.1 * (soft + (2 * es + (n + 16) * 2.0 ** -24) * ref["y_abs"]) + 1e-30


def lse_bound(ref, D, n, cap):
    fine = np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0.0)
    return 1.1 * (score_error(ref, D, cap) + (n + 16) * 2.0 ** -24 + 4 * 2.0 ** -24 * fine) + 1e-30


def within(got, want, bound, label):
    """Elementwise |got - want| <= bound; infinities have to match."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    fine = np.isfinite(want)
    assert got.shape == want.shape, (label, got.shape, want.shape)
    assert np.array_equal(got[~fine], want[~fine]), label + ": infinities"
    err = np.abs(np.where(fine, got, 0) - np.where(fine, want, 0))
    bound = np.broadcast_to(bound, want.shape)
    assert np.all(np.isfinite(got[fine])), label + ": non-finite values"
    worst = float(np.max(err / bound)) if err.size else 0.0
    print("[gpu case] %s: largest error / bound %.3f" % (label, worst), flush=True)
    assert worst <= 1.0, "%s: error %.3g times its bound" % (label, worst)


def reference(d, cu=None, cu_k=None, nseq=None, dy=None, y_err=None, **how):
    return oa.attention(f64(d["q"]), f64(d["k"]), f64(d["v"]), nseq=nseq, cu=cu, cu_k=cu_k, slopes=f64(d["slopes"]),
                        table=f64(d["table"]), dy=f64(dy), y_err=y_err, **how)


def offsets(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int64).cumsum(0)


def grad_bounds(ref, dtype, D, n, H, Hk, cap):
    """Bounds of dq, dk, dv and dtable.  dv: p rounded to bf16 and one output rounding.  dq, dk: dS rounded,
    the output rounded, and what the inexact y adds to D (``*_y``, from y_err).  fp32 parts: p has the
    relative error 2 e_s of its score and lse, on every term of dS (``*_all`` takes both terms' magnitude),
    and a cap's 1 - t^2 loses 4 u of itself in each of the two roundings of t.  Sums: n terms per head."""
    es = float(score_error(ref, D, cap).max())
    u, group = 2.0 ** -24, H // Hk
    rel = 4 * es + (n * group + 2 * D + 32) * u
    soft = U[dtype] if dtype == "bf16" else 0.0
    got = {"dv": 1.1 * (soft * ref["dv_abs"] + U[dtype] * np.abs(ref["dv"]) + rel * ref["dv_abs"]) + 1e-30}
    for x in ("dq", "dk"):
        flat = rel * ref[x + "_all"]
        if cap:  # near the cap the derivative is small, and its error is not
            flat = flat + 16 * u * ref[x + "_uncapped"]
        got[x] = 1.1 * (soft * ref[x + "_abs"] + U[dtype] * np.abs(ref[x]) + ref[x + "_y"] + flat) + 1e-30
    if "dtable" in ref:  # (its D is exact: no part of y's error)
        got["dtable"] = 1.1 * rel * ref["dtable_abs"] + 1e-30
    return got


def some_heads(d, outputs, keep=3):
    """The case and its outputs cut to the first, a middle and the last key head and their queries' heads
    (heads are independent of each other, so each is checked as if it were alone)."""
    H, Hk = d["q"].shape[1], d["k"].shape[1]
    if Hk <= keep:
        return d, outputs
    kv = [0, Hk // 2, Hk - 1]
    qh = [g * (H // Hk) + i for g in kv for i in range(H // Hk)]
    axis = {"q": (1, qh), "k": (1, kv), "v": (1, kv), "dy": (1, qh), "slopes": (0, qh), "table": (1, qh), "y": (1, qh),
            "lse": (1, qh), "dq": (1, qh), "dk": (1, kv), "dv": (1, kv), "dtable": (1, qh)}

    def cut(n, x):
        if x is None:
            return None
        at, rows = axis[n]
        return x[:, rows] if at == 1 else x[rows]

    return {n: cut(n, x) for n, x in d.items()}, {n: cut(n, x) for n, x in outputs.items()}
