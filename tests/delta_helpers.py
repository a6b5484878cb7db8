"""Inputs and error bounds of the gated delta rule's tests.

Roundings: a bf16 output is off by half a step, at most U = 2^-8 of it.  In bf16 calls y, dq and dk are sums of products
of which one operand may have been rounded to bf16 too, each product off by up to U: rounding errors being as good as
independent, a sum of such products is off by about U / 3 of its 2-norm, and five of these beside each other
(operands of both score products, both state products, and the output itself) by sqrt(5) U / 3 < U.  Bound, on the
2-norm of the difference over that of the result: 2 U.

All else is fp32, u = 2^-24: a chunk's e is three chained sums (N, 64, and N for what the state holds), the state one more
of 64, each off by about sqrt(n) u of its 2-norm, and states forget earlier errors as they forget values (|k| = 1, beta in
[0, 1]: no step lengthens an error).  Two passes of such chains (there and back) and a bound of six times the
expected: 12 u sqrt(2 N + 128 + P).  dlog_a is a difference: its error is relative to the sums it is made of, whose size
`oracle.delta` does not know; they are dy.y and dv.v of a chunk's tokens, from the reference's values.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle.delta as od

DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
FLOAT_OUTPUTS = ("final", "dlog_a", "dbeta", "dinit", "state")


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(seed, lens, H, G, N, P, dtype, state=True, decay=1.0):
    """Random inputs on the CPU: keys and queries of unit length, some writing strengths of exactly 0 and 1."""
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lens), len(lens)

    def normal(*shape):
        return torch.randn(shape, generator=g)

    d = {x: torch.nn.functional.normalize(normal(T, G, N), dim=-1).to(DTYPE[dtype]) for x in "qk"}
    d["v"] = normal(T, H, P).to(DTYPE[dtype])
    d["log_a"] = -decay * torch.nn.functional.softplus(2.0 * normal(T, H) - 3.0)
    d["beta"] = normal(T, H).mul(2.0).sigmoid()
    d["beta"][::7] = 0.0
    d["beta"][3::11] = 1.0
    d["dy"] = normal(T, H, P).to(DTYPE[dtype])
    d["init"] = normal(n, H, N, P) * 0.3 if state else None
    d["dfinal"] = normal(n, H, N, P) * 0.1 if state else None
    d["cu"] = torch.tensor([0] + list(lens), dtype=torch.int64).cumsum(0)
    return d


def cuda(d):
    return {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in d.items()}


def reference(d, scale=None, grads=True):
    scale = d["q"].shape[-1] ** -0.5 if scale is None else scale
    args = [f64(d[n]) for n in ("q", "k", "v", "log_a", "beta")] + [d["cu"].numpy(), scale]
    y, final = od.forward(*args, f64(d["init"]))
    want = dict(y=y, final=final)
    if grads:
        want.update(od.backward(*args, f64(d["dy"]), f64(d["init"]), f64(d["dfinal"])))
    return want


def bound(name, dtype, N, P):
    if dtype == "bf16" and name not in FLOAT_OUTPUTS:
        return 2 * U["bf16"]
    return 12 * U["fp32"] * np.sqrt(2 * N + 128 + P)


def sums_of_dlog_a(d, want):
    """The 2-norm of what dlog_a is a difference of."""
    a = (f64(d["dy"]) * want["y"]).sum(-1)
    b = (want["dv"] * f64(d["v"])).sum(-1)
    return np.sqrt(32.0 * (np.sum(a * a) + np.sum(b * b)))  # (a token's sum has 32 terms on average)


def check(got, want, d, dtype, label):
    N, P = d["q"].shape[-1], d["v"].shape[-1]
    worst = ""
    for n, w in want.items():
        if n not in got or got[n] is None:
            continue
        x = f64(got[n])
        assert x.shape == w.shape and np.all(np.isfinite(x)), (label, n)
        off, size = np.linalg.norm(x - w), np.linalg.norm(w)
        if n == "dlog_a":
            size = size + sums_of_dlog_a(d, want)
        lim = bound(n, dtype, N, P)
        worst += " %s %.2g/%.2g" % (n, off / size if size else off, lim)
        assert off <= lim * size + 1e-30, "%s %s: off by %.3g of the result, %.3g allowed" % (label, n, off / max(size, 1e-30), lim)
        # and no value by more than ten times its share
        if n != "dlog_a" and w.size:
            rms = size / np.sqrt(w.size)
            assert np.max(np.abs(x - w)) <= 10 * lim * max(rms, 1e-30) + lim * np.max(np.abs(w)), (label, n)
    print("[gpu case] %s:%s" % (label, worst), flush=True)
