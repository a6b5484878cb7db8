"""GPU tests of attention over packed documents against the fp64 model (oracle/attention.py)."""
import numpy as np
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from attn_helpers import U, f64, grad_bounds, lse_bound, make, offsets, reference, some_heads, within, y_bound

pytestmark = pytest.mark.gpu

# documents of no token, one token, odd sizes around the 32-, 64- and 128-row tiles
LENS = [1, 130, 0, 64, 257, 31, 128, 1, 33]
MODES = [dict(causal=True), dict(causal=False, bidirectional=True), dict(causal=True, cap=5.0),
         dict(causal=True, bias="slopes"), dict(causal=False, bias="slopes", cap=30.0),
         dict(causal=True, bias="buckets"), dict(causal=False, bias="buckets", bidirectional=True),
         dict(causal=True, prefix=True, scale=-0.3), dict(causal=True, prefix=True, bias="buckets", bidirectional=True, cap=2.0)]


# few heads: too little work for the chip, the waves of a workgroup share rows; many: each has its own
HEADS = {"few": {32: (6, 2), 64: (4, 4), 128: (3, 1)}, "many": {32: (80, 40), 64: (40, 40), 128: (44, 44)}}


def _case(mode):
    mode = dict(mode)
    bias, cap, pre = mode.pop("bias", "none"), mode.pop("cap", 0.0), mode.pop("prefix", False)
    return mode, bias, cap, pre


def _prefix(lens, pre):
    return torch.tensor([(7 * i + 3) % (n + 2) if n else 5 for i, n in enumerate(lens)], dtype=torch.int64) if pre else None


def _forward(d, cu, cu_k=None, prefix=None, cap=0.0, **how):
    g = {n: (t.cuda() if t is not None else None) for n, t in d.items()}
    move = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, lse = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], move(cu), move(cu_k), softcap=cap, slopes=g["slopes"],
                                  table=g["table"], prefix=move(prefix), lse=True, **how)
    torch.cuda.synchronize()
    return f64(y), f64(lse)


def _check_forward(label, d, dtype, cap, y, lse, **how):
    d, got = some_heads(d, dict(y=y, lse=lse))
    ref = reference(d, cap=cap, **how)
    D, n = d["q"].shape[-1], len(d["k"])
    within(got["y"], ref["y"], y_bound(ref, dtype, D, n, cap), label + " y")
    within(got["lse"], ref["lse"], lse_bound(ref, D, n, cap), label + " lse")
    return ref


@pytest.mark.parametrize("heads", ["few", "many"])
@pytest.mark.parametrize("mode", MODES, ids=lambda m: "-".join("%s=%s" % x for x in m.items()))
@pytest.mark.parametrize("dtype,D", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("fp32", 32), ("fp32", 64), ("fp32", 128)])
def test_forward_packed(dtype, D, mode, heads):
    how, bias, cap, pre = _case(mode)
    H, Hk = HEADS[heads][D]
    d = make(D, sum(LENS), sum(LENS), H, Hk, D, dtype, bias=bias)
    cu, prefix = offsets(LENS), _prefix(LENS, pre)
    y, lse = _forward(d, cu, prefix=prefix, cap=cap, **how)
    _check_forward("%s D%d %s" % (dtype, D, mode), d, dtype, cap, y, lse, cu=cu.numpy(),
                   prefix=None if prefix is None else prefix.numpy(), **how)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hk", [(4, 2), (60, 60)])
def test_forward_keys_of_their_own(H, Hk, dtype, causal):
    """Queries as the last positions of longer, shorter and empty key ranges: rows that see nothing."""
    lq, lk = [5, 70, 40, 9, 0, 130, 3], [200, 70, 10, 0, 33, 1, 64]
    d = make(3, sum(lq), sum(lk), H, Hk, 64, dtype, bias="buckets")
    cu, cu_k = offsets(lq), offsets(lk)
    how = dict(causal=causal, bidirectional=not causal)
    y, lse = _forward(d, cu, cu_k, **how)
    ref = _check_forward("own keys %s causal=%s" % (dtype, causal), d, dtype, 0.0, y, lse, cu=cu.numpy(), cu_k=cu_k.numpy(), **how)
    assert np.isneginf(ref["lse"]).any()


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("fp32", 32)])
@pytest.mark.parametrize("lq,lk", [(1, 1), (1, 500), (65, 65), (300, 300), (129, 1000)])
def test_forward_batched_and_strided(dtype, D, lq, lk):
    """Batched layout, q and k, v as views of wider rows; the dense call gives the same bits."""
    B, H, Hk = 3, 4, 2
    d = make(lq + lk, B * lq, B * lk, H, Hk, D, dtype, bias="slopes")
    wide = torch.zeros((B * lk, (H + 2 * Hk) * D), dtype=d["q"].dtype).cuda()
    wide[:, H * D:(H + Hk) * D] = d["k"].flatten(1).cuda()
    wide[:, (H + Hk) * D:] = d["v"].flatten(1).cuda()
    k = wide[:, H * D:(H + Hk) * D].view(B, lk, Hk, D)
    v = wide[:, (H + Hk) * D:].view(B, lk, Hk, D)
    q = d["q"].cuda().view(B, lq, H, D)
    y, lse = ssd.ssd_attn_forward(q, k, v, slopes=d["slopes"].cuda(), lse=True)
    y2, lse2 = ssd.ssd_attn_forward(q, k.contiguous(), v.contiguous(), slopes=d["slopes"].cuda(), lse=True)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(lse, lse2)
    _check_forward("batched %s %d %d" % (dtype, lq, lk), d, dtype, 0.0, f64(y).reshape(-1, H, D), f64(lse).reshape(-1, H), nseq=B)


def test_forward_large_scores():
    """Scores far beyond what exp takes, of both signs, and a maximum that grows along the keys."""
    d = make(11, 300, 300, 2, 1, 64, "fp32", spread=12.0)
    d["k"] *= torch.linspace(0.01, 3.0, 300)[:, None, None]
    cu = offsets([300])
    y, lse = _forward(d, cu)
    ref = _check_forward("large scores", d, "fp32", 0.0, y, lse, cu=cu.numpy())
    assert np.abs(ref["lse"]).max() > 200


def test_rows_of_no_sequence_stay_as_they_were():
    """Tokens behind the last sequence, NaN themselves, are neither written nor read into anything."""
    lens, extra = [70, 33], 45
    d = make(5, sum(lens) + extra, sum(lens) + extra, 2, 2, 64, "bf16")
    for n in "qkv":
        d[n][sum(lens):] = float("nan")
    g = {n: d[n].cuda() for n in "qkv"}
    y = torch.full_like(g["q"], 7.0)
    lse = torch.full(g["q"].shape[:2], 7.0, device="cuda")
    ssd.ssd_attn_forward(g["q"], g["k"], g["v"], offsets(lens).cuda(), causal=False, y=y, lse=lse)
    torch.cuda.synchronize()
    assert torch.all(y[sum(lens):] == 7.0) and torch.all(lse[sum(lens):] == 7.0)
    cut = {n: (t[:sum(lens)] if n in "qkv" else t) for n, t in d.items()}
    _check_forward("tail", cut, "bf16", 0.0, f64(y)[:sum(lens)], f64(lse)[:sum(lens)], cu=offsets(lens).numpy(), causal=False)


def test_documents_do_not_reach_each_other():
    """A document of NaN and infinities leaves its neighbours' outputs as they are without it."""
    lens = [50, 77, 40]
    d = make(6, sum(lens), sum(lens), 2, 1, 64, "bf16")
    cu = offsets(lens)
    clean, _ = _forward(d, cu)
    d["v"][50:127], d["k"][50:127] = float("inf"), float("nan")
    y, lse = _forward(d, cu)
    assert np.isnan(y[50:127]).all() and np.isnan(lse[50:127]).all()
    for s in (slice(0, 50), slice(127, 167)):
        assert np.array_equal(y[s], clean[s])


@pytest.mark.parametrize("heads", ["few", "many"])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp32", 32), ("fp32", 128)])
@pytest.mark.parametrize("prefix", [False, True])
def test_what_a_row_does_not_see_does_not_reach_it(dtype, D, heads, prefix):
    """NaN and infinities in later keys and values of the same document (a padded batch's tail) leave the rows
    that do not see them as they were; the rows that do are not finite."""
    H, Hk = HEADS[heads][D]
    lens, bad = [300, 90], {0: [200, 250], 1: [64]}
    d = make(90 + D, sum(lens), sum(lens), H, Hk, D, dtype)
    cu = offsets(lens)
    pre = torch.tensor([100, 70], dtype=torch.int64) if prefix else None
    clean, lse0 = _forward(d, cu, prefix=pre)
    d["v"][200], d["v"][250, 0, 3] = float("nan"), float("inf")
    d["v"][300 + 64], d["k"][300 + 64] = float("-inf"), float("nan")
    y, lse = _forward(d, cu, prefix=pre)
    first = {0: 200, 1: 0 if prefix else 64}             # (key 64 of the second is in its prefix of 70)
    for s, at in ((0, 0), (1, 300)):
        rows = slice(at, at + first[s])
        assert np.array_equal(y[rows], clean[rows]) and np.array_equal(lse[rows], lse0[rows])
        seen = y[at + first[s]:at + lens[s]]
        assert not np.isfinite(seen.reshape(len(seen), -1)).all(1).any()


def test_many_short_documents():
    """More documents than one search step takes, most of them a few tokens long."""
    lens = [(5 * i) % 7 for i in range(4500)] + [200]
    d = make(8, sum(lens), sum(lens), 1, 1, 32, "bf16")
    cu = offsets(lens)
    y, lse = _forward(d, cu)
    _check_forward("many documents", d, "bf16", 0.0, y, lse, cu=cu.numpy())


def test_no_tokens():
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    y, lse = ssd.ssd_attn_forward(z(0, 2, 64), z(0, 2, 64), z(0, 2, 64), offsets([0, 0]).cuda(), lse=True)
    assert y.shape == (0, 2, 64) and lse.shape == (0, 2)
    y, lse = ssd.ssd_attn_forward(z(2, 3, 2, 64) + 1, z(2, 0, 2, 64), z(2, 0, 2, 64), lse=True)
    torch.cuda.synchronize()
    assert torch.all(y == 0) and torch.all(torch.isneginf(lse))


def _backward(d, cu, cu_k=None, prefix=None, cap=0.0, **how):
    g = {n: (t.cuda() if t is not None else None) for n, t in d.items()}
    move = lambda t: None if t is None else t.cuda()  # noqa: E731
    how = dict(how, softcap=cap, slopes=g["slopes"], table=g["table"], prefix=move(prefix))
    y, lse = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], move(cu), move(cu_k), lse=True, **how)
    got = ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y, lse, g["dy"], move(cu), move(cu_k), **how)
    torch.cuda.synchronize()
    return {n: f64(t) for n, t in got.items()}


def _check_backward(label, d, dtype, cap, got, cu, cu_k=None, prefix=None, **how):
    d, got = some_heads(d, got)
    H, D = d["q"].shape[1:]
    n = max(len(d["q"]), len(d["k"]))
    how = dict(how, cap=cap, cu=cu.numpy(), cu_k=None if cu_k is None else cu_k.numpy(),
               prefix=None if prefix is None else prefix.numpy())
    first = reference(d, **how)
    ref = reference(d, dy=d["dy"], y_err=y_bound(first, dtype, D, n, cap), **how)
    bounds = grad_bounds(ref, dtype, D, n, H, d["k"].shape[1], cap)
    assert set(got) == set(bounds)
    for x in sorted(bounds):
        within(got[x], ref[x], bounds[x], "%s %s" % (label, x))


@pytest.mark.parametrize("heads", ["few", "many"])
@pytest.mark.parametrize("mode", MODES, ids=lambda m: "-".join("%s=%s" % x for x in m.items()))
@pytest.mark.parametrize("dtype,D", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("fp32", 32), ("fp32", 64), ("fp32", 128)])
def test_backward_packed(dtype, D, mode, heads):
    how, bias, cap, pre = _case(mode)
    H, Hk = HEADS[heads][D]
    d = make(100 + D, sum(LENS), sum(LENS), H, Hk, D, dtype, bias=bias, grads=True)
    cu, prefix = offsets(LENS), _prefix(LENS, pre)
    got = _backward(d, cu, prefix=prefix, cap=cap, **how)
    _check_backward("%s D%d %s" % (dtype, D, mode), d, dtype, cap, got, cu, prefix=prefix, **how)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hk", [(4, 2), (60, 60)])
def test_backward_keys_of_their_own(H, Hk, dtype, causal):
    lq, lk = [5, 70, 40, 9, 0, 130, 3], [200, 70, 10, 0, 33, 1, 64]
    d = make(30, sum(lq), sum(lk), H, Hk, 64, dtype, bias="buckets", grads=True)
    cu, cu_k = offsets(lq), offsets(lk)
    how = dict(causal=causal, bidirectional=not causal)
    got = _backward(d, cu, cu_k, **how)
    _check_backward("own keys %s causal=%s" % (dtype, causal), d, dtype, 0.0, got, cu, cu_k, **how)


@pytest.mark.parametrize("buckets,reach,both", [(2, 2, False), (4, 3, True), (7, 20, False), (64, 1024, False),
                                                (128, 1000, True), (32, 17, False)])
@pytest.mark.parametrize("H,Hk", [(2, 1), (80, 80)])
def test_table_shapes(H, Hk, buckets, reach, both):
    """Few and many buckets, reaches shorter and longer than a document."""
    lens = [600, 45]
    d = make(buckets, sum(lens), sum(lens), H, Hk, 32, "fp32", bias="buckets", buckets=buckets, grads=True)
    cu = offsets(lens)
    how = dict(causal=False, bidirectional=both, max_distance=reach)
    got = _backward(d, cu, **how)
    _check_backward("table %d %d %s" % (buckets, reach, both), d, "fp32", 0.0, got, cu, **how)


def test_backward_same_bits_and_batched():
    """Equal calls give equal bits; the batched layout is the packed one with equal documents."""
    B, T, H, Hk, D = 2, 200, 4, 2, 64
    d = make(40, B * T, B * T, H, Hk, D, "bf16", bias="buckets", grads=True)
    cu = offsets([T] * B)
    a, b = _backward(d, cu), _backward(d, cu)
    g = {n: d[n].cuda().view(B, T, *d[n].shape[1:]) for n in ("q", "k", "v", "dy")}
    table = d["table"].cuda()
    y, lse = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], table=table, lse=True)
    c = ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y, lse, g["dy"], table=table)
    torch.cuda.synchronize()
    for n in a:
        assert np.array_equal(a[n], b[n]), n
        assert np.array_equal(a[n], f64(c[n]).reshape(a[n].shape)), n


def test_gradients_against_differences():
    """The fp32 gradients against central differences of the fp64 model's loss."""
    d = make(50, 90, 90, 2, 1, 32, "fp32", bias="buckets", grads=True)
    cu = offsets([90])
    got = _backward(d, cu, cap=3.0)
    rng = np.random.RandomState(0)
    for n in ("q", "k", "v", "table"):
        way = torch.from_numpy(rng.randn(*d[n].shape))
        loss = lambda e: (reference(dict(d, **{n: d[n].double() + e * way}), cu=cu.numpy(), cap=3.0)["y"] * f64(d["dy"])).sum()  # noqa: E731
        want = (loss(1e-4) - loss(-1e-4)) / 2e-4
        have = float((got["d" + n] * way.numpy()).sum())
        size = float(np.linalg.norm(got["d" + n]) * np.linalg.norm(way))
        # differences: h^2 and 1e-16 / h of the loss; gradients: fp32 sums of some hundred terms
        assert abs(have - want) <= 1e-5 * size, (n, have, want)


def test_gradients_of_no_sequence_stay_as_they_were():
    lens, extra = [70, 33], 45
    total = sum(lens) + extra
    d = make(60, total, total, 2, 1, 64, "bf16", grads=True)
    for n in ("q", "k", "v", "dy"):
        d[n][sum(lens):] = float("nan")
    got = _backward(d, offsets(lens))
    cut = {n: (t[:sum(lens)] if t is not None else None) for n, t in d.items()}
    want = _backward(cut, offsets(lens))
    for n in want:
        assert np.array_equal(got[n][:sum(lens)], want[n]), n


@pytest.mark.parametrize("heads", ["few", "many"])
@pytest.mark.parametrize("cap", [0.0, 50.0, 500.0])
def test_a_row_of_one_key_is_that_value(cap, heads):
    """Whatever its score, a lone key's weight is one: y is its value to the bit, and dq and dk nothing (dS is
    dy.v - dy.y, where a y off by its rounding would be far larger than the rest of a long document's dq):
    fp32 sums of D products in two orders, times the key and the scale."""
    H, Hk = HEADS[heads][64]
    lens = [1] * 40
    d = make(77, 40, 40, H, Hk, 64, "bf16", grads=True)
    d["q"] *= 3
    y, lse = _forward(d, offsets(lens), cap=cap)
    v = f64(d["v"]).repeat(H // Hk, 1)
    assert np.array_equal(y, v)
    got = _backward(d, offsets(lens), cap=cap)
    worst = 2 * 64 * 2.0 ** -24 * (np.abs(f64(d["dy"])) * np.abs(v)).sum(-1).max() * 0.125 * 1.05
    assert np.abs(got["dq"]).max() <= worst * np.abs(f64(d["k"])).max()
    assert np.abs(got["dk"]).max() <= worst * (H // Hk) * np.abs(f64(d["q"])).max()
    assert np.array_equal(got["dv"], f64(d["dy"])) or H != Hk


@pytest.mark.parametrize("heads", ["few", "many"])
@pytest.mark.parametrize("cap", [0.0, 2.0])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_short_documents_without_the_rounding_of_y(D, cap, heads):
    """dq of rows that see one tile of keys, in bf16: dS and dq are rounded to bf16 once each, and what the
    rounding of y leaves in dy.y is not in dS.  With A_ij = sum_d |dy_id v_jd| the fp32 part of dS is off by its
    weight's error (twice the score's e_s, and the sums') times A_ij + sum_j p_ij A_ij, at dP, at D and at the sum
    of dS, and the cap's derivative by some steps."""
    H, Hk = HEADS[heads][D]
    lens = [1, 2, 3, 5, 17, 31, 32] * (4 if heads == "many" else 1) + ([33, 63, 64] * 60 if heads == "many" else [])
    n = sum(lens)
    d = make(55 + D, n, n, H, Hk, D, "bf16", grads=True)
    cu = offsets(lens)
    got = _backward(d, cu, cap=cap)["dq"]
    h = [0, H // 2, H - 1]
    q, dy = f64(d["q"])[:, h], f64(d["dy"])[:, h]
    k, v = (f64(d[x])[:, [i // (H // Hk) for i in h]] for x in ("k", "v"))
    u, scale, at = 2.0 ** -24, D ** -0.5, 0
    for n in lens:
        Q, K, V, G = (x[at:at + n].transpose(1, 0, 2) for x in (q, k, v, dy))
        z = scale * Q @ K.transpose(0, 2, 1)
        s = cap * np.tanh(z / cap) if cap else z
        w = np.where(np.tril(np.ones((n, n), bool)), np.exp(s - s.max(-1, keepdims=True)), 0.0)
        pr = w / w.sum(-1, keepdims=True)
        dp, A = G @ V.transpose(0, 2, 1), np.abs(G) @ np.abs(V).transpose(0, 2, 1)
        ds = pr * (dp - (pr * dp).sum(-1, keepdims=True))
        slope = 1 - (s / cap) ** 2 if cap else np.ones_like(s)
        es = ((D + 16) * scale * np.abs(Q) @ np.abs(K).transpose(0, 2, 1) + 4 * max(cap, 1.0)).max(-1, keepdims=True) * u
        fine = pr * (A + (pr * A).sum(-1, keepdims=True)) * 2 * (2 * es + (D + n + 32) * u)
        want = (ds * slope) @ K * scale
        bound = 1.1 * (((U["bf16"] * np.abs(ds * slope) + fine) @ np.abs(K)) * scale + U["bf16"] * np.abs(want))
        within(got[at:at + n][:, h], want.transpose(1, 0, 2), bound.transpose(1, 0, 2) + 1e-30, "D%d cap %g, %d tokens" % (D, cap, n))
        at += n
