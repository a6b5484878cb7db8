"""The attention layer at its edges, on the GPU: calls that the documentation allows and an ordinary run does not make."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.attention as oa
import ssd_chunked_scan_02_amd as ssd
from attn_helpers import U, f64, grad_bounds, make, offsets, reference, within, y_bound
from ssd_chunked_scan_02_amd import attention

pytestmark = pytest.mark.gpu

# few heads: the waves of a workgroup share rows; many: each has its own, which takes 384 workgroups (two and more to
# each of 192 key heads of 130 tokens or more)
HEADS = {"few": (4, 2), "many": (384, 192)}


def test_outputs_of_a_call_on_a_stream_are_that_streams_memory():
    """What the binding allocates for a call on a given stream is not a block that was freed on the current one,
    where work that uses it may still be queued; the next call on that stream gets it again."""
    n, H, D = 16384, 8, 64
    q = torch.randn((n, H, D), device="cuda").bfloat16()
    cu = torch.tensor([0, n], dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    want, lse0 = ssd.ssd_attn_forward(q, q, q, cu, lse=True)
    grads0 = ssd.ssd_attn_backward(q, q, q, want, lse0, q, cu)
    torch.cuda.synchronize()
    freed = [torch.empty_like(q) for _ in range(6)]
    places = {t.data_ptr() for t in freed}
    del freed
    y, lse = ssd.ssd_attn_forward(q, q, q, cu, lse=True, stream=s)
    grads = ssd.ssd_attn_backward(q, q, q, y, lse, q, cu, stream=s)
    torch.cuda.synchronize()
    assert not places & {t.data_ptr() for t in (y, *grads.values())}
    assert torch.equal(y, want) and all(torch.equal(grads[x], grads0[x]) for x in grads0)
    place = y.data_ptr()
    del y
    y, _ = ssd.ssd_attn_forward(q, q, q, cu, stream=s)
    torch.cuda.synchronize()
    assert y.data_ptr() == place and torch.equal(y, want)


def test_inputs_of_a_call_on_a_stream_are_known_to_the_allocator(monkeypatch):
    """Every tensor that a call on a given stream reads or writes is recorded there, so that a caller who drops an
    input right after the call does not get its memory back while the kernels still read it."""
    seen = []
    monkeypatch.setattr(attention, "_on_stream", lambda s, *t: seen.extend((s, x.data_ptr()) for x in t if x is not None))
    n, H, Hk, D, s = 40, 4, 2, 64, torch.cuda.Stream()
    r = lambda *shape: torch.randn(shape, device="cuda")  # noqa: E731
    i64 = lambda *x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
    q, k, v, dy, slopes, table = r(n, H, D), r(n, Hk, D), r(n, Hk, D), r(n, H, D), r(H), r(16, H)
    cu, cu_k, prefix, cu_new = i64(0, 15, n), i64(0, 20, n), i64(3, 0), i64(0, 3, 5)
    kc, vc, inv, lens = r(4, 16, Hk, D), r(4, 16, Hk, D), r(16), i64(30, 9)
    pages = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def check(*tensors):
        torch.cuda.synchronize()
        assert {(s, t.data_ptr()) for t in tensors} <= set(seen)
        seen.clear()

    y, lse = ssd.ssd_attn_forward(q, k, v, cu, cu_k, slopes=slopes, prefix=prefix, lse=True, stream=s)
    check(q, k, v, cu, cu_k, slopes, prefix, y, lse)
    y, lse = ssd.ssd_attn_forward(q, k, v, cu, cu_k, table=table, prefix=prefix, lse=True, stream=s)
    check(q, k, v, cu, cu_k, table, prefix, y, lse)
    got = ssd.ssd_attn_backward(q, k, v, y, lse, dy, cu, cu_k, table=table, prefix=prefix, stream=s)
    check(q, k, v, y, lse, dy, cu, cu_k, table, prefix, *got.values())
    q_out = ssd.ssd_kv_append(k[:5], v[:5], kc, vc, pages, lens, cu_new, inv, q=q[:5], stream=s)
    check(k, v, q, kc, vc, pages, lens, cu_new, inv, q_out)
    y = ssd.ssd_attn_decode(q[:2], kc, vc, pages, lens, table=table, stream=s)
    check(q, kc, vc, pages, lens, table, y)


def test_append_more_tokens_than_a_launch_has_workgroups():
    """2^24 tokens and some: each in its place, and its first pair rotated by its own position."""
    n, page, D = (1 << 24) + 37, 16, 32
    pages = -(-n // page)
    k = torch.randn((n, 1, D), device="cuda").bfloat16()
    table = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    kc, vc = (torch.zeros((pages, page, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    seq, cu = (torch.tensor(x, dtype=torch.int64, device="cuda") for x in ([n], [0, n]))
    inv = torch.zeros(8, device="cuda")
    inv[0] = 1.0
    ssd.ssd_kv_append(k, k, kc, vc, table, seq, cu, inv)
    torch.cuda.synchronize()
    assert torch.equal(vc.flip(0).flatten(0, 1)[:n], k)
    got = kc.flip(0).flatten(0, 1)[:n, 0]
    keep = [i for i in range(D) if i not in (0, 8)]
    assert torch.equal(got[:, keep], k[:, 0, keep])
    angle = torch.arange(n, device="cuda").double()
    a, b = k[:, 0, 0].double(), k[:, 0, 8].double()
    for have, want in ((got[:, 0], a * angle.cos() - b * angle.sin()), (got[:, 8], b * angle.cos() + a * angle.sin())):
        # one rounding to bf16, and in fp32 the sine and cosine and two products: 12 u (|a| + |b|)
        assert torch.all((have.double() - want).abs() <= 1.05 * 2.0 ** -8 * want.abs() + 12 * 2.0 ** -24 * (a.abs() + b.abs()))


def _capped_bound(ref, dtype, D, n):
    """y_bound of attn_helpers with a score's error that does not grow with the cap.  bf16: tanh's series (arguments
    within 1/4) is off by 3.3e-7 = 5.6 u of its argument and some roundings, the other form by 1.3e-7 (exp2, reciprocal
    and the subtraction, half a step of 1 each and one more) of a tanh over 0.24, 9 u of the score: 16 u of |z|, which
    is at most the sum of its terms' magnitudes.  fp32: the math library's tanh, a few u."""
    es = ((D + 32) * ref["s_abs"] * 2.0 ** -24)[..., None]
    soft = U[dtype] * ((ref["y_abs"] if dtype == "bf16" else 0) + np.abs(ref["y"]))
    return 1.1 * (soft + (2 * es + (n + 16) * 2.0 ** -24) * ref["y_abs"]) + 1e-30


CAPS = [0.5, 30.0, 500.0, 1e4, 1e6, 1e9]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cap", CAPS)
def test_caps_of_any_size_in_a_decode_step(cap, dtype):
    """A cap far above the scores is no cap; the sequences are long enough for their weights to tell."""
    H, Hk, D, page, lens = 8, 2, 64, 16, [900, 17, 1]
    total, n = [-(-x // page) for x in lens], len(lens)
    d = make(21, n, sum(total) * page, H, Hk, D, dtype, spread=1.5)
    table = torch.full((n, max(total)), -1, dtype=torch.int32)
    rows, at = [], 0
    for i, (pages, length) in enumerate(zip(total, lens)):
        table[i, :pages] = torch.arange(at, at + pages)
        rows.append(torch.arange(at * page, at * page + length))
        at += pages
    kc, vc = (d[x].unflatten(0, (at, page)).contiguous().cuda() for x in "kv")
    y = ssd.ssd_attn_decode(d["q"].cuda(), kc, vc, table.cuda(), torch.tensor(lens, dtype=torch.int64).cuda(), softcap=cap)
    torch.cuda.synchronize()
    d["k"], d["v"] = d["k"][torch.cat(rows)], d["v"][torch.cat(rows)]
    ref = reference(d, cu=list(range(n + 1)), cu_k=offsets(lens).numpy(), cap=cap)
    within(f64(y), ref["y"], _capped_bound(ref, dtype, D, max(lens)), "decode cap %g %s" % (cap, dtype))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cap", CAPS)
def test_caps_of_any_size_in_a_prompt(cap, dtype, heads):
    H, Hk = HEADS[heads]
    d = make(22, 300, 300, H, Hk, 64, dtype, spread=1.5)
    cu = offsets([300])
    y, _ = ssd.ssd_attn_forward(*(d[x].cuda() for x in "qkv"), cu.cuda(), softcap=cap)
    torch.cuda.synchronize()
    keep = slice(0, 4)
    one = dict(d, q=d["q"][:, keep], k=d["k"][:, :4 * Hk // H], v=d["v"][:, :4 * Hk // H])
    ref = reference(one, cu=cu.numpy(), cap=cap)
    within(f64(y)[:, keep], ref["y"], _capped_bound(ref, dtype, 64, 300), "prompt cap %g %s" % (cap, dtype))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("cap", [5.0, 50.0])
def test_hidden_keys_do_not_choose_the_form_of_the_cap(cap, heads):
    """Keys that a row does not see, however large, leave its capped scores' bits as they were."""
    H, Hk = HEADS[heads]
    d = make(23, 300, 300, H, Hk, 64, "bf16")
    q, k, v, cu = (x.cuda() for x in (d["q"], d["k"], d["v"], offsets([300])))
    y, lse = ssd.ssd_attn_forward(q, k, v, cu, softcap=cap, lse=True)
    k[200:] *= 1000
    k[250] = float("inf")
    y2, lse2 = ssd.ssd_attn_forward(q, k, v, cu, softcap=cap, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(y[:200], y2[:200]) and torch.equal(lse[:200], lse2[:200])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
def test_a_row_does_not_depend_on_its_neighbours(dtype, D, heads):
    """Queries of the same tile whose maxima grow along the keys leave the other rows' bits as they were."""
    H, Hk = HEADS[heads]
    d = make(24, 300, 300, H, Hk, D, dtype)
    q, k, v, cu = (x.cuda() for x in (d["q"], d["k"], d["v"], offsets([300])))
    y, lse = ssd.ssd_attn_forward(q, k, v, cu, lse=True)
    loud = torch.arange(300, device="cuda") % 7 == 3
    q[loud] *= 40
    y2, lse2 = ssd.ssd_attn_forward(q, k, v, cu, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(y[~loud], y2[~loud]) and torch.equal(lse[~loud], lse2[~loud])
    assert not torch.equal(y[loud], y2[loud])


def _slope_error(d, cap, D):
    """What errors of the cap's derivative c1 = 1 - tanh^2(z / cap) leave in dq and dk of one causal document.
    z is off by (D + 32) u sum_d |q_d k_d| scale: c1, which falls with |z|, by its change over that, which is all of it
    where the cap is under z's error.  Formed from a t off by 6 u (the capped score 4 u, 1 / cap and the product one
    each), c1 is off by 12 u more: 16 u.  It multiplies dS with its own error (y's rounding and fp32's, all that dS is
    in a row of one key): within p (A + sum p A), A = |dy| . |v|."""
    q, k, v, dy = (f64(d[x]).transpose(1, 0, 2) for x in ("q", "k", "v", "dy"))
    group, n, u, scale = len(q) // len(k), q.shape[1], 2.0 ** -24, D ** -0.5
    dq, dk = np.zeros_like(q), np.zeros_like(k)
    for h in range(len(q)):
        K, V = k[h // group], v[h // group]
        z, off = scale * q[h] @ K.T, (D + 32) * u * scale * np.abs(q[h]) @ np.abs(K).T

        def c1(x):
            return 1 - np.tanh(np.maximum(x, 0) / cap) ** 2

        e = np.maximum(c1(np.abs(z) - off) - c1(np.abs(z)), c1(np.abs(z)) - c1(np.abs(z) + off)) + 16 * u
        p = np.where(np.tril(np.ones((n, n), bool)), np.exp(cap * np.tanh(z / cap)), 0.0)
        p /= p.sum(-1, keepdims=True)
        A = np.abs(dy[h]) @ np.abs(V).T
        w = e * p * (A + (p * A).sum(-1, keepdims=True)) * scale
        dq[h] = w @ np.abs(K)
        dk[h // group] += w.T @ np.abs(q[h])
    return dq.transpose(1, 0, 2), dk.transpose(1, 0, 2)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("cap", [1e-38, 1e-20, 1e-9, 1e-6, 1e-3, 1e6, 1e16, 3e38])
def test_gradients_under_caps_of_any_size(cap, dtype, D, heads):
    """Forward and backward, rows of zero scores among them (a padded batch's).  A score's error does not grow with the
    cap (_capped_bound); for the sum of its magnitudes (D + 32) u instead of grad_bounds' (D + 16) u.
    What the cap's derivative is off by is added (_slope_error)."""
    H, Hk = HEADS[heads]
    n = 130
    d = make(25, n, n, H, Hk, D, dtype, grads=True)
    d["q"][40:75] = 0
    d["k"][:20] = 0
    cu = offsets([n])
    g = {x: d[x].cuda() for x in ("q", "k", "v", "dy")}
    y, lse = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], cu.cuda(), softcap=cap, lse=True)
    got = ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y, lse, g["dy"], cu.cuda(), softcap=cap)
    torch.cuda.synchronize()
    hk, hq = slice(0, 2), slice(0, 2 * H // Hk)
    d = dict(d, q=d["q"][:, hq], dy=d["dy"][:, hq], k=d["k"][:, hk], v=d["v"][:, hk])
    label = "cap %g %s D%d " % (cap, dtype, D)
    first = reference(d, cu=cu.numpy(), cap=cap)
    bound = _capped_bound(first, dtype, D, n)
    within(f64(y)[:, hq], first["y"], bound, label + "y")
    ref = reference(d, cu=cu.numpy(), cap=cap, dy=d["dy"], y_err=bound)
    bounds = grad_bounds(dict(ref, s_abs=ref["s_abs"] * (D + 32) / (D + 16)), dtype, D, n, 2 * H // Hk, 2, 1.0)
    for x, more in zip(("dq", "dk"), _slope_error(d, cap, D)):
        bounds[x] = bounds[x] + 1.1 * more
    for x, heads_of in (("dq", hq), ("dk", hk), ("dv", hk)):
        within(f64(got[x])[:, heads_of], ref[x], bounds[x], label + x)


def _not_finite(v, at):
    """v with +inf, -inf and NaN in single columns of some keys, and the same with zeros there; [(key, head, column, value)]."""
    inf, nan = float("inf"), float("nan")
    places = [(120, 0, 3, inf), (150, 0, 3, -inf), (64, 0, 9, -inf), (200, 0, 5, nan), (130, 0, 7, inf), (260, 0, 7, nan),
              (0, 1, 0, inf), (299, 1, 31, -inf), (256, 1, 30, nan), (255, 1, 29, inf)]
    with_them, without = v.clone(), v.clone()
    for key, head, column, x in places:
        with_them[at + key, head, column], without[at + key, head, column] = x, 0
    return with_them, without, places


def _with_rest(y, places, at, n, seen, group):
    """What becomes of y (of the values without them) by the formula: a seen infinity is the column's, a seen NaN or two
    infinities make it NaN.  seen(key): first row that sees it."""
    y = y.clone()
    for key, head, column, x in places:
        rows = slice(at + seen(key), at + n)
        y[rows, head * group:(head + 1) * group, column] += x
    return y


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,D", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("fp32", 32), ("fp32", 64), ("fp32", 128)])
@pytest.mark.parametrize("how", [{}, dict(prefix=140), dict(cap=50.0), dict(bias="buckets"), dict(causal=False), dict(cap=60.0),
                                 dict(bias="slopes"), dict(bias="slopes", cap=5.0), dict(bias="buckets", cap=5.0)], ids=str)
def test_columns_of_seen_and_hidden_values_are_told_apart(dtype, D, heads, how):
    """Infinities and NaN of V in single columns: a row has those that it sees, in their columns, and its other columns,
    and every column of rows that see none, are as they are without them, to the bit."""
    H, Hk = HEADS[heads]
    lens, at, n = [33, 300, 20], 33, 300
    d = make(26 + D, sum(lens), sum(lens), H, Hk, D, dtype, bias=how.get("bias", "none"))
    pre = how.get("prefix", 0 if how.get("causal", True) else n)
    args = dict(causal=how.get("causal", True), softcap=how.get("cap", 0.0),
                **{x: None if d[x] is None else d[x].cuda() for x in ("slopes", "table")},
                prefix=torch.tensor([0, pre, 0], dtype=torch.int64).cuda() if "prefix" in how else None)
    bad, good, places = _not_finite(d["v"], at)
    q, k, cu = d["q"].cuda(), d["k"].cuda(), offsets(lens).cuda()
    y0, lse0 = ssd.ssd_attn_forward(q, k, good.cuda(), cu, lse=True, **args)
    y, lse = ssd.ssd_attn_forward(q, k, bad.cuda(), cu, lse=True, **args)
    torch.cuda.synchronize()
    want = _with_rest(y0, places, at, n, lambda key: 0 if key < pre else key, H // Hk)
    assert torch.equal(lse, lse0)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y, 7.0, 1e30, -1e30), torch.nan_to_num(want, 7.0, 1e30, -1e30))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cap", [50.0, 55.0, 60.0])
@pytest.mark.parametrize("sign,size", [(1, 1e18), (-1, 1e-18), (1, 1e-18), (-1, 1e18)])
def test_scores_at_the_cap_with_values_of_any_size(sign, size, cap, dtype, heads):
    """Rows all of whose scores are at the cap or at its negative, where weights are e^cap or e^-cap before they are
    divided by their sum; other rows of the same tiles keep the bits that they have without them."""
    H, Hk = HEADS[heads]
    n, D = 200, 64
    d = make(27, n, n, H, Hk, D, dtype)
    d["v"] *= size
    d["k"][:, :, 0] = 8.0
    d["q"][:, :, 0] = 0.0
    cu = offsets([n])
    q, k, v = (d[x].cuda() for x in "qkv")
    plain, _ = ssd.ssd_attn_forward(q, k, v, cu.cuda(), softcap=cap)
    loud = torch.arange(n) % 5 == 2
    d["q"][loud, :, 0] = sign * 1000.0
    y, _ = ssd.ssd_attn_forward(d["q"].cuda(), k, v, cu.cuda(), softcap=cap)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu()[~loud], plain.cpu()[~loud])
    hk, hq = slice(0, 2), slice(0, 2 * H // Hk)
    d = dict(d, q=d["q"][:, hq], k=d["k"][:, hk], v=d["v"][:, hk])
    ref = reference(d, cu=cu.numpy(), cap=cap)
    # at the cap a score is off by the 4 u of its tanh times the cap, whatever its terms' magnitudes
    keep = np.where(loud.numpy()[:, None], 2 * cap / (D + 32), ref["s_abs"])
    within(f64(y)[:, hq], ref["y"], _capped_bound(dict(ref, s_abs=keep), dtype, D, n), "at the cap %g %s" % (cap, dtype))


GUARD = 64  # rows


class _Guarded:
    """Outputs and a workspace with a pattern in them and behind them, and the C entry points called on them."""

    def __init__(self, g, cu, table):
        self.g, self.cu, self.table, q, k = g, cu, table, g["q"], g["k"]
        self.dims = attention._dims(q, k, g["v"], cu, None, True, None, 0.0, None, table, 128, False, None)
        need = ssd.ssd_attn_backward_workspace_bytes(self.dims, table is not None)
        self.ws, self.need = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda"), need
        self.out = {n: torch.full((len(t) + GUARD, *t.shape[1:]), 7.0, dtype=t.dtype, device="cuda")
                    for n, t in (("y", q), ("dq", q), ("dk", k), ("dv", k))}
        self.out["lse"] = torch.full((len(q) + GUARD, q.shape[1]), 7.0, device="cuda")
        if table is not None:
            self.out["dtable"] = torch.full((len(table) + GUARD, q.shape[1]), 7.0, device="cuda")

    def run(self):
        a, o, g = attention._addr, {n: attention._addr(t) for n, t in self.out.items()}, self.g
        ins = [ctypes.byref(self.dims), a(self.cu), None, None, a(g["q"]), a(g["k"]), a(g["v"]), None, a(self.table)]
        dev = g["q"].device
        attention._call("ssd_attn_forward", dev, None, *ins, o["y"], o["lse"])
        attention._call("ssd_attn_backward", dev, None, *ins, o["y"], o["lse"], a(g["dy"]), o["dq"], o["dk"], o["dv"],
                        o.get("dtable"), a(self.ws), self.need)
        torch.cuda.synchronize()

    def check_untouched(self, first):
        """Rows from ``first`` on (of a table: behind its last) and what is behind the workspace are as they were."""
        for n, t in self.out.items():
            assert torch.all(t[len(self.table) if n == "dtable" else first:] == 7.0), n
        assert torch.all(self.ws[self.need:] == 0x5A)


def _guarded(heads, dtype, total, table):
    H, Hk = HEADS[heads]
    d = make(28, total, total, H, Hk, 64, dtype, bias="buckets" if table else "none", grads=True)
    return {n: d[n].cuda() for n in ("q", "k", "v", "dy")}, d["table"].cuda() if table else None


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("table", [False, True])
def test_backward_writes_no_row_of_no_sequence(table, dtype, heads):
    """Tokens behind the last sequence (NaN themselves) keep what their rows of every output held, and nothing is
    written behind the outputs and the workspace; the sequences' rows have nothing of that pattern."""
    lens, extra = [70, 0, 133], 45
    n = sum(lens)
    g, table = _guarded(heads, dtype, n + extra, table)
    for t in g.values():
        t[n:] = float("nan")
    case = _Guarded(g, offsets(lens).cuda(), table)
    case.run()
    case.check_untouched(n)
    for name, t in case.out.items():
        rows = t[:len(table)] if name == "dtable" else t[:n]
        assert torch.all(torch.isfinite(rows)) and not torch.any(torch.all(rows.flatten(1) == 7.0, 1)), name


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [[0, 500, -7, 300], [200, 100, 300, 250], [-1, -1, 10 ** 12, 5], [300, 300, 300, 300],
                                 [290, 10, 290, 10]], ids=str)
def test_malformed_offsets_write_inside_the_outputs(bad, dtype, heads):
    """Offsets that fall, repeat or lie outside the axis: some gradients, and nothing behind any output."""
    g, table = _guarded(heads, dtype, 300, True)
    case = _Guarded(g, torch.tensor(bad, dtype=torch.int64, device="cuda"), table)
    case.run()
    case.check_untouched(300)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
@pytest.mark.parametrize("how", [{}, dict(cap=50.0), dict(bias="buckets")], ids=str)
def test_gradients_of_rows_with_one_dominating_key(how, dtype, D, heads):
    """A key that takes 90 to 99% of every row's weight, in rows of several tiles: within grad_bounds, whose part for
    the rounding of y is the largest there, and the table's gradient without it."""
    H, Hk = HEADS[heads]
    n, cap = 260, how.get("cap", 0.0)
    d = make(29, n, n, H, Hk, D, dtype, bias=how.get("bias", "none"), grads=True)
    d["q"] += 6 * D ** -0.5
    d["k"][0] = 16 * D ** -0.5 * (D / 64) ** 0.5
    if d["table"] is not None:
        d["table"] *= 0.25
    cu = offsets([n])
    args = dict(softcap=cap, table=None if d["table"] is None else d["table"].cuda())
    g = {x: d[x].cuda() for x in ("q", "k", "v", "dy")}
    y, lse = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], cu.cuda(), lse=True, **args)
    got = ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y, lse, g["dy"], cu.cuda(), **args)
    torch.cuda.synchronize()
    hk, hq = slice(0, 2), slice(0, 2 * H // Hk)
    d = dict(d, q=d["q"][:, hq], dy=d["dy"][:, hq], k=d["k"][:, hk], v=d["v"][:, hk],
             table=None if d["table"] is None else d["table"][:, hq])
    first = reference(d, cu=cu.numpy(), cap=cap)
    ref = reference(d, cu=cu.numpy(), cap=cap, dy=d["dy"], y_err=y_bound(first, dtype, D, n, cap))
    top = np.exp(D ** -0.5 * np.einsum("ihd,hd->ih", f64(d["q"]), f64(d["k"][0]).repeat(H // Hk, 0)) - first["lse"])
    assert cap or d["table"] is not None or np.median(top[130:]) > 0.9
    bounds = grad_bounds(ref, dtype, D, n, 2 * H // Hk, 2, cap)
    for x in sorted(bounds):
        within(f64(got[x])[:, hk if x in ("dk", "dv") else hq], ref[x], bounds[x], "peaked %s %s D%d %s" % (how, dtype, D, x))


def _rounding_variance(d, causal, cap, rounded_sum, D):
    """What independent roundings leave in dq and dk of one document, as elementwise variances: a rounding is off by at most
    U of its value, its variance at most U^2 / 3 of the square.  dS (times the cap's derivative) is rounded once on its way to
    the matrix unit, dq and dk once at the end; where D is put right by the sum of rounded dS, their roundings' sum goes
    with p into both."""
    q, k, v, dy = (f64(d[x]).transpose(1, 0, 2) for x in ("q", "k", "v", "dy"))
    group, n, var, scale = len(q) // len(k), q.shape[1], U["bf16"] ** 2 / 3, D ** -0.5
    got = {x: np.zeros_like(y) for x, y in (("dq", q), ("dk", k), ("dq_var", q), ("dk_var", k))}
    for h in range(len(q)):
        K, V = k[h // group], v[h // group]
        z = scale * q[h] @ K.T
        c1 = 1 - np.tanh(z / cap) ** 2 if cap else 1.0
        z = cap * np.tanh(z / cap) if cap else z
        if d["slopes"] is not None or d["table"] is not None:
            rel = np.arange(n)[None] - np.arange(n)[:, None]
            z = z + oa.bias_of(rel, h, f64(d["slopes"]), f64(d["table"]), 128, not causal)[0]
        w = np.where(np.tril(np.ones((n, n), bool)), np.exp(z - z.max(-1, keepdims=True)), 0.0) if causal else np.exp(z - z.max(-1, keepdims=True))
        p = w / w.sum(-1, keepdims=True)
        dp = dy[h] @ V.T
        ds = p * (dp - (p * dp).sum(-1, keepdims=True))
        all_ds = (ds ** 2).sum(-1, keepdims=True) if rounded_sum else np.zeros((n, 1))
        ds, pc = ds * c1 * scale, p * c1 * scale
        got["dq"][h] = ds @ K
        got["dk"][h // group] += ds.T @ q[h]
        got["dq_var"][h] = var * ((ds ** 2) @ K ** 2 + all_ds * (pc @ K) ** 2)
        got["dk_var"][h // group] += var * (ds.T ** 2 @ q[h] ** 2 + (pc ** 2 * all_ds).T @ q[h] ** 2)
    for x in ("dq", "dk"):
        got[x + "_var"] += var * got[x] ** 2
    return {x: y.transpose(1, 0, 2) for x, y in got.items()}


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("how", [{}, dict(cap=50.0), dict(bias="slopes"), dict(bias="buckets"), dict(bias="buckets", cap=50.0),
                                 dict(causal=False)], ids=str)
@pytest.mark.parametrize("data", ["common part", "dominating key"])
def test_gradients_without_the_rounding_of_y(data, how, D, heads):
    """dq and dk in bf16 are off by the roundings of dS and of themselves, and not by what the rounding of y leaves in
    dy.y, which keys and values with a common part, or one key with most of the weight, pass on whole (10 to 40 times
    the rest).  In the 2-norm, where independent errors add up to the root of their variances' sum: some 1e4 of them, so
    within 1.2 of it; the fp32 parts are under a hundredth of that."""
    H, Hk = HEADS[heads]
    n, cap, causal = 300, how.get("cap", 0.0), how.get("causal", True)
    d = make(31, n, n, H, Hk, D, "bf16", bias=how.get("bias", "none"), grads=True)
    if data == "common part":
        d["k"] += 2.0
        d["v"] += 2.0
    else:
        d["q"] += 6 * D ** -0.5
        d["k"][0] = 16 * D ** -0.5 * (D / 64) ** 0.5
    if d["slopes"] is not None:
        d["slopes"] *= 0.01
    cu = offsets([n])
    g = {x: d[x].cuda() for x in ("q", "k", "v", "dy")}
    args = dict(softcap=cap, causal=causal, bidirectional=not causal, **{x: None if d[x] is None else d[x].cuda() for x in ("slopes", "table")})
    y, lse = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], cu.cuda(), lse=True, **args)
    got = ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y, lse, g["dy"], cu.cuda(), **args)
    torch.cuda.synchronize()
    hk, hq = slice(0, 2), slice(0, 2 * H // Hk)
    d = dict(d, q=d["q"][:, hq], dy=d["dy"][:, hq], k=d["k"][:, hk], v=d["v"][:, hk],
             slopes=None if d["slopes"] is None else d["slopes"][hq], table=None if d["table"] is None else d["table"][:, hq])
    ref = _rounding_variance(d, causal, cap, not cap and d["table"] is None, D)
    for x, h in (("dq", hq), ("dk", hk)):
        err, want = np.linalg.norm(f64(got[x])[:, h] - ref[x]), np.sqrt(ref[x + "_var"].sum())
        print("[gpu case] %s %s D%d %s %s: error %.3g of its bound, %.3g of %s" % (data, how, D, heads, x, err / (1.2 * want),
                                                                                  err / np.linalg.norm(ref[x]), x), flush=True)
        assert err <= 1.2 * want, (x, err, want)
