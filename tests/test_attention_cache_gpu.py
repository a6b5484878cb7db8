"""GPU tests of the paged cache: the append with its rotation and attention of single tokens."""
import numpy as np
import pytest
import torch

import oracle.attention as oa
import ssd_chunked_scan_02_amd as ssd
from attn_helpers import DTYPE, U, f64, make, offsets, reference, within, y_bound

pytestmark = pytest.mark.gpu


def _pool(seed, lens, page, Hk, D, dtype, spare=2):
    """Caches of random values and a block table with the pages in shuffled order; unused entries are no pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g)
    table = torch.tensor([[-1, 1 << 30][i % 2] for i in range(len(lens) * (max(need) + 1))], dtype=torch.int32).view(len(lens), -1)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n].to(torch.int32)
        at += n
    caches = [torch.randn((pool, page, Hk, D), generator=g).to(DTYPE[dtype]) for _ in range(2)]
    return caches, table


def _gathered(cache, table, lens):
    """The sequences' cached rows, packed."""
    page = cache.shape[1]
    return torch.cat([cache[table[i, :-(-n // page)].long()].flatten(0, 1)[:n] for i, n in enumerate(lens)])


def _decode_case(dtype, D, H, Hk, page, lens, bias="none", cap=0.0, seed=1, **how):
    n = len(lens)
    d = make(seed, n, 1, H, Hk, D, dtype, bias=bias)
    (kc, vc), table = _pool(seed, lens, page, Hk, D, dtype)
    gpu = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = ssd.ssd_attn_decode(gpu(d["q"]), gpu(kc), gpu(vc), gpu(table), torch.tensor(lens, dtype=torch.int64).cuda(),
                            softcap=cap, slopes=gpu(d["slopes"]), table=gpu(d["table"]), **how)
    torch.cuda.synchronize()
    d["k"], d["v"] = _gathered(kc, table, lens), _gathered(vc, table, lens)
    ref = reference(d, cu=list(range(n + 1)), cu_k=offsets(lens).numpy(), cap=cap, **how)
    within(f64(y), ref["y"], y_bound(ref, dtype, D, max(lens), cap), "decode %s D%d H%d/%d page %d %s" % (dtype, D, H, Hk, page, lens[:4]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,H,Hk", [(32, 3, 3), (64, 16, 2), (64, 40, 2), (128, 8, 1), (128, 6, 2)])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_decode_shapes(dtype, D, H, Hk, page):
    """Groups below, at and above the 16 heads of a workgroup; pages that end inside a block; odd lengths."""
    _decode_case(dtype, D, H, Hk, page, [1, 16, 17, 31, 32, 33, 500, 129])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bias,cap,how", [("slopes", 0.0, {}), ("buckets", 0.0, {}), ("none", 4.0, {}), ("slopes", 4.0, {}),
                                          ("buckets", 30.0, dict(max_distance=17, bidirectional=True)),
                                          ("buckets", 0.0, dict(max_distance=1024))])
def test_decode_bias_and_cap(dtype, bias, cap, how):
    _decode_case(dtype, 64, 6, 3, 32, [700, 3, 130, 1100], bias=bias, cap=cap, **how)


def test_decode_one_long_sequence():
    """Split 64 ways, with a block table far wider than the sequence."""
    _decode_case("bf16", 128, 8, 2, 64, [20001], seed=3)


def test_decode_many_sequences():
    """More workgroups than the split rule wants: no split, no workspace."""
    _decode_case("bf16", 64, 32, 32, 16, [1 + (37 * i) % 90 for i in range(40)], seed=4)


def test_decode_lengths_and_pages_out_of_range():
    """Empty and negative lengths give zeros, a length past the table is cut, and keys of no page are not seen."""
    dtype, D, H, Hk, page = "bf16", 64, 4, 2, 16
    lens = [0, -5, 40, 64, 48]
    (kc, vc), table = _pool(9, [64] * 5, page, Hk, D, dtype)
    table = table[:, :4].contiguous()
    table[4, 1] = -1                      # positions 16 .. 31 of the last sequence are nowhere
    table[3, 0] = kc.shape[0]             # one past the last page
    d = make(9, 5, 1, H, Hk, D, dtype)
    given = torch.tensor(lens, dtype=torch.int64)
    given[2] = 10 ** 12
    y = ssd.ssd_attn_decode(d["q"].cuda(), kc.cuda(), vc.cuda(), table.cuda(), given.cuda())
    torch.cuda.synchronize()
    assert torch.all(y[:2] == 0)
    for s, keep in ((2, range(64)), (3, range(16, 64)), (4, list(range(16)) + list(range(32, 48)))):
        rows = torch.tensor([int(table[s, t // page]) * page + t % page for t in keep])
        one = dict(q=d["q"][s:s + 1], k=kc.flatten(0, 1)[rows], v=vc.flatten(0, 1)[rows], slopes=None, table=None)
        ref = reference(one, cu=[0, 1], cu_k=[0, len(rows)])
        within(f64(y[s:s + 1]), ref["y"], y_bound(ref, dtype, D, len(rows), 0.0), "pages of sequence %d" % s)


def test_decode_ignores_what_lies_past_a_length():
    """NaN in the rest of the last page and in unused pages reach nothing; strided queries give the same bits."""
    lens, page, H, Hk, D = [21, 50], 32, 4, 2, 64
    (kc, vc), table = _pool(11, lens, page, Hk, D, "bf16")
    used = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for s, n in enumerate(lens):
        for t in range(n):
            used[int(table[s, t // page]), t % page] = True
    kn, vn = kc.clone(), vc.clone()
    kn[~used], vn[~used] = float("nan"), float("inf")
    q = make(11, 2, 1, H, Hk, D, "bf16")["q"].cuda()
    wide = torch.zeros((2, H * D + 64), dtype=q.dtype, device="cuda")
    wide[:, :H * D] = q.flatten(1)
    seq = torch.tensor(lens, dtype=torch.int64).cuda()
    a = ssd.ssd_attn_decode(q, kc.cuda(), vc.cuda(), table.cuda(), seq)
    b = ssd.ssd_attn_decode(wide[:, :H * D].unflatten(1, (H, D)), kn.cuda(), vn.cuda(), table.cuda(), seq)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def _angle_bound(x, dtype):
    """One output rounding, and in fp32 the sine and cosine (each off by some units of 2^-24, taken as 8) and
    the products: 12 u (|a| + |b|) with |a| + |b| at most twice the row's largest value."""
    return 1.05 * U[dtype] * np.abs(x) + 24 * 2.0 ** -24 * np.abs(x).max() + 1e-30


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,pairs,with_q", [(32, 16, True), (64, 8, True), (128, 64, True), (64, 32, False), (128, 0, True)])
def test_append(dtype, interleaved, D, pairs, with_q):
    """Prompts of odd lengths, one of them empty, after what is cached already; partial and no rotation."""
    new, past, page, H, Hk = [5, 0, 70, 1, 33], [0, 9, 3, 1000, 15], 16, 4, 2
    lens = [a + b for a, b in zip(new, past)]
    d = make(D + pairs, sum(new), sum(new), H, Hk, D, dtype)
    (kc, vc), table = _pool(5, lens, page, Hk, D, dtype)
    inv = 10000.0 ** (-torch.arange(pairs, dtype=torch.float32) / max(pairs, 1)) if pairs else None
    cu, seq = offsets(new), torch.tensor(lens, dtype=torch.int64)
    gk, gv = kc.cuda(), vc.cuda()
    q = ssd.ssd_kv_append(d["k"].cuda(), d["v"].cuda(), gk, gv, table.cuda(), seq.cuda(), cu.cuda(),
                          None if inv is None else inv.cuda(), interleaved, d["q"].cuda() if with_q else None)
    torch.cuda.synchronize()
    wk, wv, wq = oa.append(f64(d["k"]), f64(d["v"]), f64(kc), f64(vc), table.numpy(), lens, cu.numpy(),
                           None if inv is None else f64(inv), interleaved, f64(d["q"]) if with_q else None)
    label = "append %s D%d %d %s" % (dtype, D, pairs, interleaved)
    within(f64(gk), wk, _angle_bound(wk, dtype), label + " k")
    assert np.array_equal(f64(gv), wv)
    if with_q:
        within(f64(q), wq, _angle_bound(wq, dtype), label + " q")
    else:
        assert q is None


def test_append_far_positions():
    """A position of two million: its fastest angle has to be reduced before it is rounded to 32 bits."""
    page, H, Hk, D = 65536, 2, 1, 64
    d = make(2, 1, 1, H, Hk, D, "fp32")
    table = torch.full((1, 32), -1, dtype=torch.int32)
    table[0, 30] = 0
    pos = 30 * page + 33333
    cache = torch.zeros((1, page, Hk, D))
    inv = 10000.0 ** (-torch.arange(32, dtype=torch.float32) / 32)
    seq = torch.tensor([pos + 1], dtype=torch.int64)
    gk, gv = cache.cuda(), cache.cuda()
    q = ssd.ssd_kv_append(d["k"].cuda(), d["v"].cuda(), gk, gv, table.cuda(), seq.cuda(), inv_freq=inv.cuda(), q=d["q"].cuda())
    torch.cuda.synchronize()
    wk, _, wq = oa.append(f64(d["k"]), f64(d["v"]), f64(cache), f64(cache), table.numpy(), [pos + 1], None, f64(inv), False, f64(d["q"]))
    within(f64(gk), wk, _angle_bound(wk, "fp32"), "far k")
    within(f64(q), wq, _angle_bound(wq, "fp32"), "far q")


def test_append_places_out_of_range():
    """Positions before the start or past the table and entries that are no page leave the cache as it was."""
    page, Hk, D = 16, 1, 32
    (kc, vc), table = _pool(7, [32, 32, 32], page, Hk, D, "fp32")
    table = table[:, :2].contiguous()
    table[1, 0] = kc.shape[0]
    new = [3, 20, 2]
    lens = [1, 20, 33]  # first: positions -2, -1, 0; second: page 0 is none; third: 31, 32 of 32
    d = make(8, sum(new) + 2, sum(new) + 2, 2, Hk, D, "fp32")  # two tokens of no sequence
    cu = offsets(new)
    gk, gv = kc.cuda(), vc.cuda()
    out = torch.full_like(d["q"], 7.0).cuda()
    ssd.ssd_kv_append(d["k"].cuda(), d["v"].cuda(), gk, gv, table.cuda(), torch.tensor(lens, dtype=torch.int64).cuda(), cu.cuda(),
                      q=d["q"].cuda(), q_out=out)
    torch.cuda.synchronize()
    wk, wv, _ = oa.append(f64(d["k"]), f64(d["v"]), f64(kc), f64(vc), table.numpy(), lens, cu.numpy())
    assert np.array_equal(f64(gk), wk) and np.array_equal(f64(gv), wv)
    assert torch.equal(out[:25].cpu(), d["q"][:25]) and torch.all(out[25:] == 7.0)


def test_prompt_then_steps():
    """The operators as they are used together: a packed prompt's attention, its append, then single tokens,
    each appended and attended, in a HIP graph; every token against attention over the whole sequence."""
    torch.manual_seed(0)
    H, Hk, D, page, steps, prompts = 4, 2, 64, 16, 6, [37, 5]
    total = [n + steps for n in prompts]
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float32) / 32)).cuda()
    dtype = torch.float32
    q, k, v = (torch.randn((sum(total), h, D), device="cuda", dtype=dtype) for h in (H, Hk, Hk))
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625], device="cuda")
    cu_all = offsets(total)
    first = [int(c) for c in cu_all[:-1]]
    # the whole sequences at once, rotated through a cache of their own
    width = -(-max(total) // page)
    pages = torch.arange(2 * width, dtype=torch.int32, device="cuda").view(2, width).flip(0).contiguous()
    full = [torch.zeros((2 * width, page, Hk, D), device="cuda", dtype=dtype) for _ in range(2)]
    lens = torch.tensor(total, dtype=torch.int64, device="cuda")
    qr = ssd.ssd_kv_append(k, v, *full, pages, lens, cu_all.cuda(), inv, q=q)
    kr = torch.cat([full[0][pages[s].long()].flatten(0, 1)[:n] for s, n in enumerate(total)])
    want, _ = ssd.ssd_attn_forward(qr, kr, v, cu_all.cuda(), softcap=20.0, slopes=slopes)

    rows = torch.cat([torch.arange(f, f + n) for f, n in zip(first, prompts)]).cuda()
    cache = [torch.zeros_like(full[0]) for _ in range(2)]
    seq = torch.tensor(prompts, dtype=torch.int64, device="cuda")
    cu = offsets(prompts).cuda()
    qp = ssd.ssd_kv_append(k[rows], v[rows], *cache, pages, seq, cu, inv, q=q[rows])
    got, _ = ssd.ssd_attn_forward(qp, kr[rows], v[rows], cu, softcap=20.0, slopes=slopes)
    # same keys in the same tiles: the prompt's rows are the same sums in both calls
    assert torch.allclose(got, want[rows], rtol=0, atol=1e-6)

    one = [t[:2].clone() for t in (q, k, v)]
    y, q1 = torch.empty_like(one[0]), torch.empty_like(one[0])
    dims = ssd.attention._cache_dims(one[0], H, *cache, pages, seq, (0, 0, 0), None, 20.0, 0, 0, False)
    ws = torch.empty(max(1, ssd.ssd_attn_decode_workspace_bytes(dims)), dtype=torch.uint8, device="cuda")

    def step():
        ssd.ssd_kv_append(one[1], one[2], *cache, pages, seq, None, inv, q=one[0], q_out=q1)
        ssd.ssd_attn_decode(q1, *cache, pages, seq, softcap=20.0, slopes=slopes, y=y, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    seq += 1  # (the capture runs nothing; the first replay appends at this length)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        at = torch.tensor([f + n + i for f, n in zip(first, prompts)], device="cuda")
        for to, x in zip(one, (q, k, v)):
            to.copy_(x[at])
        graph.replay()
        torch.cuda.synchronize()
        # (fp32 sums of 50 terms of size 1 to 20 in another order)
        assert torch.allclose(y, want[at], rtol=0, atol=2e-5), i
        seq += 1
