"""GPU tests of the paged cache in 8 bits: the append that quantises, the decode step over it and the read-back.

What the cache holds stands for scale * x8.  The decode step is tested on those values against the fp64 attention, with
the bounds of the 16-bit cache's (both forms of x8 are exact operands; a key's scale is one more rounding of its score and a
value's one of its weight, 2^-24 each)."""
import numpy as np
import pytest
import torch

import oracle.attention as oa
import ssd_chunked_scan_02_amd as ssd
from attn_helpers import DTYPE, U, f64, make, offsets, reference, within, y_bound
from test_attention_cache_gpu import _angle_bound

pytestmark = pytest.mark.gpu
FORMS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}


def values(cache, scale):
    """What a cache stands for, in fp64 on the CPU."""
    return cache.cpu().float().double() * scale.cpu().double()[..., None]


def pool(seed, lens, page, Hk, D, form, spare=2):
    """Random pages (cpu): caches, scales, and a block table in shuffled order; unused entries are no pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    count = sum(need) + spare
    order = torch.randperm(count, generator=g)
    table = torch.tensor([[-1, 1 << 30][i % 2] for i in range(len(lens) * (max(need) + 1))], dtype=torch.int32).view(len(lens), -1)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n].to(torch.int32)
        at += n
    kv = []
    for _ in "kv":
        x = torch.randn((count, page, Hk, D), generator=g) * 0.4 * TOP[form]
        kv.append(x.clamp(-TOP[form], TOP[form]).round().to(FORMS[form]))
    scales = [(0.3 + torch.rand((count, page, Hk), generator=g)) * 2.5 / TOP[form] for _ in "kv"]
    return kv, scales, table


def gathered(x, table, lens):
    page = x.shape[1]
    return torch.cat([x[table[i, :-(-n // page)].long()].flatten(0, 1)[:n] for i, n in enumerate(lens)])


def decode_case(dtype, form, D, H, Hk, page, lens, bias="none", cap=0.0, seed=1, **how):
    n = len(lens)
    d = make(seed, n, 1, H, Hk, D, dtype, bias=bias)
    (kc, vc), (ks, vs), table = pool(seed, lens, page, Hk, D, form)
    gpu = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = ssd.ssd_kv8_decode(gpu(d["q"]), gpu(kc), gpu(vc), gpu(ks), gpu(vs), gpu(table), torch.tensor(lens, dtype=torch.int64).cuda(),
                           softcap=cap, slopes=gpu(d["slopes"]), table=gpu(d["table"]), **how)
    torch.cuda.synchronize()
    d["k"], d["v"] = gathered(values(kc, ks), table, lens), gathered(values(vc, vs), table, lens)
    ref = reference(d, cu=list(range(n + 1)), cu_k=offsets(lens).numpy(), cap=cap, **how)
    within(f64(y), ref["y"], y_bound(ref, dtype, D, max(lens), cap), "kv8 decode %s %s D%d H%d/%d page %d %s" % (dtype, form, D, H, Hk, page, lens[:4]))


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,H,Hk", [(32, 3, 3), (64, 16, 2), (64, 40, 2), (128, 8, 1), (128, 6, 2)])
@pytest.mark.parametrize("page", [16, 48])
def test_decode_shapes(dtype, form, D, H, Hk, page):
    """Groups below, at and above the 16 heads of a workgroup; pages that end inside a block; odd lengths."""
    decode_case(dtype, form, D, H, Hk, page, [1, 16, 17, 31, 32, 33, 500, 129])


@pytest.mark.parametrize("dtype,form", [("bf16", "int8"), ("bf16", "e4m3"), ("fp32", "int8"), ("fp32", "e4m3")])
@pytest.mark.parametrize("bias,cap,how", [("slopes", 0.0, {}), ("buckets", 0.0, {}), ("none", 4.0, {}), ("slopes", 4.0, {}),
                                          ("buckets", 30.0, dict(max_distance=17, bidirectional=True)), ("none", 0.0, dict(scale=-0.3))])
def test_decode_bias_cap_and_scale(dtype, form, bias, cap, how):
    decode_case(dtype, form, 64, 6, 3, 32, [700, 3, 130, 1100], bias=bias, cap=cap, **how)


def test_decode_one_long_sequence():
    decode_case("bf16", "e4m3", 128, 8, 2, 64, [20001], seed=3)


def test_decode_many_sequences():
    """More workgroups than the split rule wants, and (24 of 90 keys) the eight-wave form."""
    decode_case("bf16", "int8", 64, 32, 32, 16, [1 + (37 * i) % 90 for i in range(40)], seed=4)
    decode_case("fp32", "e4m3", 128, 8, 8, 16, [1 + (37 * i) % 90 for i in range(24)], seed=5)


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_every_value_of_a_byte(form):
    """All 256 (254) values of either form come back exactly, in the read-back and through the decode's operands."""
    codes = torch.arange(256, dtype=torch.uint8)
    if form == "e4m3":
        codes[0x7f], codes[0xff] = 0, 0  # (NaN)
    page, Hk, D = 16, 1, 32
    kc = codes.repeat(2).view(1, page, Hk, D).view(FORMS[form])
    ks = torch.ones((1, page, Hk))
    table, seq = torch.zeros((1, 1), dtype=torch.int32), torch.tensor([page])
    args = [t.cuda() for t in (kc, kc, ks, ks, table, seq)]
    for dtype in ("fp32", "bf16"):
        k, v = ssd.ssd_kv8_read(*args, None, page, dtype=DTYPE[dtype])
        assert torch.equal(k.cpu().float(), kc[0].float()) and torch.equal(k, v)
        # one key at a time: the softmax of one score is one, and y the value itself
        for t in range(page):
            one = (kc[:, t:t + 1].expand(1, page, Hk, D).contiguous().cuda(),) * 2
            y = ssd.ssd_kv8_decode(torch.zeros((1, 1, D), dtype=DTYPE[dtype], device="cuda"), *one, *args[2:5], torch.tensor([1], device="cuda"))
            assert torch.equal(y[0, 0].cpu().float(), kc[0, t, 0].float()), t


def test_decode_lengths_and_pages_out_of_range():
    """Empty and negative lengths give zeros, a length past the table is cut, and keys of no page are not seen."""
    dtype, D, H, Hk, page = "bf16", 64, 4, 2, 16
    lens = [0, -5, 40, 64, 48]
    (kc, vc), (ks, vs), table = pool(9, [64] * 5, page, Hk, D, "int8")
    table = table[:, :4].contiguous()
    table[4, 1] = -1                      # positions 16 .. 31 of the last sequence are nowhere
    table[3, 0] = kc.shape[0]             # one past the last page
    d = make(9, 5, 1, H, Hk, D, dtype)
    given = torch.tensor(lens, dtype=torch.int64)
    given[2] = 10 ** 12
    cache = [t.cuda() for t in (kc, vc, ks, vs, table, given)]
    y = ssd.ssd_kv8_decode(d["q"].cuda(), *cache)
    rows = torch.tensor([0, 5, 10, 80, 144, 200]).cuda()
    k, v = ssd.ssd_kv8_read(*cache, rows, 200, dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.all(y[:2] == 0)
    kd, vd = values(kc, ks).flatten(0, 1), values(vc, vs).flatten(0, 1)
    assert torch.all(k[:10] == 0) and torch.all(v[:10] == 0)
    for s, keep in ((2, range(64)), (3, range(16, 64)), (4, list(range(16)) + list(range(32, 48)))):
        at = torch.tensor([int(table[s, t // page]) * page + t % page for t in keep])
        one = dict(q=d["q"][s:s + 1], k=kd[at], v=vd[at], slopes=None, table=None)
        ref = reference(one, cu=[0, 1], cu_k=[0, len(at)])
        within(f64(y[s:s + 1]), ref["y"], y_bound(ref, dtype, D, len(at), 0.0), "pages of sequence %d" % s)
        want = torch.zeros((int(rows[s + 1] - rows[s]), Hk, D))
        want[list(keep)] = kd[at].float()
        assert torch.equal(k[int(rows[s]):int(rows[s + 1])].cpu(), want)


def test_decode_ignores_what_lies_past_a_length():
    """NaN scales in the rest of the last page and in unused pages reach nothing; strided queries give the same bits."""
    lens, page, H, Hk, D = [21, 50], 32, 4, 2, 64
    (kc, vc), (ks, vs), table = pool(11, lens, page, Hk, D, "e4m3")
    used = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for s, n in enumerate(lens):
        for t in range(n):
            used[int(table[s, t // page]), t % page] = True
    bad = [t.clone() for t in (ks, vs)]
    for t in bad:
        t[~used] = float("nan")
    q = make(11, 2, 1, H, Hk, D, "bf16")["q"].cuda()
    wide = torch.zeros((2, H * D + 64), dtype=q.dtype, device="cuda")
    wide[:, :H * D] = q.flatten(1)
    seq = torch.tensor(lens, dtype=torch.int64).cuda()
    kc, vc, table = kc.cuda(), vc.cuda(), table.cuda()
    a = ssd.ssd_kv8_decode(q, kc, vc, ks.cuda(), vs.cuda(), table, seq)
    b = ssd.ssd_kv8_decode(wide[:, :H * D].unflatten(1, (H, D)), kc, vc, *[t.cuda() for t in bad], table, seq)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def append_case(dtype, form, H, Hk, D, page, new, past, rot, interleaved, seed=1):
    """One append on the GPU, and its exact rotations in fp64."""
    lens = [a + b for a, b in zip(new, past)]
    (kc, vc), (ks, vs), table = pool(seed, lens, page, Hk, D, form)
    n = sum(new)
    d = make(seed, n, n, H, Hk, D, dtype)
    d["v"][::3] = 0                                     # (a head of zeros has scale zero)
    inv = (10000.0 ** (-torch.arange(rot, dtype=torch.float64) / max(rot, 1))).float()
    cu, seq = offsets(new), torch.tensor(lens, dtype=torch.int64)
    before = [t.clone() for t in (kc, vc, ks, vs)]
    cache = [t.cuda() for t in (kc, vc, ks, vs)]
    q = ssd.ssd_kv8_append(d["k"].cuda(), d["v"].cuda(), *cache, table.cuda(), seq.cuda(), cu_seqlens=cu.cuda(),
                           inv_freq=inv.cuda() if rot else None, interleaved=interleaved, q=d["q"].cuda())
    torch.cuda.synchronize()
    wide = [torch.zeros(kc.shape, dtype=torch.float64).numpy() for _ in "kv"]
    want = oa.append(f64(d["k"]), f64(d["v"]), *wide, table.numpy(), seq.numpy(), cu=cu.numpy(), inv_freq=f64(inv) if rot else None,
                     interleaved=interleaved, q=f64(d["q"]))
    return d, q, cache, before, want, (table, lens, new)


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,H,Hk,rot,interleaved", [(32, 3, 3, 16, False), (64, 8, 2, 32, True), (128, 4, 4, 64, False), (128, 6, 1, 8, True),
                                                    (64, 2, 2, 16, False), (64, 4, 1, 0, False)])
def test_append(dtype, form, D, H, Hk, rot, interleaved):
    """Scales to an fp32's last bits, held values within half a step, the rest of the cache to the bit."""
    d, q, cache, before, want, (table, lens, new) = append_case(dtype, form, H, Hk, D, 16, [1, 37, 0, 16, 5], [100, 3, 9, 0, 20000], rot, interleaved)
    wk, wv, wq = (np.asarray(x) for x in want[:3])
    within(f64(q), wq, _angle_bound(wq, dtype), "kv8 append q")
    page = 16
    written = torch.zeros(cache[0].shape[:2], dtype=torch.bool)
    for s, n in enumerate(new):
        for t in range(lens[s] - n, lens[s]):
            written[int(table[s, t // page]), t % page] = True
    for name, x8, sc, old8, olds, exact in (("k", cache[0], cache[2], before[0], before[2], wk), ("v", cache[1], cache[3], before[1], before[3], wv)):
        x8, sc = x8.cpu(), sc.cpu()
        assert torch.equal(x8[~written].view(torch.uint8), old8[~written].view(torch.uint8)) and torch.equal(sc[~written], olds[~written])
        got, scale, x = values(x8, sc)[written].numpy(), sc[written].double().numpy(), exact[written.numpy()]
        top = np.abs(x).max(-1)
        # the rotation's own error, relative to the head's largest value: 24 u (see _angle_bound), then the scale's two
        assert np.all(np.abs(scale - top / TOP[form]) <= (24 + 3) * 2.0 ** -24 * top / TOP[form] + 1e-45), name
        step = scale[..., None] / 2 if form == "int8" else np.maximum(2.0 ** -4 * np.abs(x), scale[..., None] * 2.0 ** -10)
        assert np.all(np.abs(got - x) <= step * (1 + 2.0 ** -20) + 30 * 2.0 ** -24 * top[..., None]), name
        assert np.all(np.abs(x8[written].float().numpy()).max(-1)[top > 0] == TOP[form]), name


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_append_values_to_the_bit(form):
    """Without a rotation the held values are the formula's in fp32, ties to even, element by element."""
    d, _, cache, before, _, (table, lens, new) = append_case("bf16", form, 4, 2, 64, 16, [50, 3], [7, 0], 0, False, seed=3)
    inv = torch.tensor(1.0 / TOP[form], dtype=torch.float64).float()
    first = 0
    for s, n in enumerate(new):
        at = [(int(table[s, t // 16]), t % 16) for t in range(lens[s] - n, lens[s])]
        for x, x8, sc in ((d["k"], cache[0], cache[2]), (d["v"], cache[1], cache[3])):
            x = x[first:first + n].float()
            scale = x.abs().amax(-1) * inv
            r = x / torch.where(scale > 0, scale, 1.0)[..., None]
            want = (r.round() if form == "int8" else r).clamp(-TOP[form], TOP[form]).to(FORMS[form])
            got = torch.stack([x8[p, o].cpu().view(torch.uint8) for p, o in at])
            assert torch.equal(torch.stack([sc[p, o].cpu() for p, o in at]), scale)
            assert torch.equal(got, want.view(torch.uint8))
        first += n


def test_append_of_extreme_heads():
    """Infinities and NaN make their own head NaN and no other; zeros, subnormals and the largest values are held."""
    D, Hk, page = 32, 6, 16
    x = torch.randn((1, Hk, D), generator=torch.Generator().manual_seed(1))
    x[0, 0, 3], x[0, 1, 4] = float("nan"), float("-inf")
    x[0, 2], x[0, 3] = 0.0, x[0, 3] * 1e-44
    x[0, 4] = x[0, 4].sign() * 3e38
    for form in FORMS:
        cache = [torch.zeros((1, page, Hk, D), dtype=torch.uint8, device="cuda").view(FORMS[form]) for _ in "kv"]
        scale = [torch.zeros((1, page, Hk), device="cuda") for _ in "kv"]
        table, seq = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([1], device="cuda")
        ssd.ssd_kv8_append(x.cuda(), x.cuda(), *cache, *scale, table, seq)
        k, v = ssd.ssd_kv8_read(*cache, *scale, table, seq, None, 1, dtype=torch.float32)
        torch.cuda.synchronize()
        k = k.cpu()
        assert torch.equal(k.nan_to_num(7.0), v.cpu().nan_to_num(7.0))
        assert torch.all(k[0, :2].isnan()) and torch.all(k[0, 2] == 0)
        assert torch.all((k[0, 3] - x[0, 3]).abs() <= x[0, 3].abs().max() / 4 + 1e-43)
        assert torch.all((k[0, 4] / x[0, 4] - 1).abs() < 1e-6)
        assert torch.all((k[0, 5] - x[0, 5]).abs() <= x[0, 5].abs().max() / 12)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_read(dtype, form):
    """The product in fp32, rounded once; rows past a length are zeros, rows of no sequence are left."""
    lens, page, Hk, D = [70, 0, 33, 16], 16, 3, 64
    (kc, vc), (ks, vs), table = pool(5, lens, page, Hk, D, form)
    rows = torch.tensor([2, 72, 75, 110, 126])                 # (the second and third have rows past their lengths)
    out = [torch.full((130, Hk, D), 5.0, dtype=DTYPE[dtype], device="cuda") for _ in "kv"]
    k, v = ssd.ssd_kv8_read(kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(), torch.tensor(lens).cuda(), rows.cuda(), 130,
                            dtype=DTYPE[dtype], k=out[0], v=out[1])
    torch.cuda.synchronize()
    assert k is out[0] and v is out[1]
    for got, x8, sc in ((k.cpu(), kc, ks), (v.cpu(), vc, vs)):
        want = torch.full((130, Hk, D), 5.0, dtype=DTYPE[dtype])
        want[2:126] = 0
        for s, n in enumerate(lens):
            at = [(int(table[s, t // page]), t % page) for t in range(n)]
            for i, (p, o) in enumerate(at):
                want[int(rows[s]) + i] = (x8[p, o].float() * sc[p, o][..., None]).to(DTYPE[dtype])
        assert torch.equal(got, want)


def test_prompt_continued_over_the_cache():
    """A prompt's second half attends to what is read back of the first, and the decode step to the same values."""
    torch.manual_seed(0)
    lens, more, H, Hk, D, page = [40, 7], [5, 3], 4, 2, 64, 16
    total = [a + b for a, b in zip(lens, more)]
    need = [-(-n // page) for n in total]
    table = torch.full((2, max(need)), -1, dtype=torch.int32)
    table[0, :need[0]], table[1, :need[1]] = torch.arange(need[0], dtype=torch.int32), need[0] + torch.arange(need[1], dtype=torch.int32)
    cache = [torch.zeros((sum(need), page, Hk, D), dtype=torch.int8, device="cuda") for _ in "kv"]
    scale = [torch.zeros((sum(need), page, Hk), device="cuda") for _ in "kv"]
    table = table.cuda()
    inv = ssd.ssd_rotary_frequencies(D)[0].cuda()
    for n, now in ((lens, lens), (more, total)):
        k, v = (torch.randn((sum(n), Hk, D), device="cuda").bfloat16() for _ in "kv")
        q = torch.randn((sum(n), H, D), device="cuda").bfloat16()
        q = ssd.ssd_kv8_append(k, v, *cache, *scale, table, torch.tensor(now).cuda(), cu_seqlens=offsets(n).cuda(), inv_freq=inv, q=q)
    seq, cu, cu_k = torch.tensor(total).cuda(), offsets(more).cuda(), offsets(total).cuda()
    kd, vd = ssd.ssd_kv8_read(*cache, *scale, table, seq, cu_k, sum(total))
    y, _ = ssd.ssd_attn_forward(q, kd, vd, cu, cu_seqlens_k=cu_k)
    last = q[[more[0] - 1, sum(more) - 1]].contiguous()
    one = ssd.ssd_kv8_decode(last, *cache, *scale, table, seq)
    torch.cuda.synchronize()
    # (the two see bf16 roundings of the held values and the values themselves: a few half steps of 2^-8 of values under 4)
    assert (one.float() - y[[more[0] - 1, sum(more) - 1]].float()).abs().max() < 4 * 4 * 2.0 ** -8


def test_graph_streams_and_workspaces():
    """Captured appends and decode steps of two caches with workspaces of their own, replayed on two streams at once as the
    caches grow, give the eager bits; so do workspaces of any contents, and calls on a given stream."""
    torch.manual_seed(1)
    n, H, Hk, D, page = 2, 8, 2, 64, 16
    state = []
    for i in range(2):
        (kc, vc), (ks, vs), table = pool(20 + i, [700, 333], page, Hk, D, "e4m3")
        state.append(dict(cache=[t.cuda() for t in (kc, vc, ks, vs)], table=table.cuda(), seq=torch.tensor([600, 300]).cuda(),
                          q=torch.randn((n, H, D), device="cuda").bfloat16(), k=torch.randn((n, Hk, D), device="cuda").bfloat16(),
                          v=torch.randn((n, Hk, D), device="cuda").bfloat16(), y=torch.empty((n, H, D), dtype=torch.bfloat16, device="cuda"),
                          inv=ssd.ssd_rotary_frequencies(D)[0].cuda(), q2=torch.empty((n, H, D), dtype=torch.bfloat16, device="cuda")))

    def step(st, y, **how):
        q = ssd.ssd_kv8_append(st["k"], st["v"], *st["cache"], st["table"], st["seq"], inv_freq=st["inv"], q=st["q"], q_out=st["q2"])
        return ssd.ssd_kv8_decode(q, *st["cache"], st["table"], st["seq"], y=y, **how)

    graphs = []
    for st in state:
        step(st, st["y"])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(st, st["y"])
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for st in state:
            st["seq"] += 1
            st["y"].zero_()
            for x in "qkv":
                st[x].normal_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for st in state:
            want = step(st, torch.empty_like(st["y"]))
            torch.cuda.synchronize()
            assert torch.equal(st["y"], want), i
    st = state[0]
    dims, _ = ssd.kv8._pages(torch.bfloat16, st["q"].device, H, *st["cache"], st["table"], st["seq"])
    need = ssd.ssd_kv8_decode_workspace_bytes(dims)
    assert need > 0
    for fill in (0x00, 0xFF):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        got = step(st, torch.empty_like(st["y"]), workspace=ws[:need])
        torch.cuda.synchronize()
        assert torch.equal(got, st["y"]) and torch.all(ws[need:] == fill)
    got = ssd.ssd_kv8_decode(st["q2"], *st["cache"], st["table"], st["seq"], stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(got, st["y"])


def test_far_into_a_large_cache():
    """Byte offsets past 2^32: the last pages of a cache give what the same rows give at its front."""
    pages, page, Hk, D, H, n = 280000, 64, 2, 128, 4, 130
    cache = [torch.empty((pages, page, Hk, D), dtype=torch.int8, device="cuda") for _ in "kv"]
    scale = [torch.empty((pages, page, Hk), device="cuda") for _ in "kv"]
    assert cache[0].numel() > 1 << 32
    d = make(4, n, n, H, Hk, D, "bf16")
    seq, cu = torch.tensor([n], device="cuda"), torch.tensor([0, n], device="cuda")
    got = []
    for row in ([pages - 1, pages - 2, pages - 5], [0, 2, 1]):
        table = torch.tensor([row], dtype=torch.int32, device="cuda")
        ssd.ssd_kv8_append(d["k"].cuda(), d["v"].cuda(), *cache, *scale, table, seq, cu)
        y = ssd.ssd_kv8_decode(d["q"][-1:].cuda(), *cache, *scale, table, seq)
        got.append((y, *ssd.ssd_kv8_read(*cache, *scale, table, seq, cu, n)))
    torch.cuda.synchronize()
    assert torch.equal(cache[0][pages - 1], cache[0][0]) and all(torch.equal(a, b) for a, b in zip(*got))


def test_binding_refusals():
    (kc, vc), (ks, vs), table = pool(1, [20, 30], 16, 2, 64, "int8")
    c = dict(k_cache=kc.cuda(), v_cache=vc.cuda(), k_scale=ks.cuda(), v_scale=vs.cuda(), block_table=table.cuda(), seq_lens=torch.tensor([20, 30]).cuda())
    q, k = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(k_cache=c["k_cache"].view(torch.uint8)), dict(v_cache=c["v_cache"].float()), dict(k_scale=c["k_scale"].bfloat16())):
        with pytest.raises(TypeError):
            ssd.ssd_kv8_decode(q, **dict(c, **kw))
        with pytest.raises(TypeError):
            ssd.ssd_kv8_append(k, k, **dict(c, **kw))
    for kw in (dict(k_scale=c["k_scale"][:, :, :1]), dict(v_scale=c["v_scale"].cpu()), dict(block_table=c["block_table"][:1]),
               dict(seq_lens=c["seq_lens"][:1]), dict(v_cache=c["v_cache"][:1])):
        with pytest.raises(ValueError):
            ssd.ssd_kv8_decode(q, **dict(c, **kw))
        with pytest.raises(ValueError):
            ssd.ssd_kv8_read(*dict(c, **kw).values(), None, 50)
    with pytest.raises(ValueError):
        ssd.ssd_kv8_append(k[:1], k[:1], **c)
    with pytest.raises(ValueError):
        ssd.ssd_kv8_append(k, k, **c, q=q[:, :3])
    with pytest.raises(TypeError):
        ssd.ssd_kv8_read(*c.values(), None, 50, dtype=torch.float16)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_kv8_read(*c.values(), None, 51)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_kv8_append(k, k, **c, inv_freq=torch.ones(4, device="cuda"))
    with pytest.raises(ssd.SSDError):
        ssd.ssd_kv8_decode(q, **dict(c, v_cache=c["v_cache"]), y=q)
