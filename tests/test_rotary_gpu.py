"""GPU tests of rotary positions: the rotation against complex numbers in fp64, and its gradient."""
import numpy as np
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from attn_helpers import DTYPE, f64, make, offsets, within
from test_attention_cache_gpu import _angle_bound

pytestmark = pytest.mark.gpu


def turned(x, pos, inv_freq, interleaved, m, sign):
    """x [T, heads, D] in fp64."""
    x, pairs = f64(x), len(inv_freq)
    w = np.exp(1j * sign * np.outer(pos, f64(inv_freq)))[:, None]
    y = x.copy()
    if interleaved:
        z = (x[..., 0:2 * pairs:2] + 1j * x[..., 1:2 * pairs:2]) * w * m
        y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2] = z.real, z.imag
    else:
        z = (x[..., :pairs] + 1j * x[..., pairs:2 * pairs]) * w * m
        y[..., :pairs], y[..., pairs:2 * pairs] = z.real, z.imag
    return y


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,H,Hk,pairs,interleaved", [(32, 3, 3, 16, False), (64, 8, 2, 32, True), (128, 4, 4, 64, False), (128, 5, 1, 8, True),
                                                      (64, 2, 3, 16, False), (32, 1, 1, 0, False)])
@pytest.mark.parametrize("inverse", [False, True])
def test_against_complex_numbers(dtype, D, H, Hk, pairs, interleaved, inverse):
    """Packed sequences that start anywhere, far positions among them; rows of no sequence are left."""
    lens, start = [1, 0, 70, 33], [0, 5, 1_000_000, 100]
    lead, T = 3, 3 + sum(lens) + 2
    d = make(D + H, T, T, H, Hk, D, dtype)
    inv = (10000.0 ** (-torch.arange(max(pairs, 1), dtype=torch.float64) / max(pairs, 1))).float()[:pairs]
    cu = offsets(lens) + lead
    out = [torch.full((T, h, D), 7.0, dtype=DTYPE[dtype], device="cuda") for h in (H, Hk)]
    m = 1.25
    q, k = ssd.ssd_rotate(d["q"].cuda(), inv.cuda(), cu_seqlens=cu.cuda(), start=torch.tensor(start).cuda(), k=d["k"].cuda(),
                          interleaved=interleaved, magnitude=m, inverse=inverse, q_out=out[0], k_out=out[1])
    torch.cuda.synchronize()
    assert q is out[0] and k is out[1]
    pos = np.concatenate([np.arange(n) + s for n, s in zip(lens, start)])
    for got, x in ((q, d["q"]), (k, d["k"])):
        want = turned(x[lead:-2], pos, inv, interleaved, m, -1.0 if inverse else 1.0)
        within(f64(got)[lead:-2], want, _angle_bound(want, dtype), "rotate %s D%d %d pairs" % (dtype, D, pairs))
        assert torch.all(got[:lead] == 7.0) and torch.all(got[-2:] == 7.0)
        assert torch.equal(got[lead:-2, :, 2 * pairs:].cpu(), x[lead:-2, :, 2 * pairs:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layouts(dtype):
    """[B, L, ...] is the packed batch of equal sequences; views of a projection are read where they lie; q alone."""
    B, L, H, Hk, D = 3, 21, 4, 2, 64
    d = make(2, B * L, B * L, H, Hk, D, dtype)
    inv = ssd.ssd_rotary_frequencies(D)[0].cuda()
    q, k = d["q"].cuda(), d["k"].cuda()
    want = ssd.ssd_rotate(q, inv, cu_seqlens=offsets([L] * B).cuda(), k=k)
    wide = torch.full((B * L, (H + Hk) * D + 16), float("nan"), dtype=DTYPE[dtype], device="cuda")
    wide[:, :H * D], wide[:, H * D:(H + Hk) * D] = q.flatten(1), k.flatten(1)
    vq, vk = wide[:, :H * D].unflatten(1, (H, D)), wide[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    got = ssd.ssd_rotate(vq.unflatten(0, (B, L)), inv, k=vk.unflatten(0, (B, L)))
    one, none = ssd.ssd_rotate(vq, inv, cu_seqlens=offsets([L] * B).cuda())
    torch.cuda.synchronize()
    assert none is None and torch.equal(one, want[0])
    assert torch.equal(got[0].flatten(0, 1), want[0]) and torch.equal(got[1].flatten(0, 1), want[1])


def test_gradient():
    """<g, R x> = <R' g, x> with R' the inverse call (fp32: to the sums' rounding), and differences agree."""
    d = make(3, 50, 50, 4, 2, 64, "fp32")
    inv, m = ssd.ssd_rotary_frequencies(64, factor=4.0)
    assert m > 1.1
    q, g = d["q"].cuda(), torch.randn((50, 4, 64), device="cuda")
    cu = offsets([20, 30]).cuda()
    how = dict(inv_freq=inv.cuda(), cu_seqlens=cu, magnitude=m, interleaved=True)
    y, _ = ssd.ssd_rotate(q, **how)
    back, _ = ssd.ssd_rotate(g, inverse=True, **how)
    a, b = (y.double() * g.double()).sum(), (back.double() * q.double()).sum()
    size = y.double().norm() * g.double().norm()
    assert abs(a - b) <= 16 * 2.0 ** -24 * size
    step = torch.randn_like(q)
    diff = ((ssd.ssd_rotate(q + step, **how)[0].double() - ssd.ssd_rotate(q - step, **how)[0].double()) / 2 * g.double()).sum()
    assert abs(diff - (back.double() * step.double()).sum()) <= 64 * 2.0 ** -24 * size * 2


def test_matches_the_append():
    """The rotation of training is the one that ssd_kv_append writes into a cache."""
    H, Hk, D, n, page = 4, 2, 64, 37, 16
    d = make(5, n, n, H, Hk, D, "bf16")
    inv = ssd.ssd_rotary_frequencies(D)[0].cuda()
    cache = [torch.zeros((3, page, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    table, seq, cu = torch.tensor([[2, 0, 1]], dtype=torch.int32).cuda(), torch.tensor([n]).cuda(), torch.tensor([0, n]).cuda()
    q1 = ssd.ssd_kv_append(d["k"].cuda(), d["v"].cuda(), *cache, table, seq, cu, inv_freq=inv, q=d["q"].cuda())
    q2, k2 = ssd.ssd_rotate(d["q"].cuda(), inv, cu_seqlens=cu, k=d["k"].cuda())
    torch.cuda.synchronize()
    k1 = cache[0][[2, 0, 1]].flatten(0, 1)[:n]
    # (rounded once each, from fp32 values some units of 2^-24 apart: a step of bf16 where those lie across a border)
    for a, b in ((q1, q2), (k1, k2)):
        off = (a.float() - b.float()).abs()
        assert torch.all(off <= 2.0 ** -7 * b.float().abs() + 1e-6) and (off > 0).float().mean() < 1e-3


def test_graph_and_stream():
    d = make(6, 300, 300, 4, 2, 64, "bf16")
    q, inv, cu = d["q"].cuda(), ssd.ssd_rotary_frequencies(64)[0].cuda(), offsets([100, 200]).cuda()
    out = torch.empty_like(q)
    ssd.ssd_rotate(q, inv, cu_seqlens=cu, q_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_rotate(q, inv, cu_seqlens=cu, q_out=out)
    s = torch.cuda.Stream()
    for i, lens in enumerate(([100, 200], [0, 300], [299, 1])):
        q.normal_()
        cu.copy_(offsets(lens))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want, _ = ssd.ssd_rotate(q, inv, cu_seqlens=cu)
        other, _ = ssd.ssd_rotate(q, inv, cu_seqlens=cu, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(other, want), i


def test_malformed_offsets_stay_inside():
    q = torch.randn((300, 2, 32), device="cuda")
    inv = ssd.ssd_rotary_frequencies(32)[0].cuda()
    for bad in ([0, 500, -7, 300], [200, 100, 300, 250], [-1, -1, 10 ** 12, 5]):
        out = torch.full((400, 2, 32), 3.0, device="cuda")
        ssd.ssd_rotate(q, inv, cu_seqlens=torch.tensor(bad).cuda(), q_out=out[:300])
        torch.cuda.synchronize()
        assert torch.all(out[300:] == 3.0)


def test_binding_refusals():
    q, inv = torch.zeros((10, 2, 32), device="cuda"), torch.ones(16, device="cuda")
    cu = torch.tensor([0, 10]).cuda()
    for kw in (dict(k=q[:5]), dict(k=torch.zeros((10, 2, 64), device="cuda")), dict(k_out=q), dict(q_out=q[:, :1]), dict(start=cu),
               dict(cu_seqlens=cu.int()), dict(cu_seqlens=None)):
        with pytest.raises(ValueError):
            ssd.ssd_rotate(q, inv, **dict(dict(cu_seqlens=cu), **kw))
    with pytest.raises(TypeError):
        ssd.ssd_rotate(q.half(), inv, cu_seqlens=cu)
    with pytest.raises(TypeError):
        ssd.ssd_rotate(q, inv.double(), cu_seqlens=cu)
    for bad in (inv[:4].contiguous(), torch.ones(24, device="cuda")):
        with pytest.raises(ssd.SSDError):
            ssd.ssd_rotate(q, bad, cu_seqlens=cu)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_rotate(q, inv, cu_seqlens=cu, q_out=q)
