"""What an 8-bit cache's decode step may round: its output, once.  The values that the pages stand for enter a bf16 call's
sums with weights of two bf16 terms, off by at most 2^-8 2^-8 = 2^-16 of each, and the rest is fp32.
"""
import numpy as np
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from attn_helpers import U, f64, make, offsets, reference, score_error, within
from test_kv8_gpu import gathered, pool, values

pytestmark = pytest.mark.gpu


def decode(seed, form, D, H, Hk, lens, page=16, bias="none", cap=0.0):
    n = len(lens)
    d = make(seed, n, 1, H, Hk, D, "bf16", bias=bias)
    (kc, vc), (ks, vs), table = pool(seed, lens, page, Hk, D, form)
    cache = [t.cuda() for t in (kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int64))]
    slopes = None if d["slopes"] is None else d["slopes"].cuda()
    y = ssd.ssd_kv8_decode(d["q"].cuda(), *cache, softcap=cap, slopes=slopes)
    torch.cuda.synchronize()
    d["k"], d["v"] = gathered(values(kc, ks), table, lens), gathered(values(vc, vs), table, lens)
    return d, y, cache


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("D,H,Hk", [(32, 3, 3), (64, 8, 2), (128, 4, 4)])
def test_one_key_is_read_back(form, D, H, Hk):
    """The softmax of one score is one: y is the value that ssd_kv8_read gives, before its rounding 2^-16 and an fp32's
    last bits away from it, so that it is off by half a step of 2^-8 and 2^-16 of that value."""
    lens = [1] * 19
    d, y, cache = decode(3, form, D, H, Hk, lens)
    want = np.repeat(f64(d["v"]), H // Hk, 1)
    within(f64(y), want, U["bf16"] * (1 + 2.0 ** -7) * np.abs(want) + 1e-30, "one key %s D%d" % (form, D))
    _, v = ssd.ssd_kv8_read(*cache, None, len(lens))
    torch.cuda.synchronize()
    read = v.cpu().float().repeat_interleave(H // Hk, 1)
    # (they differ where the value lies next to the middle between two steps, within 2^-16 of a step of 2^-7 at least: one in
    # a hundred on either side)
    assert (y.cpu().float() == read).float().mean() > 0.97


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("D,H,Hk,bias,cap", [(32, 3, 3, "none", 0.0), (64, 16, 2, "slopes", 0.0), (128, 8, 1, "none", 4.0), (64, 6, 6, "slopes", 4.0)])
def test_only_the_output_is_rounded(form, D, H, Hk, bias, cap):
    """Against the fp64 attention on the held values: half a step of the output, and no half steps of the weights."""
    lens = [2, 5, 17, 33, 300, 129, 1000]
    d, y, _ = decode(4, form, D, H, Hk, lens, bias=bias, cap=cap)
    ref = reference(d, cu=list(range(len(lens) + 1)), cu_k=offsets(lens).numpy(), cap=cap)
    es = score_error(ref, D, cap)[..., None]
    fine = 2.0 ** -16 + 2 * es + (max(lens) + 16) * 2.0 ** -24
    within(f64(y), ref["y"], 1.1 * (U["bf16"] * np.abs(ref["y"]) + fine * ref["y_abs"]) + 1e-30, "kv8 roundings %s D%d" % (form, D))
    # as a whole: the rounding of the exact result, and of the weights' terms
    exact = torch.from_numpy(ref["y"])
    once = float((exact.bfloat16().double() - exact).norm() / exact.norm())
    off = float((y.cpu().double() - exact).norm() / exact.norm())
    # (1.1: some 2000 elements' own scatter; the weights' second terms: 2^-16 of the values' 2-norm, which is that of y or a
    # few times it)
    assert off <= 1.1 * once + 8 * 2.0 ** -16, (off, once)
