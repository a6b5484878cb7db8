"""What the 8-bit cache holds of values next to the smallest that fp32 has, where a scale itself has few bits."""
import numpy as np
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from test_kv8_gpu import FORMS, TOP

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_off_by_the_declared_step(form):
    """Off by scale / 2 at most (int8), 2^-4 of the value or scale 2^-10 (e4m3), at every magnitude; only zeros have a scale of zero.
    The largest value may lie 2^-24 past the form's own largest (the scale's two roundings)."""
    g = torch.Generator().manual_seed(1)
    tops = [2.0 ** -149 * m for m in (1, 2, 63, 64, 95, 100, 127, 190, 191, 300, 448, 670, 671, 1000, 5000)]
    tops += [2.0 ** e * f for e in (-140, -130, -127, -126, -120, -119, -118, -117, -100, 0) for f in (1.0, 1.37)]
    Hk, D, page = len(tops), 64, 16
    x = (torch.rand((1, Hk, D), generator=g, dtype=torch.float64) * 2 - 1) * torch.tensor(tops, dtype=torch.float64)[None, :, None]
    x[0, :, 5] = -torch.tensor(tops, dtype=torch.float64)
    x = x.float()
    cache = [torch.zeros((1, page, Hk, D), dtype=torch.uint8, device="cuda").view(FORMS[form]) for _ in "kv"]
    scale = [torch.zeros((1, page, Hk), device="cuda") for _ in "kv"]
    ssd.ssd_kv8_append(x.cuda(), x.cuda(), *cache, *scale, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([1], device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(cache[0].view(torch.uint8), cache[1].view(torch.uint8)) and torch.equal(*scale)
    sc = scale[0][0, 0].cpu().double().numpy()[:, None]
    held = cache[0][0, 0].cpu().float().double().numpy() * sc
    want = x[0].double().numpy()
    assert np.all(sc > 0)
    step = sc / 2 if form == "int8" else np.maximum(2.0 ** -4 * np.abs(want), sc * 2.0 ** -10)
    off = np.abs(held - want) - step * (1 + 2.0 ** -20) - 2.0 ** -23 * np.abs(want)
    assert np.all(off <= 0), [(tops[h], float(np.max(off[h]) / sc[h, 0])) for h in range(Hk) if np.max(off[h]) > 0]
    normal = sc[:, 0] >= 2.0 ** -126  # there a scale is the formula's to the bit
    inv = np.float32(1.0 / TOP[form])
    assert np.array_equal(sc[normal, 0], (np.abs(x[0].numpy()).max(-1) * inv).astype(np.float64)[normal])
