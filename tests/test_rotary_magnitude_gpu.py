"""A rotation with a magnitude, trained by ssd_rotate, and served from a cache whose append has none."""
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd

pytestmark = pytest.mark.gpu


def place(n, page):
    return torch.arange(-(-n // page), dtype=torch.int32, device="cuda")[None].flip(1).contiguous()


@pytest.mark.parametrize("interleaved", [False, True])
def test_square_of_the_magnitude_in_the_scale(interleaved):
    """All of a head rotated: scores are m^2 times those of turns alone.  fp32: each way rounds its turns, products and scores to about
    1e-6 of y's values, of order one."""
    L, H, Hk, D, page = 75, 4, 2, 64, 16
    inv, m = ssd.ssd_rotary_frequencies(D, factor=8.0, trained=64)
    inv = inv.cuda()
    assert m > 1.2
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((1, L, h, D), device="cuda", generator=g) for h in (H, Hk, Hk))
    qr, kr = ssd.ssd_rotate(q, inv, k=k, magnitude=m, interleaved=interleaved)
    y, _ = ssd.ssd_attn_forward(qr, kr, v)
    table, seq, cu = place(L, page), torch.tensor([L], device="cuda"), torch.tensor([0, L], device="cuda")
    cache = [torch.zeros((table.numel(), page, Hk, D), device="cuda") for _ in "kv"]
    qt = ssd.ssd_kv_append(k[0], v[0], *cache, table, seq, cu_seqlens=cu, inv_freq=inv, interleaved=interleaved, q=q[0])
    one = ssd.ssd_attn_decode(qt[-1:].contiguous(), *cache, table, seq, scale=m * m * D ** -0.5)
    torch.cuda.synchronize()
    assert (one[0] - y[0, -1]).abs().max() < 1e-5


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_part_of_a_head_rotated_before_the_append(dtype):
    """Where a part of a head stays as it is: ssd_rotate, and an append without frequencies.  Read back, each element is off by the form's
    step of the head's largest (int8) or of itself (e4m3)."""
    L, Hk, D, page, rot, m = 40, 3, 64, 16, 16, 1.3
    inv = ssd.ssd_rotary_frequencies(2 * rot)[0].cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((1, L, Hk, D), device="cuda", generator=g) for _ in "kv")
    kr, _ = ssd.ssd_rotate(k, inv, magnitude=m)
    assert torch.equal(kr[..., 2 * rot:], k[..., 2 * rot:])
    table, seq, cu = place(L, page), torch.tensor([L], device="cuda"), torch.tensor([0, L], device="cuda")
    cache = [torch.zeros((table.numel(), page, Hk, D), dtype=torch.uint8, device="cuda").view(dtype) for _ in "kv"]
    scale = [torch.zeros((table.numel(), page, Hk), device="cuda") for _ in "kv"]
    ssd.ssd_kv8_append(kr[0], v[0], *cache, *scale, table, seq, cu_seqlens=cu)
    kd, vd = ssd.ssd_kv8_read(*cache, *scale, table, seq, cu, L, dtype=torch.float32)
    torch.cuda.synchronize()
    for got, want in ((kd, kr[0]), (vd, v[0])):
        top = want.abs().amax(-1, keepdim=True)
        step = top / 254 if dtype is torch.int8 else torch.maximum(want.abs() / 16, top / 448 / 1024)
        assert torch.all((got - want).abs() <= step * 1.0001 + 1e-6)
