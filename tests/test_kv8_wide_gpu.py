"""The 8-bit decode step with eight waves a workgroup: the form of a serving batch over short caches."""
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from attn_helpers import DTYPE
from test_kv8_gpu import FORMS, decode_case

pytestmark = pytest.mark.gpu


def workspace(dtype, form, n, H, Hk, D, page, columns):
    page_of = torch.empty((4, page, Hk, D), dtype=FORMS[form], device="cuda")
    scale = torch.empty((4, page, Hk), device="cuda")
    dims, _ = ssd.kv8._pages(DTYPE[dtype], page_of.device, H, page_of, page_of, scale, scale,
                             torch.zeros((n, columns), dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda"))
    return ssd.ssd_kv8_decode_workspace_bytes(dims)


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("bias,cap,how", [("none", 0.0, {}), ("slopes", 0.0, {}), ("buckets", 0.0, dict(max_distance=60)), ("slopes", 30.0, {}),
                                          ("none", 4.0, {}), ("buckets", 4.0, {})])
def test_eight_waves(dtype, form, D, bias, cap, how):
    """33 sequences of up to 230 keys, four key heads of three query heads: 132 workgroups, whose eight waves have up to one block
    each.  Split in two they would need a workspace, so that none says that they are not."""
    lens, page, H, Hk = [(i * 53 + 7) % 231 for i in range(32)] + [230], 16, 12, 4
    assert workspace(dtype, form, len(lens), H, Hk, D, page, -(-max(lens) // page) + 1) == 0
    assert workspace(dtype, form, 8, H, Hk, D, page, -(-max(lens) // page) + 1) > 0
    decode_case(dtype, form, D, H, Hk, page, lens, bias=bias, cap=cap, seed=6, **how)


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,lens", [(128, [1024 - 31 * i for i in range(32)]), (64, [129] * 17 + [1000] * 15), (128, [128] * 16 + [3] * 16)])
def test_eight_waves_of_longer_caches(dtype, form, D, lens):
    """128 to 511 workgroups are not split up to 1024 keys, of either type and at every width; of 128 keys or fewer they are not for
    want of keys."""
    H, Hk, page = 8, 4, 32
    assert workspace(dtype, form, len(lens), H, Hk, D, page, 1024 // page) == 0
    assert workspace(dtype, form, len(lens), H, Hk, D, page, 1056 // page) > 0
    decode_case(dtype, form, D, H, Hk, page, lens, bias="slopes", seed=8)
