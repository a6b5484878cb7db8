"""The attention layer at its edges, on the GPU: calls that the documentation allows and an ordinary run does not make."""
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd

pytestmark = pytest.mark.gpu


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
