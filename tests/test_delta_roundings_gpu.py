"""What the gated delta rule's backward pass may round in a bf16 call: its outputs, once."""
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from delta_helpers import U, bound, check, cuda, make, reference
from test_delta_gpu import ARGS, run

pytestmark = pytest.mark.gpu

CASES = [  # lens, H, G, N, P, state
    ([300, 41], 4, 2, 128, 64, True), ([200, 64, 7], 6, 2, 64, 32, False), ([513], 3, 3, 32, 96, True), ([130, 190], 2, 1, 128, 128, True),
    ([129, 200], 24, 8, 64, 64, True),
]


@pytest.mark.parametrize("lens,H,G,N,P,state", CASES, ids=range(len(CASES)))
def test_only_the_outputs_are_rounded(lens, H, G, N, P, state):
    """dq and dk are sums of products of computed values, whose operands have two bf16 terms: off by at most U^2 = 2^-16 of
    each, by less than U^2 of the 2-norm for five groups of them beside each other, as in delta_helpers; bound at six
    times that, beside the fp32 sums' own.  The rest is the rounding of the exact result, up to its scatter over thousands of elements."""
    d = make(41 + N, lens, H, G, N, P, "bf16", state=state)
    want = reference(d)
    got = run(cuda(d))
    check(got, want, d, "bf16", "roundings %s" % lens)
    for n in ("y", "dq", "dk", "dv"):
        exact = torch.from_numpy(want[n])
        once = float((exact.bfloat16().double() - exact).norm() / exact.norm())
        off = float((got[n].cpu().double() - exact).norm() / exact.norm())
        print("[gpu case] %s %s: %.3g, of which its own rounding %.3g" % (n, lens, off, once), flush=True)
        assert off <= 1.05 * once + 6 * U["bf16"] ** 2 + bound("final", "bf16", N, P), (n, off, once)


@pytest.mark.parametrize("P", [128, 160, 256])
def test_second_terms_in_a_workspace_of_nan(P):
    """Their place is that of operands no longer needed, or (160 and wider) one of their own: nothing of what was there is read,
    and what is behind the workspace is left."""
    d = make(77, [130, 0, 65, 20], 4, 2, 128, P, "bf16")
    g, want = cuda(d), reference(d)
    args = [g[x] for x in ARGS]
    size = ssd.ssd_delta_backward_workspace_bytes(ssd.delta._dims(*args, g["cu"], None, 3))
    got = []
    for fill in (0xFF, 0x7F):
        ws = torch.full((size + 64,), fill, dtype=torch.uint8, device="cuda")
        got.append(ssd.ssd_delta_backward(*args, g["dy"], cu_seqlens=g["cu"], init_state=g["init"], dfinal=g["dfinal"], want_dinit=True,
                                          workspace=ws[:size]))
        torch.cuda.synchronize()
        assert torch.all(ws[size:] == fill)
    assert all(torch.equal(got[0][n], got[1][n]) for n in got[0])
    check(got[0], want, d, "bf16", "second terms P%d" % P)
    for n in ("dq", "dk"):
        exact = torch.from_numpy(want[n])
        once = float((exact.bfloat16().double() - exact).norm() / exact.norm())
        off = float((got[0][n].cpu().double() - exact).norm() / exact.norm())
        assert off <= 1.05 * once + 6 * U["bf16"] ** 2 + bound("final", "bf16", 128, P), (n, off, once)
