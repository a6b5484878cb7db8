"""Writing strengths up to the largest declared, beta |k|^2 = 2, where a step reflects the state instead of forgetting."""
import numpy as np
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from delta_helpers import bound, cuda, f64, make, reference, sums_of_dlog_a
from test_delta_gpu import ARGS, run

pytestmark = pytest.mark.gpu


def growth():
    """How much larger the errors of a chunk may be than with keys apart.

    With one key for all tokens and beta = 2 the chunk's system is I + L B with ones on the diagonal and 2 below it, and its
    inverse has entries of 2 of either sign there.  A row's rounding errors are twice as large as for entries of one, and the inverse
    adds up those of 64 rows, each times 2: 2 sqrt(64) for independent ones."""
    return 2 * 2 * np.sqrt(64.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("keys", ["one", "close", "apart"])
@pytest.mark.parametrize("low", [1.0, 1.9, 2.0])
def test_strengths_up_to_two(dtype, keys, low):
    for H, G, N, P, lens in ((2, 1, 32, 32, [128]), (4, 2, 128, 64, [150, 64, 3]), (20, 10, 64, 64, [100, 70, 129, 64])):
        d = make(50 + N, lens, H, G, N, P, dtype, decay=0.01)
        if keys != "apart":
            d["k"][:] = d["k"][:1]
        if keys == "close":
            d["k"] = torch.nn.functional.normalize(d["k"].float() + 0.02 * torch.randn(d["k"].shape, generator=torch.Generator().manual_seed(2)), dim=-1).to(d["k"].dtype)
        d["beta"].uniform_(low, 2.0, generator=torch.Generator().manual_seed(1))
        # (a key of rounded elements is not of length one: the declared range is of beta |k|^2)
        k2 = d["k"].float().pow(2).sum(-1).repeat_interleave(H // G, 1)
        d["beta"] = torch.minimum(d["beta"] / k2, 2.0 / k2 * (1 - 2.0 ** -20))
        want, got = reference(d), run(cuda(d))
        for n, w in want.items():
            x = f64(got[n])
            assert np.all(np.isfinite(x)), n
            size = np.linalg.norm(w) + (sums_of_dlog_a(d, want) if n == "dlog_a" else 0.0)
            lim = bound(n, dtype, N, P)
            if not (dtype == "bf16" and n in ("y", "dq", "dk", "dv")):
                lim = lim * growth()
            off = np.linalg.norm(x - w) / size
            print("[gpu case] beta to 2 %s %s %s %g: %s %.3g of %.3g" % (dtype, (H, G, N, P), keys, low, n, off, lim), flush=True)
            assert off <= lim, (n, off, lim)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_reflecting_step(dtype):
    """The single token's step with beta |k|^2 = 2, over and over: the state is reflected, not lost, and no step lengthens an error."""
    n, H, G, N, P = 3, 2, 1, 64, 32
    d = make(60, [1] * n, H, G, N, P, dtype)
    k2 = d["k"].float().pow(2).sum(-1).repeat_interleave(H // G, 1)
    d["beta"], d["log_a"] = 2.0 / k2, torch.zeros_like(d["log_a"])
    d["v"] = torch.zeros_like(d["v"])
    g = cuda(d)
    state = g["init"].clone()
    for _ in range(64):
        ssd.ssd_delta_step(state, *[g[x] for x in ARGS])
    torch.cuda.synchronize()
    # an even number of reflections is none: 64 steps, each off by some sqrt(N) u and the rounding of beta, 2 u of twice the part along k
    off = float((state - g["init"]).norm() / g["init"].norm())
    assert off <= 64 * 12 * 2.0 ** -24 * np.sqrt(N), off
