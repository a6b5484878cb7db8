"""Every gradient of the delta rule's kernels along itself, against central differences of the forward pass in the kernels."""
import numpy as np
import pytest
import torch

import ssd_chunked_scan_02_amd as ssd
from delta_helpers import cuda, make
from test_delta_gpu import ARGS, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,N,P,lens", [(2, 1, 32, 32, [100]), (4, 2, 64, 32, [70, 0, 65]), (2, 2, 128, 64, [150])])
def test_along_the_gradient(H, G, N, P, lens):
    """The direction is the gradient's own, of length one a value (a tenth for the gates), so that the quotient is its 2-norm and
    many times what a random direction has.

    Tolerance: the third derivative's part of a central difference, 2 in 100 of the quotient at h = 2e-3; and the rounding of the two
    values, sums of dy y that are off by 12 u sqrt(2 N + 128 + P) of their 2-norm at most (delta_helpers), over h."""
    d = make(19, lens, H, G, N, P, "fp32", decay=0.3)
    g = cuda(d)
    grads = run(g)

    def value(z):
        y, final = ssd.ssd_delta_forward(*[z[n] for n in ARGS], cu_seqlens=z["cu"], init_state=z["init"], final_state=True)
        return float((y.double() * g["dy"].double()).sum() + (final.double() * g["dfinal"].double()).sum())

    h = 2e-3
    size = float(g["dy"].double().norm() * grads["y"].double().norm() / np.sqrt(grads["y"].numel())
                 + g["dfinal"].double().norm() * grads["final"].double().norm() / np.sqrt(grads["final"].numel()))
    noise = 12 * 2.0 ** -24 * np.sqrt(2 * N + 128 + P) * size / h
    for n in ARGS + ("init",):
        slope = grads["d" + n].double()
        step = (slope / slope.pow(2).mean().sqrt()).float()
        if n in ("log_a", "beta"):
            step = step * 0.1
        along = float((slope * step.double()).sum())
        diff = (value(dict(g, **{n: g[n] + h * step})) - value(dict(g, **{n: g[n] - h * step}))) / (2 * h)
        allowed = 0.02 * abs(along) + noise
        print("[gpu case] along %s: %.6g by differences, %.6g, allowed %.2g" % (n, diff, along, allowed), flush=True)
        assert abs(along) > 20 * allowed, (n, along, allowed)
        assert abs(diff - along) <= allowed, (n, diff, along, allowed)
