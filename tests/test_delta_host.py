"""The gated delta rule's C ABI and binding on a machine without a GPU: every declared function is exported, workspaces are
sized and bad arguments refused before any HIP call; and the fp64 model's own pins."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import oracle.delta as od
import ssd_chunked_scan_02_amd as ssd
from delta_helpers import f64, make, reference
from ssd_chunked_scan_02_amd.delta import DeltaDims

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssd_delta.h")
OK, INVALID, UNSUPPORTED, ALIGN = 0, -1, -2, -3
P = 1 << 20  # an aligned address that no refused call follows


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.library_path()):
        from ssd_chunked_scan_02_amd.build import build
        build()
    return ssd.load_library()


def test_header_and_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ssd_[a-z_]+)\s*\(", text)))
    assert names == ["ssd_delta_backward", "ssd_delta_backward_workspace_bytes", "ssd_delta_forward",
                     "ssd_delta_forward_workspace_bytes", "ssd_delta_step"]
    for n in names:
        assert hasattr(lib, n) and hasattr(ssd, n) and n in ssd.__all__


def _dims(**kw):
    d = dict(nseq=2, total=100, nheads=4, ngroups=2, keydim=64, valuedim=96, q_stride=0, k_stride=0, v_stride=0, scale=0.125, dtype=1)
    d.update(kw)
    return DeltaDims(**d)


BIG = 1 << 40
SHAPES = [
    (None, INVALID), (dict(nseq=-1), INVALID), (dict(total=-2), INVALID), (dict(total=1 << 31), INVALID), (dict(nheads=0), INVALID),
    (dict(nheads=5), INVALID), (dict(ngroups=0), INVALID), (dict(nheads=1 << 17), INVALID), (dict(dtype=2), INVALID),
    (dict(keydim=0), INVALID), (dict(valuedim=0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(keydim=96), UNSUPPORTED), (dict(keydim=256), UNSUPPORTED), (dict(valuedim=48), UNSUPPORTED), (dict(valuedim=288), UNSUPPORTED),
    (dict(nheads=1 << 16, valuedim=256), UNSUPPORTED), (dict(nseq=1 << 22, nheads=1024, total=0), UNSUPPORTED),
    (dict(total=1 << 30, nheads=1024, ngroups=1024, keydim=32, valuedim=32), UNSUPPORTED),
    (dict(q_stride=127), INVALID), (dict(k_stride=132), ALIGN), (dict(v_stride=1 << 24), INVALID),
    (dict(total=101), INVALID),  # not two equal sequences
]


@pytest.mark.parametrize("change,want", SHAPES, ids=range(len(SHAPES)))
def test_shape_refusals(lib, change, want):
    d = None if change is None else ctypes.byref(_dims(**change))
    assert lib.ssd_delta_forward(d, None, P, P, P, P, P, None, P + 64, None, P + 4096, BIG, None) == want
    outs = [P + 64 * i for i in range(1, 7)]
    assert lib.ssd_delta_backward(d, None, P, P, P, P, P, None, P, None, *outs, P + 4096, BIG, None) == want
    if change and ("total" in change):
        return
    assert lib.ssd_delta_step(d, P + 64, P, P, P, P, P, P + 128, None) == want


def test_forward_refusals(lib):
    d = _dims()
    need = ssd.ssd_delta_forward_workspace_bytes(d)

    def call(d=d, cu=None, q=P, k=P, v=P, log_a=P, beta=P, init=None, y=P + 64, final=None, ws=P + 4096, n=need):
        return lib.ssd_delta_forward(ctypes.byref(d), cu, q, k, v, log_a, beta, init, y, final, ws, n, None)

    for name in ("q", "k", "v", "log_a", "beta", "y", "ws"):
        assert call(**{name: None}) == INVALID, name
    for name in ("q", "k", "v", "log_a", "beta", "y", "ws", "init", "final"):
        assert call(**{name: P + 8}) == ALIGN, name
    assert call(cu=P + 4) == ALIGN
    assert call(n=need - 1) == INVALID
    for name in ("y", "final", "ws"):   # an output that is an input, or another output
        assert call(**{name: P}) == INVALID, name
    assert call(cu=2 * P, y=2 * P) == INVALID and call(init=2 * P, y=2 * P) == INVALID
    assert call(init=2 * P, ws=2 * P) == INVALID and call(final=P + 64) == INVALID
    assert call(d=_dims(nseq=0), ws=None, n=0, y=None) == OK
    assert call(d=_dims(total=0), ws=None, n=0, q=None, k=None, v=None, log_a=None, beta=None, y=None) == OK


def test_backward_refusals(lib):
    d = _dims()
    need = ssd.ssd_delta_backward_workspace_bytes(d)

    def call(d=d, cu=None, init=None, dfinal=None, dinit=None, ws=P + 4096, n=need, **kw):
        a = dict(q=P, k=P, v=P, log_a=P, beta=P, dy=P, **{x: P + 64 * (i + 1) for i, x in enumerate(("dq", "dk", "dv", "dlog_a", "dbeta"))})
        a.update(kw)
        return lib.ssd_delta_backward(ctypes.byref(d), cu, a["q"], a["k"], a["v"], a["log_a"], a["beta"], init, a["dy"], dfinal,
                                      a["dq"], a["dk"], a["dv"], a["dlog_a"], a["dbeta"], dinit, ws, n, None)

    for name in ("q", "k", "v", "log_a", "beta", "dy", "dq", "dk", "dv", "dlog_a", "dbeta", "ws"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: P + 8}) == ALIGN, name
    for name in ("init", "dfinal", "dinit"):
        assert call(**{name: P + 8}) == ALIGN, name
    for name in ("dq", "dk", "dv", "dlog_a", "dbeta", "dinit", "ws"):
        assert call(**{name: P}) == INVALID, name
    assert call(dinit=2 * P, dfinal=2 * P) == INVALID and call(dinit=P + 64) == INVALID
    assert call(n=need - 1) == INVALID
    assert call(d=_dims(nseq=0), ws=None, n=0) == OK


def test_step_refusals(lib):
    d = _dims(total=-7)  # (ignored)

    def call(d=d, state=P + 64, q=P, k=P, v=P, log_a=P, beta=P, y=P + 128):
        return lib.ssd_delta_step(ctypes.byref(d), state, q, k, v, log_a, beta, y, None)

    for name in ("state", "q", "k", "v", "log_a", "beta", "y"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: P + 8}) == ALIGN, name
    assert call(state=P) == INVALID and call(y=P) == INVALID and call(y=P + 64) == INVALID
    assert call(d=_dims(nseq=0)) == OK


def test_workspace_bytes():
    """bf16 operands of computed values are three terms: Z, and the scores in two where only y takes them; rows of K and Q."""
    slots = 100 // 64 + 2
    chunk = 64 * 64 * 2
    rows = 2 * slots * 2 * 64 * 64 * 2
    forward = slots * 4 * (3 + 2) * chunk + rows + slots * 4 * 5 * 64 * 4
    assert ssd.ssd_delta_forward_workspace_bytes(_dims()) == forward
    state, blocks = 64 * 96, 96 // 16
    backward = (slots * 4 * 12 * chunk + rows + slots * 4 * 5 * 64 * 4 + (slots + 2) * 4 * state * 4
                + 100 * 4 * 96 * 4 + slots * 4 * state * 2 + 3 * slots * 4 * blocks * 64 * 4 + (slots + 2) * 4 * blocks * 16)
    assert ssd.ssd_delta_backward_workspace_bytes(_dims()) == backward
    for bad in (dict(keydim=48), dict(nseq=0), dict(total=0), dict(dtype=7)):
        assert ssd.ssd_delta_forward_workspace_bytes(_dims(**bad)) == 0
        assert ssd.ssd_delta_backward_workspace_bytes(_dims(**bad)) == 0


def test_binding_refuses_cpu_tensors():
    d = make(1, [5], 2, 1, 32, 32, "fp32")
    args = [d[n] for n in ("q", "k", "v", "log_a", "beta")]
    with pytest.raises(ValueError):
        ssd.ssd_delta_forward(*args, cu_seqlens=d["cu"])
    with pytest.raises(ValueError):
        ssd.ssd_delta_backward(*args, d["dy"], cu_seqlens=d["cu"])
    with pytest.raises(ValueError):
        ssd.ssd_delta_step(d["init"], *[a[:1] for a in args])
    with pytest.raises(TypeError):
        ssd.ssd_delta_forward(*[a.half() for a in args], cu_seqlens=d["cu"])


# ------------------------------------------------------------------ the fp64 model

def test_model_by_hand():
    """Two tokens, one key dimension: S1 = b1 k1 v1, S2 = a2 S1 (1 - b2 k2^2) + b2 k2 v2."""
    q, k, v = np.array([[[2.0]], [[3.0]]]), np.array([[[0.5]], [[-1.0]]]), np.array([[[4.0]], [[6.0]]])
    la, b = np.log(np.array([[0.3], [0.5]])), np.array([[0.5], [0.25]])
    y, final = od.forward(q, k, v, la, b, np.array([0, 2]), 2.0)
    s1 = 0.5 * 0.5 * 4.0
    s2 = 0.5 * s1 * (1 - 0.25) + 0.25 * -1.0 * 6.0
    assert np.allclose(final.ravel(), s2) and np.allclose(y.ravel(), [2.0 * s1 * 2.0, 2.0 * s2 * 3.0])


def test_model_writes_and_recalls():
    """With beta 1 and no decay the state holds exactly the last value of a unit key; with beta 0 it only decays."""
    d = make(2, [9], 2, 1, 32, 32, "fp32", state=True)
    d["log_a"].zero_()
    d["beta"].fill_(1.0)
    d["q"] = d["k"]
    want = reference(d, scale=1.0, grads=False)
    assert np.allclose(want["y"], f64(d["v"]), atol=1e-5)  # (the keys' lengths are 1 to fp32)
    d["beta"].zero_()
    d["log_a"].fill_(-0.1)
    want = reference(d, grads=False)
    assert np.allclose(want["final"], f64(d["init"]) * math.exp(np.float32(-0.1) * 9.0))


def test_model_gradients_by_differences():
    """Every gradient against central differences along random directions."""
    d = make(5, [7, 0, 4], 4, 2, 5, 3, "fp32")
    names = ("q", "k", "v", "log_a", "beta", "init")
    x = {n: f64(d[n]) for n in names}
    dy, dfinal, cu = f64(d["dy"]), f64(d["dfinal"]), d["cu"].numpy()

    def value(z):
        y, final = od.forward(z["q"], z["k"], z["v"], z["log_a"], z["beta"], cu, 0.7, z["init"])
        return np.sum(y * dy) + np.sum(final * dfinal)

    grads = od.backward(x["q"], x["k"], x["v"], x["log_a"], x["beta"], cu, 0.7, dy, x["init"], dfinal)
    rng = np.random.default_rng(0)
    for n in names:
        step = rng.standard_normal(x[n].shape)
        h = 1e-5
        diff = (value(dict(x, **{n: x[n] + h * step})) - value(dict(x, **{n: x[n] - h * step}))) / (2 * h)
        assert np.isclose(diff, np.sum(grads["d" + n] * step), rtol=1e-7, atol=1e-7), n


def test_a_planted_mistake_is_seen():
    """The checks would notice a decay that is applied after the write, and a state that is not decayed for the error."""
    d = make(4, [40], 2, 2, 32, 32, "fp32")
    want = reference(d, grads=False)
    late = dict(d, log_a=torch.cat([d["log_a"][1:], torch.zeros(1, 2)]))
    assert np.linalg.norm(reference(late, grads=False)["y"] - want["y"]) > 1e-2 * np.linalg.norm(want["y"])
