"""The gated delta rule on the GPU against the fp64 recurrence, token by token (oracle/delta.py): both passes and the
step, over widths, groups, lengths and types; what the calls leave alone; strides, streams, graphs and workspaces."""
import numpy as np
import pytest
import torch

import oracle.delta as od
import ssd_chunked_scan_02_amd as ssd
from delta_helpers import DTYPE, bound, check, cuda, f64, make, reference

pytestmark = pytest.mark.gpu
ARGS = ("q", "k", "v", "log_a", "beta")


def run(g, grads=True, **how):
    args = [g[n] for n in ARGS]
    y, final = ssd.ssd_delta_forward(*args, cu_seqlens=g["cu"], init_state=g["init"], final_state=True, **how)
    got = dict(y=y, final=final)
    if grads:
        got.update(ssd.ssd_delta_backward(*args, g["dy"], cu_seqlens=g["cu"], init_state=g["init"], dfinal=g["dfinal"],
                                          want_dinit=True, **how))
    torch.cuda.synchronize()
    return got


CASES = [  # lens, H, G, N, P
    ([1], 1, 1, 32, 32), ([64], 2, 1, 64, 64), ([65, 63], 2, 2, 128, 64), ([200], 3, 1, 64, 32), ([130, 1, 0, 77], 4, 2, 128, 128),
    ([0, 0, 33, 0], 2, 2, 32, 96), ([15, 16, 17, 128], 6, 3, 32, 64), ([257], 2, 1, 128, 256), ([129, 191], 8, 2, 64, 160), ([48], 5, 5, 128, 32),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("lens,H,G,N,P", CASES, ids=range(len(CASES)))
def test_against_the_recurrence(lens, H, G, N, P, state, dtype):
    d = make(H + N, lens, H, G, N, P, dtype, state=state)
    want = reference(d)
    check(run(cuda(d)), want, d, dtype, "delta %s %s" % (lens, dtype))


MANY = [  # lens, H, G, N, P: enough heads and sequences for walks of 32 columns
    ([130, 1, 0, 77, 64, 3, 200], 12, 4, 128, 64), ([257, 40, 64], 16, 16, 128, 96), ([65, 0, 190], 20, 5, 64, 96), ([129, 128], 40, 8, 32, 64),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("lens,H,G,N,P", MANY, ids=range(len(MANY)))
def test_many_heads(lens, H, G, N, P, state, dtype):
    """As above, in a workspace of NaN, twice with the same bits."""
    d = make(31 + N, lens, H, G, N, P, dtype, state=state)
    g = cuda(d)
    assert len(lens) * H * P // 16 > 256
    got = run(g)
    check(got, reference(d), d, dtype, "many heads %s %s" % (dtype, (lens, H, G, N, P, state)))
    args = [g[x] for x in ARGS]
    size = ssd.ssd_delta_backward_workspace_bytes(ssd.delta._dims(*args, g["cu"], None, 3))
    again = ssd.ssd_delta_backward(*args, g["dy"], cu_seqlens=g["cu"], init_state=g["init"], dfinal=g["dfinal"], want_dinit=True,
                                   workspace=torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert all(torch.equal(again[n], got[n]) for n in again)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_batched_layout(dtype):
    """[B, T, ...] without offsets is the packed batch of equal sequences, bit for bit; a scale of the caller's."""
    d = make(8, [70, 70, 70], 4, 2, 64, 64, dtype)
    g = cuda(d)
    want = run(g, scale=0.7)
    check(want, reference(d, scale=0.7), d, dtype, "scale")
    b = {n: (t.unflatten(0, (3, 70)) if n in ARGS + ("dy",) else t) for n, t in g.items()}
    b["cu"] = None
    got = run(b, scale=0.7)
    for n in want:
        assert torch.equal(got[n].reshape(want[n].shape), want[n]), n


@pytest.mark.parametrize("decay", [0.0, 30.0])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_no_decay_and_strong_decay(dtype, decay):
    """Sums of log a over a chunk that are zero, or so far out that fp32 would lose what its differences are made of."""
    d = make(3, [150], 2, 1, 64, 32, dtype, decay=decay)
    check(run(cuda(d)), reference(d), d, dtype, "decay %g" % decay)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_resets(dtype):
    """log a of -1e30 and of minus infinity in the middle of a chunk forget everything before, and nothing after."""
    d = make(6, [90, 100], 2, 2, 32, 64, dtype)
    for t, x in ((17, -1e30), (63, float("-inf")), (64, -200.0), (140, float("-inf"))):
        d["log_a"][t] = x
    want = reference(dict(d, log_a=d["log_a"].clamp(min=-800.0)))  # (exp of either is zero; 64 bits have no use for infinities)
    got = run(cuda(d))
    check(got, want, d, dtype, "resets")
    for t in (17, 63, 64, 140):
        assert torch.all(got["dlog_a"][t] == 0)


def test_correlated_keys():
    """Every key the same: the triangular system of a chunk is as far from the identity as unit keys make it."""
    for dtype in ("fp32", "bf16"):
        d = make(9, [128], 2, 1, 32, 32, dtype, decay=0.01)
        d["k"][:] = d["k"][:1]
        d["beta"].uniform_(0.5, 1.0, generator=torch.Generator().manual_seed(1))
        check(run(cuda(d)), reference(d), d, dtype, "one key %s" % dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_step_continues_a_prompt(dtype):
    """A prompt by the chunked pass, then tokens one by one: the recurrence over all of them."""
    H, G, N, P, n, L, more = 4, 2, 64, 64, 3, 77, 6
    d = make(2, [L + more] * n, H, G, N, P, dtype)
    want = reference(d, grads=False)
    g = cuda(d)
    seq = {x: g[x].unflatten(0, (n, L + more)) for x in ARGS}
    y0, state = ssd.ssd_delta_forward(*[seq[x][:, :L].contiguous() for x in ARGS], init_state=g["init"], final_state=True)
    ys = [y0]
    for t in range(L, L + more):
        ys.append(ssd.ssd_delta_step(state, *[seq[x][:, t].contiguous() for x in ARGS])[:, None])
    got = dict(y=torch.cat(ys, 1).flatten(0, 1), final=state)
    torch.cuda.synchronize()
    check(got, want, d, dtype, "prompt and steps")


STEPS = [(1, 1, 1, 32, 32), (5, 6, 2, 64, 96), (3, 4, 4, 128, 256), (17, 3, 1, 128, 128)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n,H,G,N,P", STEPS, ids=range(len(STEPS)))
def test_step(n, H, G, N, P, dtype):
    d = make(n, [1] * n, H, G, N, P, dtype)
    y, final = od.step(f64(d["init"]), *[f64(d[x]) for x in ARGS], N ** -0.5)
    g = cuda(d)
    got = dict(y=ssd.ssd_delta_step(g["init"], *[g[x] for x in ARGS]), final=g["init"])
    torch.cuda.synchronize()
    check(got, dict(y=y, final=final), d, dtype, "step")


def test_a_state_is_handed_on_in_place():
    """final_state may be init_state itself, and a sequence in parts gives what it gives whole."""
    d = cuda(make(11, [150, 40], 4, 2, 128, 64, "bf16"))
    args = [d[x] for x in ARGS]
    y, final = ssd.ssd_delta_forward(*args, cu_seqlens=d["cu"], init_state=d["init"], final_state=True)
    state, n = d["init"].clone(), 0
    for cut in ([[0, 64], [150, 170]], [[64, 150], [170, 190]]):
        cu = torch.tensor([0, cut[0][1] - cut[0][0], cut[0][1] - cut[0][0] + cut[1][1] - cut[1][0]], device="cuda")
        part = [torch.cat([a[lo:hi] for lo, hi in cut]) for a in args]
        y2, same = ssd.ssd_delta_forward(*part, cu_seqlens=cu, init_state=state, final_state=state)
        assert same is state
        whole = torch.cat([y[lo:hi] for lo, hi in cut])
        torch.cuda.synchronize()
        assert (y2.float() - whole.float()).norm() <= 2 * bound("y", "bf16", 128, 64) * whole.float().norm()
    assert (state - final).norm() <= 2 * bound("final", "bf16", 128, 64) * final.norm()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_views_of_a_projection(dtype):
    """q, k and v as views of wider rows are read where they lie: the bits of dense copies."""
    H, G, N, P = 4, 2, 64, 64
    d = make(12, [70, 33], H, G, N, P, dtype)
    g = cuda(d)
    T = g["q"].shape[0]
    wide = torch.full((T, 2 * G * N + H * P + 64), float("nan"), dtype=DTYPE[dtype], device="cuda")
    at, view = 16, {}
    for x, heads, dim in (("q", G, N), ("k", G, N), ("v", H, P)):
        view[x] = wide[:, at:at + heads * dim].unflatten(1, (heads, dim))
        view[x].copy_(g[x])
        at += heads * dim + 16
    want, got = run(g), run(dict(g, **view))
    for n in want:
        assert torch.equal(want[n], got[n]), n
    one = {x: t[:5] for x, t in dict(g, **view).items() if x in ARGS}
    state = [torch.ones((5, H, N, P), device="cuda") for _ in range(2)]
    a = ssd.ssd_delta_step(state[0], *[one[x] for x in ARGS])
    b = ssd.ssd_delta_step(state[1], *[g[x][:5] for x in ARGS])
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(*state)


def test_what_is_left_alone():
    """Rows of no sequence are neither read into anything nor written; NaN and infinities stay in their sequence, and
    those of values, gates and states in their head."""
    d = make(13, [40, 70, 20], 4, 2, 64, 32, "bf16")
    g = cuda(d)
    want = run(g)
    lead, tail = 7, 9
    pad = lambda t, x: torch.cat([torch.full((lead,) + t.shape[1:], x, dtype=t.dtype, device="cuda"), t,  # noqa: E731
                                  torch.full((tail,) + t.shape[1:], x, dtype=t.dtype, device="cuda")])
    args = [pad(g[x], float("nan")) for x in ARGS]
    cu = g["cu"] + lead
    y = torch.full_like(args[2], 3.0)
    ssd.ssd_delta_forward(*args, cu_seqlens=cu, init_state=g["init"], y=y)
    torch.cuda.synchronize()
    assert torch.equal(y[lead:-tail], want["y"]) and torch.all(y[:lead] == 3.0) and torch.all(y[-tail:] == 3.0)
    back = ssd.ssd_delta_backward(*args, pad(g["dy"], float("nan")), cu_seqlens=cu, init_state=g["init"], dfinal=g["dfinal"])
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv", "dlog_a", "dbeta"):
        assert torch.equal(back[n][lead:-tail], want[n]), n
    assert torch.equal(back["dinit"], want["dinit"])

    for x, where in (("v", (50, 1)), ("log_a", (50, 1)), ("beta", (109, 1)), ("init", (1, 1)), ("k", (50, 0)), ("q", (45, 0))):
        bad = dict(g, **{x: g[x].clone()})
        bad[x][where] = float("nan")
        got = run(bad)
        others = [0, 2, 3] if x not in "kq" else [2, 3]
        for n in ("y", "dv", "dlog_a", "dbeta"):
            assert torch.equal(got[n][:40], want[n][:40]) and torch.equal(got[n][110:], want[n][110:]), (x, n)
            assert torch.equal(got[n][40:110][:, others], want[n][40:110][:, others]), (x, n)
        for n in ("final", "dinit"):
            assert torch.equal(got[n][[0, 2]], want[n][[0, 2]]) and torch.equal(got[n][1][others], want[n][1][others]), (x, n)
        for n in ("dq", "dk"):
            assert torch.equal(got[n][:40], want[n][:40]) and torch.equal(got[n][40:110, 1], want[n][40:110, 1]), (x, n)


def test_malformed_offsets_stay_inside():
    """Offsets that fall, repeat, or lie outside the axis give some outputs and touch nothing else."""
    d = cuda(make(14, [150, 50, 100], 2, 1, 64, 32, "bf16"))
    args = [d[x] for x in ARGS]
    for bad in ([0, 500, -7, 300], [200, 100, 300, 250], [-1, -1, 10 ** 12, 5], [300, 300, 300, 300]):
        cu = torch.tensor(bad, dtype=torch.int64, device="cuda")
        y = torch.full((556, 2, 32), 3.0, dtype=torch.bfloat16, device="cuda")
        ssd.ssd_delta_forward(*args, cu_seqlens=cu, y=y[:300])
        need = ssd.ssd_delta_backward_workspace_bytes(ssd.delta._dims(*args, cu, None, 3))
        ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
        ssd.ssd_delta_backward(*args, d["dy"], cu_seqlens=cu, workspace=ws[:need])
        torch.cuda.synchronize()
        assert torch.all(y[300:] == 3.0) and torch.all(ws[need:] == 0), bad


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_workspace_contents_and_repeats(dtype):
    d = cuda(make(15, [100, 3, 130], 6, 2, 64, 64, dtype))
    args = [d[x] for x in ARGS]
    dims = ssd.delta._dims(*args, d["cu"], None, 3)
    sizes = ssd.ssd_delta_forward_workspace_bytes(dims), ssd.ssd_delta_backward_workspace_bytes(dims)
    got = []
    for fill in (0x00, 0xFF, 0x7F):
        ws = [torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda") for n in sizes]
        y, final = ssd.ssd_delta_forward(*args, cu_seqlens=d["cu"], init_state=d["init"], final_state=True, workspace=ws[0][:sizes[0]])
        back = ssd.ssd_delta_backward(*args, d["dy"], cu_seqlens=d["cu"], init_state=d["init"], dfinal=d["dfinal"], workspace=ws[1][:sizes[1]])
        torch.cuda.synchronize()
        assert all(torch.all(w[n:] == fill) for w, n in zip(ws, sizes))
        got.append(dict(back, y=y, final=final))
    for n in got[0]:
        assert torch.equal(got[0][n], got[1][n]) and torch.equal(got[0][n], got[2][n]), n


def test_training_step_in_a_graph():
    """A captured forward and backward, replayed on new inputs and lengths with eager work between, gives the eager bits."""
    d = cuda(make(16, [200, 5, 0, 131], 4, 2, 64, 64, "bf16"))
    args = [d[x] for x in ARGS]
    dims = ssd.delta._dims(*args, d["cu"], None, 3)
    ws = [torch.empty(f(dims), dtype=torch.uint8, device="cuda") for f in (ssd.ssd_delta_forward_workspace_bytes, ssd.ssd_delta_backward_workspace_bytes)]
    y, final = torch.empty_like(d["v"]), torch.empty_like(d["init"])

    def step():
        ssd.ssd_delta_forward(*args, cu_seqlens=d["cu"], init_state=d["init"], y=y, final_state=final, workspace=ws[0])
        return ssd.ssd_delta_backward(*args, d["dy"], cu_seqlens=d["cu"], init_state=d["init"], dfinal=d["dfinal"], workspace=ws[1])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i, lens in enumerate(([200, 5, 0, 131], [1, 1, 333, 1], [84, 84, 84, 84], [0, 336, 0, 0])):
        new = make(20 + i, lens, 4, 2, 64, 64, "bf16")
        for n in ARGS + ("dy", "init", "dfinal", "cu"):
            d[n].copy_(new[n])
        for w in ws:
            w.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in captured.items()}
        got.update(y=y.clone(), final=final.clone())
        want = step()
        torch.cuda.synchronize()
        want.update(y=y, final=final)
        for n in want:
            assert torch.equal(got[n], want[n]), (i, n)


def test_decode_steps_in_a_graph():
    """Captured steps update one state, replay after replay."""
    d = cuda(make(17, [1, 1, 1], 4, 2, 128, 64, "bf16"))
    a, b = d["init"].clone(), d["init"].clone()
    y = torch.empty_like(d["v"])
    ssd.ssd_delta_step(a.clone(), *[d[x] for x in ARGS], y_t=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_delta_step(a, *[d[x] for x in ARGS], y_t=y)
    for i in range(4):
        new = make(30 + i, [1, 1, 1], 4, 2, 128, 64, "bf16")
        for x in ARGS:
            d[x].copy_(new[x])
        graph.replay()
        torch.cuda.synchronize()
        want = ssd.ssd_delta_step(b, *[d[x] for x in ARGS])
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(y, want), i


def test_streams_and_two_at_once():
    d = cuda(make(18, [300, 20, 64], 4, 2, 64, 64, "bf16"))
    want = run(d)
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(6):
        args = [d[x] for x in ARGS]
        s = streams[i % 2]
        y, final = ssd.ssd_delta_forward(*args, cu_seqlens=d["cu"], init_state=d["init"], final_state=True, stream=s)
        got.append(dict(ssd.ssd_delta_backward(*args, d["dy"], cu_seqlens=d["cu"], init_state=d["init"], dfinal=d["dfinal"], stream=s),
                        y=y, final=final))
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(want[n], x[n]) for n in want)


def test_gradients_by_differences():
    """fp32: <dy, y> along a random direction of every input, by central differences of the forward pass in the kernels."""
    d = make(19, [100], 2, 1, 32, 32, "fp32", decay=0.3)
    g = cuda(d)
    grads = run(g)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def value(z):
        y, final = ssd.ssd_delta_forward(*[z[n] for n in ARGS], cu_seqlens=z["cu"], init_state=z["init"], final_state=True)
        return (y.double() * g["dy"].double()).sum() + (final.double() * g["dfinal"].double()).sum()

    for n in ARGS + ("init",):
        step = torch.randn(g[n].shape, generator=gen, device="cuda")
        if n in ("log_a", "beta"):
            step = step * 0.1
        # the quotient's error: of second order in h, and the values' rounding (about 1e-6 of |dy||y|) over h
        h = 2e-3
        diff = float((value(dict(g, **{n: g[n] + h * step})) - value(dict(g, **{n: g[n] - h * step}))) / (2 * h))
        along = float((grads["d" + n].double() * step.double()).sum())
        size = float(grads["d" + n].double().norm() * step.double().norm()) / np.sqrt(step.numel())
        noise = 1e-6 * float(g["dy"].double().norm() * grads["y"].double().norm()) / h
        assert abs(diff - along) <= 0.02 * size + noise, (n, diff, along, size)


def test_binding_refusals():
    d = cuda(make(21, [10, 20], 4, 2, 64, 32, "bf16"))
    args = {x: d[x] for x in ARGS}

    def forward(**kw):
        a = dict(args, cu_seqlens=d["cu"])
        a.update(kw)
        return ssd.ssd_delta_forward(**a)

    for kw in (dict(k=d["k"][:, :1]), dict(v=d["v"][:20]), dict(log_a=d["log_a"][:, :2]), dict(init_state=d["init"][:1]),
               dict(q=d["q"].transpose(0, 1)), dict(cu_seqlens=d["cu"].int()), dict(cu_seqlens=d["cu"].cpu()),
               dict(v=d["v"][:, :3], log_a=d["log_a"][:, :3].contiguous(), beta=d["beta"][:, :3].contiguous()),
               dict(y=torch.empty_like(d["v"]).float()[:, :, :16]), dict(workspace=torch.empty(10 ** 6, dtype=torch.uint8)),
               dict(cu_seqlens=None)):
        with pytest.raises((ValueError, TypeError)):
            forward(**kw)
    for kw in (dict(beta=d["beta"].bfloat16()), dict(k=d["k"].float()), dict(init_state=d["init"].bfloat16())):
        with pytest.raises(TypeError):
            forward(**kw)
    for kw in (dict(y=d["v"]), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), dict(scale=float("nan"))):
        with pytest.raises(ssd.SSDError):
            forward(**kw)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_delta_step(d["init"][:, :, :, :16].contiguous(), *[args[x][:2] if x != "v" else args[x][:2, :, :16].contiguous() for x in ARGS])


def test_far_into_large_tensors():
    """Element offsets past 2^31: the last tokens of a long packed axis with many wide heads."""
    T, H, G, N, P, L = 70000, 128, 2, 64, 256, 90
    v = torch.zeros((T, H, P), dtype=torch.bfloat16, device="cuda")
    assert v.numel() > 1 << 31
    d = cuda(make(22, [L], H, G, N, P, "bf16"))
    v[-L:].copy_(d["v"])
    dy = torch.zeros_like(v)
    dy[-L:].copy_(d["dy"])
    q, k, log_a, beta = (torch.zeros((T,) + d[x].shape[1:], dtype=d[x].dtype, device="cuda") for x in ("q", "k", "log_a", "beta"))
    for x, t in (("q", q), ("k", k), ("log_a", log_a), ("beta", beta)):
        t[-L:].copy_(d[x])
    cu = torch.tensor([T - L, T], dtype=torch.int64, device="cuda")
    want = run(d)
    got = run(dict(d, q=q, k=k, v=v, log_a=log_a, beta=beta, dy=dy, cu=cu))
    for n in want:
        assert torch.equal(got[n][-L:] if n not in ("final", "dinit") else got[n], want[n]), n
