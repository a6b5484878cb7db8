"""A hybrid stack's layers as a program runs them together: rotary positions, attention and the gated delta rule on one packed
batch, there and back; and serving it, a prompt's one pass and then token after token over an 8-bit cache, captured."""
import numpy as np
import pytest
import torch

import oracle.attention as oa
import oracle.delta as od
import ssd_chunked_scan_02_amd as ssd
from attn_helpers import DTYPE, f64, offsets
from gpu_helpers import TOL, rel_l2
from test_kv8_gpu import FORMS, gathered, values
from test_rotary_gpu import turned

pytestmark = pytest.mark.gpu


def _normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def _unit(seed, *shape):
    return torch.nn.functional.normalize(_normal(seed, *shape), dim=-1)


def _gates(seed, *shape):
    return -0.2 * torch.nn.functional.softplus(_normal(seed, *shape)), _normal(seed + 1, *shape).sigmoid()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_training_step(dtype):
    """Rotation, attention and the delta rule over the attention's output, and the way back through the three, against the
    fp64 models.  Each layer is within the scan's bound; there and back are two of them, and two more for the rotations."""
    lens, H, Hk, G, D, N = [130, 1, 0, 77, 200], 4, 2, 2, 64, 64
    T, dt = sum(lens), DTYPE[dtype]
    q, k, v = _normal(1, T, H, D).to(dt), _normal(2, T, Hk, D).to(dt), _normal(3, T, Hk, D).to(dt)
    kd, qd = _unit(4, T, G, N).to(dt), _unit(5, T, G, N).to(dt)
    log_a, beta = _gates(6, T, H)
    dy, cu = _normal(8, T, H, D).to(dt), offsets(lens)
    inv, m = ssd.ssd_rotary_frequencies(D, factor=4.0, trained=64)
    g = [t.cuda() for t in (q, k, v, qd, kd, log_a, beta, dy, cu, inv)]
    Q, K, V, QD, KD, A, B, DY, CU, INV = g
    rq, rk = ssd.ssd_rotate(Q, INV, CU, k=K, magnitude=m)
    y1, lse = ssd.ssd_attn_forward(rq, rk, V, CU, lse=True)
    y2, _ = ssd.ssd_delta_forward(QD, KD, y1, A, B, CU)
    far = ssd.ssd_delta_backward(QD, KD, y1, A, B, DY, CU)
    back = ssd.ssd_attn_backward(rq, rk, V, y1, lse, far["dv"], CU)
    dq, dk = ssd.ssd_rotate(back["dq"], INV, CU, k=back["dk"], magnitude=m, inverse=True)
    torch.cuda.synchronize()

    c, pos = cu.numpy(), np.concatenate([np.arange(n) for n in lens])
    tq, tk = turned(q, pos, inv, False, m, 1), turned(k, pos, inv, False, m, 1)
    r1 = oa.attention(tq, tk, f64(v), cu=c)["y"]
    args = [f64(qd), f64(kd), r1, f64(log_a), f64(beta), c, N ** -0.5]
    r2, _ = od.forward(*args, None)
    want = od.backward(*args, f64(dy), None, None)
    ref = oa.attention(tq, tk, f64(v), cu=c, dy=want["dv"])
    want.update(y=r2, dv0=ref["dv"], **{n: turned(torch.from_numpy(ref[n]), pos, inv, False, m, -1) for n in ("dq", "dk")})
    got = dict(y=y2, dq=dq, dk=dk, dv0=back["dv"], dbeta=far["dbeta"])
    errors = {n: rel_l2(f64(t), want[n]) for n, t in got.items()}
    print("[gpu case] hybrid training step %s: %s" % (dtype, errors), flush=True)
    assert all(e <= 4 * TOL[dtype] for e in errors.values()), errors


@pytest.mark.parametrize("dtype,form", [("bf16", "e4m3"), ("fp32", "int8")])
def test_serving(dtype, form):
    """Prompts of several lengths (one of a single token) through the stack, the attention reading them back from the 8-bit
    cache, then five tokens each from a captured graph, which gives an eager run's bits; all of it against the fp64
    models on what the cache holds.  The bound is that of the training step."""
    lens, more, H, Hk, G, D, N, page = [70, 1, 33, 128], 5, 8, 2, 4, 64, 128, 16
    n, T, dt = len(lens), sum(lens), DTYPE[dtype]
    need = [-(-(x + more) // page) for x in lens]
    table = torch.full((n, max(need)), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(need), generator=torch.Generator().manual_seed(0)).to(torch.int32), 0
    for i, x in enumerate(need):
        table[i, :x] = order[at:at + x]
        at += x
    inv = ssd.ssd_rotary_frequencies(D)[0]
    cu, total = offsets(lens), T + n * more
    q, k, v = (_normal(s, total, h, D).to(dt) for s, h in ((1, H), (2, Hk), (3, Hk)))
    kd, qd = (_unit(s, total, G, N).to(dt) for s in (4, 5))
    log_a, beta = _gates(6, total, H)

    def gpu(t):
        return t.cuda()

    def new(i):
        """The rows of token i after the prompts."""
        return slice(T + i * n, T + (i + 1) * n)

    pages = [torch.zeros((sum(need), page, Hk, D), dtype=FORMS[form]).cuda() for _ in "kv"]
    scales = [torch.zeros((sum(need), page, Hk), device="cuda") for _ in "kv"]
    cache = pages + scales + [gpu(table)]
    INV, CU = gpu(inv), gpu(cu)
    length = torch.tensor(lens).cuda()
    p = slice(0, T)
    rq = ssd.ssd_kv8_append(gpu(k[p]), gpu(v[p]), *cache, length, CU, INV, q=gpu(q[p]))
    ck, cv = ssd.ssd_kv8_read(*cache, length, CU, T, dtype=dt)
    y1, _ = ssd.ssd_attn_forward(rq, ck, cv, CU)
    y2, state = ssd.ssd_delta_forward(gpu(qd[p]), gpu(kd[p]), y1, gpu(log_a[p]), gpu(beta[p]), CU, final_state=True)

    names = dict(q=q, k=k, v=v, qd=qd, kd=kd, log_a=log_a, beta=beta)
    now = {x: gpu(t[new(0)]) for x, t in names.items()}

    def token(cache, length, state, y):
        length.add_(1)
        turned_q = ssd.ssd_kv8_append(now["k"], now["v"], *cache, length, inv_freq=INV, q=now["q"])
        z = ssd.ssd_kv8_decode(turned_q, *cache, length)
        ssd.ssd_delta_step(state, now["qd"], now["kd"], z, now["log_a"], now["beta"], y_t=y)

    one = ([t.clone() for t in cache], length.clone(), state.clone(), torch.empty((n, H, D), dtype=dt, device="cuda"))
    two = ([t.clone() for t in cache], length.clone(), state.clone(), torch.empty((n, H, D), dtype=dt, device="cuda"))
    warm = ([t.clone() for t in cache], length.clone(), state.clone(), torch.empty((n, H, D), dtype=dt, device="cuda"))
    token(*warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token(*two)
    tokens = []
    for i in range(more):
        for x, t in names.items():
            now[x].copy_(t[new(i)])
        token(*one)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one[3], two[3]) and torch.equal(one[2], two[2])
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(one[0][:4], two[0][:4]))
        tokens.append(f64(two[3]))

    held = [gathered(values(c, s), table, [x + more for x in lens]) for c, s in ((one[0][0], one[0][2]), (one[0][1], one[0][3]))]
    at, worst = 0, {}
    for s, x in enumerate(lens):
        rows = list(range(int(cu[s]), int(cu[s]) + x)) + [T + i * n + s for i in range(more)]
        keys, vals = (f64(t[at:at + x + more]) for t in held)
        at += x + more
        c = np.array([0, x + more])
        a = oa.attention(turned(q[rows], np.arange(x + more), inv, False, 1.0, 1), keys, vals, cu=c)["y"]
        want, final = od.forward(f64(qd[rows]), f64(kd[rows]), a, f64(log_a[rows]), f64(beta[rows]), c, N ** -0.5, None)
        got = np.concatenate([f64(y2[int(cu[s]):int(cu[s + 1])])] + [t[s:s + 1] for t in tokens])
        for name, e in (("y", rel_l2(got, want)), ("state", rel_l2(f64(one[2][s]), final[0]))):
            worst[name] = max(worst.get(name, 0.0), e)
    print("[gpu case] serving %s %s: %s" % (dtype, form, worst), flush=True)
    assert all(e <= 4 * TOL[dtype] for e in worst.values()), worst
