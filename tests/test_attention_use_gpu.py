"""The attention layer as a program uses it: beside the SSD scan on one packed batch, captured into HIP graphs, on
other streams, with workspaces of any contents, and far into large tensors."""
import numpy as np
import pytest
import torch

import oracle
import oracle.attention as oa
import oracle.backward
import oracle.varlen
import ssd_inputs
import ssd_chunked_scan_02_amd as ssd
from attn_helpers import f64, make, offsets
from gpu_helpers import TOL, rel_l2

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_hybrid_stack(dtype):
    """Two layers of a hybrid stack on one packed batch, the scan's output being the attention's queries, keys
    and values, and the way back through both, against the fp64 models: bounds as for the scan alone."""
    lens = [130, 1, 0, 77, 200]
    cfg = ssd_inputs.config("mamba2_layer" if dtype == "bf16" else "tiny_fp32", nheads=4, skip=True)
    p = ssd_inputs.packed_inputs(cfg, lens, 3)
    g = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in p.items()}
    cu, H, P = g["cu_seqlens"], cfg["nheads"], cfg["headdim"]
    table = torch.randn((16, H), generator=torch.Generator().manual_seed(1))
    how = dict(table=table.cuda(), max_distance=64, softcap=8.0)
    y1, _, _ = ssd.ssd_forward_varlen(g["x"], g["log_a"], g["B"], g["C"], cu, max(lens), g["D"], chunk=cfg["chunk"])
    kv = y1[:, ::2].contiguous()                         # two key heads of the four
    y2, lse = ssd.ssd_attn_forward(y1, kv, kv, cu, lse=True, **how)
    dy = ssd_inputs.output_gradients(dict(cfg, batch=1, seqlen=sum(lens)), 5)["dy"][0]
    back = ssd.ssd_attn_backward(y1, kv, kv, y2, lse, dy.cuda(), cu, **how)
    dy1 = back["dq"].clone()
    dy1[:, ::2] += back["dk"] + back["dv"]
    dx = ssd.ssd_backward_varlen(g["x"], g["log_a"], g["B"], g["C"], dy1, cu, max(lens), g["D"])["dx"]
    torch.cuda.synchronize()

    c = p["cu_seqlens"].numpy()
    args = [f64(p[n]) for n in ("x", "log_a", "B", "C")]
    r1, _ = oracle.varlen.forward_varlen(oracle.default_oracle(), *args, c, f64(p["D"]))
    ref = oa.attention(r1, r1[:, ::2], r1[:, ::2], cu=c, cap=8.0, table=f64(table), max_distance=64, dy=f64(dy))
    rdy1 = ref["dq"].copy()
    rdy1[:, ::2] += ref["dk"] + ref["dv"]
    want = oracle.varlen.backward_varlen(oracle.backward.default_adjoint(), *args, c, f64(p["D"]), dy=rdy1)
    errors = dict(y=rel_l2(f64(y2), ref["y"]), dtable=rel_l2(f64(back["dtable"]), ref["dtable"]), dx=rel_l2(f64(dx), want["dx"]))
    print("[gpu case] hybrid stack %s: %s" % (dtype, errors), flush=True)
    # two layers, each within the scan's bound, forward and back: four times that at the far end
    assert all(e <= 4 * TOL[dtype] for e in errors.values()), errors


def _training_case(H, Hk):
    lens = [300, 5, 0, 131]
    d = make(7, sum(lens), sum(lens), H, Hk, 64, "bf16", bias="buckets", grads=True)
    return {n: (t.cuda() if t is not None else None) for n, t in d.items()}, offsets(lens).cuda()


# few and many heads: the split kernels, and the whole ones with their plan
@pytest.mark.parametrize("H,Hk", [(4, 2), (80, 80)])
def test_training_step_in_a_graph(H, Hk):
    """A captured forward and backward, replayed on new inputs and new document lengths with eager work and
    synchronizations in between, gives the eager call's bits every time."""
    g, cu = _training_case(H, Hk)
    how = dict(table=g["table"], softcap=20.0)
    y, lse = torch.empty_like(g["q"]), torch.empty(g["q"].shape[:2], device="cuda")
    dims = ssd.attention._dims(g["q"], g["k"], g["v"], cu, None, True, None, 20.0, None, g["table"], 128, False, None)
    ws = torch.empty(ssd.ssd_attn_backward_workspace_bytes(dims, True), dtype=torch.uint8, device="cuda")

    def step():
        ssd.ssd_attn_forward(g["q"], g["k"], g["v"], cu, y=y, lse=lse, **how)
        return ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y, lse, g["dy"], cu, workspace=ws, **how)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i, lens in enumerate(([300, 5, 0, 131], [1, 1, 433, 1], [100, 112, 112, 112], [0, 436, 0, 0])):
        for n in ("q", "k", "v", "dy"):
            g[n].copy_(torch.randn(g[n].shape, generator=torch.Generator().manual_seed(i)))
        cu.copy_(offsets(lens))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in captured.items()}
        got["y"], got["lse"] = y.clone(), lse.clone()
        want = step()
        torch.cuda.synchronize()
        want.update(y=y, lse=lse)
        for n in want:
            assert torch.equal(got[n], want[n]), (i, n)


@pytest.mark.parametrize("H,Hk", [(4, 2), (80, 80)])
def test_workspace_contents_do_not_matter(H, Hk):
    g, cu = _training_case(H, Hk)
    y, lse = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], cu, table=g["table"], lse=True)
    dims = ssd.attention._dims(g["q"], g["k"], g["v"], cu, None, True, None, 0.0, None, g["table"], 128, False, None)
    need = ssd.ssd_attn_backward_workspace_bytes(dims, True)
    got = []
    for fill in (0x00, 0xFF, 0x7F):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        got.append(ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y, lse, g["dy"], cu, table=g["table"], workspace=ws[:need]))
        torch.cuda.synchronize()
        assert torch.all(ws[need:] == fill)              # nothing past its end
    for n in got[0]:
        assert torch.equal(got[0][n], got[1][n]) and torch.equal(got[0][n], got[2][n]), n


def test_another_stream_and_two_at_once():
    """Calls on streams of their own, two at a time, give the bits of calls on the current one."""
    g, cu = _training_case(4, 2)
    y, lse = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], cu, table=g["table"], lse=True)
    want = ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y, lse, g["dy"], cu, table=g["table"])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(6):
        s = streams[i % 2]
        y2, lse2 = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], cu, table=g["table"], lse=True, stream=s)
        got.append((y2, lse2, ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y2, lse2, g["dy"], cu, table=g["table"], stream=s)))
    torch.cuda.synchronize()
    for y2, lse2, grads in got:
        assert torch.equal(y, y2) and torch.equal(lse, lse2)
        assert all(torch.equal(want[n], grads[n]) for n in want)


def test_two_decode_graphs_share_a_cache():
    """Two captured decode steps with workspaces of their own, replayed in turn and on two streams at once."""
    torch.manual_seed(1)
    n, H, Hk, D, page = 2, 8, 2, 64, 16
    kc, vc = (torch.randn((100, page, Hk, D), device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(100, device="cuda")[:96].view(2, 48).to(torch.int32)
    seq = torch.tensor([700, 333], dtype=torch.int64, device="cuda")
    qs = [torch.randn((n, H, D), device="cuda").bfloat16() for _ in range(2)]
    want = [ssd.ssd_attn_decode(q, kc, vc, table, seq) for q in qs]
    ys, graphs = [torch.empty_like(q) for q in qs], []
    torch.cuda.synchronize()
    for q, y in zip(qs, ys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ssd.ssd_attn_decode(q, kc, vc, table, seq, y=y)
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1]), i


def test_far_into_large_tensors():
    """Element offsets past 2^31 (and byte offsets past 2^32): a wide token stride, and a cache's last pages."""
    H, Hk, D, wide = 4, 2, 64, 1 << 16
    total, lens = 40000, [39800, 200]
    big = torch.empty((total, wide), dtype=torch.bfloat16, device="cuda")
    assert big.numel() > 1 << 31
    d = make(3, 200, 200, H, Hk, D, "bf16", grads=True)
    q, k, v = (big[:, at:at + h * D].unflatten(1, (h, D)) for at, h in ((0, H), (512, Hk), (1024, Hk)))
    for to, n in ((q, "q"), (k, "k"), (v, "v")):
        to[39800:].copy_(d[n])
    cu = torch.tensor([39800, 39800, 40000], dtype=torch.int64, device="cuda")  # (the rest is of no sequence)
    y, lse = ssd.ssd_attn_forward(q, k, v, cu, lse=True)
    dy = torch.zeros((total, H, D), dtype=torch.bfloat16, device="cuda")
    dy[39800:].copy_(d["dy"])
    got = ssd.ssd_attn_backward(q, k, v, y, lse, dy, cu)
    g = {n: d[n].cuda() for n in ("q", "k", "v", "dy")}
    one = torch.tensor([0, 0, 200], dtype=torch.int64, device="cuda")
    y2, lse2 = ssd.ssd_attn_forward(g["q"], g["k"], g["v"], one, lse=True)
    torch.cuda.synchronize()
    near = lambda a, b: rel_l2(f64(a), f64(b))  # noqa: E731  (the two calls may share the work differently)
    assert near(y[39800:], y2) < 4e-3 and near(lse[39800:], lse2) < 1e-6
    want = ssd.ssd_attn_backward(g["q"], g["k"], g["v"], y2, lse2, g["dy"], one)
    torch.cuda.synchronize()
    for n in want:
        assert near(got[n][39800:], want[n]) < 1e-2, n
    del big, q, k, v, dy, got, y, lse
    torch.cuda.empty_cache()

    pages, page, Hk, D = 140000, 64, 2, 128
    kc, vc = (torch.empty((pages, page, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 1 << 31
    new = make(4, 130, 130, 4, Hk, D, "bf16")
    table = torch.tensor([[pages - 1, pages - 2, pages - 5]], dtype=torch.int32, device="cuda")
    seq = torch.tensor([130], dtype=torch.int64, device="cuda")
    cu = torch.tensor([0, 130], dtype=torch.int64, device="cuda")
    ssd.ssd_kv_append(new["k"].cuda(), new["v"].cuda(), kc, vc, table, seq, cu)
    a = ssd.ssd_attn_decode(new["q"][-1:].cuda(), kc, vc, table, seq)
    low = torch.tensor([[0, 2, 1]], dtype=torch.int32, device="cuda")
    small = [torch.empty((3, page, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ssd.ssd_kv_append(new["k"].cuda(), new["v"].cuda(), *small, low, seq, cu)
    b = ssd.ssd_attn_decode(new["q"][-1:].cuda(), *small, low, seq)
    torch.cuda.synchronize()
    assert torch.equal(kc[pages - 1], small[0][0]) and torch.equal(vc[pages - 5, :2], small[1][1, :2])
    assert torch.equal(a, b)


def test_malformed_offsets_stay_inside():
    """Offsets that fall, repeat, or lie outside the axis give some outputs and touch nothing else."""
    T, H, D = 300, 4, 64
    guard = torch.full((T + 256, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    x = torch.randn((T, H, D), device="cuda").bfloat16()
    for bad in ([0, 500, -7, 300], [200, 100, 300, 250], [-1, -1, 10 ** 12, 5], [300, 300, 300, 300]):
        cu = torch.tensor(bad, dtype=torch.int64, device="cuda")
        y = guard.clone()
        lse = torch.zeros((T, H), device="cuda")
        ssd.ssd_attn_forward(x, x, x, cu, y=y[:T], lse=lse)
        ssd.ssd_attn_backward(x, x, x, y[:T], lse, x, cu)
        torch.cuda.synchronize()
        assert torch.all(y[T:] == 3.0), bad
