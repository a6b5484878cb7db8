"""Cases and plain forms of the operators that a hybrid stack needs beside its SSD scan and attention.

Three operators: the gated delta rule (chunked forward, training step, single-token step), on the states, gates and packed
axes of the SSD scan; a paged cache held in 8 bits (append with rotation, decode, read-back); and rotary positions for
training and prompts, whose gradient is the rotation back.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a toy model's layer at the shape of the tiny fp32 workload: one head, launch latency
        dict(name="delta_fwd_tiny_fp32", op="delta", train=False, dtype="fp32", nseq=1, tokens=256, spread=0.0, heads=1,
             groups=1, key=64, value=64, state=True),
        # one long prompt, two value heads to a key head, the state handed on to decoding
        dict(name="delta_fwd_prompt", op="delta", train=False, dtype="bf16", nseq=1, tokens=16384, spread=0.0, heads=32,
             groups=16, key=128, value=128, state=True),
        # a training step at the Mamba-2 layer workload's tokens, heads and widths
        dict(name="delta_train_layer", op="delta", train=True, dtype="bf16", nseq=8, tokens=16384, spread=0.0, heads=24,
             groups=24, key=128, value=64, state=False),
        # a small training step in fp32 on packed documents of odd lengths, with states in and out
        dict(name="delta_train_small_fp32", op="delta", train=True, dtype="fp32", nseq=5, tokens=901, spread=0.7, heads=6,
             groups=2, key=64, value=32, state=True),
        # decoding one user's chat, and a serving batch
        dict(name="delta_step_one", op="step", dtype="bf16", nseq=1, heads=32, groups=16, key=128, value=128),
        dict(name="delta_step_batch", op="step", dtype="bf16", nseq=64, heads=32, groups=16, key=128, value=128),
        # a batch of prompts written after what the cache holds already
        dict(name="kv8_append_prompts", op="append", dtype="bf16", form="e4m3", nseq=7, tokens=16385, spread=0.7, past=1500,
             heads=32, kv_heads=8, dim=128, page=16, pairs="interleaved"),
        # the past of a batch of prompts read back, for the attention of what follows it
        dict(name="kv8_read_past", op="read", dtype="bf16", form="int8", nseq=9, longest=4001, heads=32, kv_heads=8, dim=128,
             page=64),
        # a serving batch at the grouped-heads workload's heads and context
        dict(name="kv8_decode_batch", op="decode", dtype="bf16", form="e4m3", nseq=64, longest=8192, heads=64, kv_heads=8,
             dim=128, page=64, cap=0.0, bias="none"),
        # a few chats of odd lengths, no grouping, capped scores and a bias by distance
        dict(name="kv8_decode_ragged", op="decode", dtype="bf16", form="int8", nseq=17, longest=4001, heads=24, kv_heads=24,
             dim=64, page=32, cap=50.0, bias="slopes"),
        # queries and keys of a packed training batch, and the gradient through the rotation
        dict(name="rotate_train", op="rotate", dtype="bf16", nseq=32, tokens=16385, spread=1.0, heads=32, kv_heads=8, dim=128,
             part=128, pairs="half", train=True, factor=8.0),
        # one short prompt in fp32, a quarter of each head turned
        dict(name="rotate_small_fp32", op="rotate", dtype="fp32", nseq=1, tokens=77, spread=0.0, heads=6, kv_heads=2, dim=64,
             part=16, pairs="interleaved", train=False, factor=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "step", "append", "read", "decode", "decode", "rotate"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("delta", "step"):
        groups = rng.choice([1, 2, 3, 4, 8])
        case = dict(op=op, dtype=dtype, heads=groups * rng.choice([1, 2, 3]), groups=groups, key=rng.choice([32, 64, 128]),
                    value=rng.choice([32, 64, 128]))
        if op == "step":
            return dict(case, nseq=_log(rng, 1, 64))
        train, nseq = rng.random() < 0.5, _log(rng, 1, 32)
        return dict(case, train=train, nseq=nseq, tokens=max(nseq, _log(rng, 16, 4096 if train else 8192)),
                    spread=rng.choice([0.0, 0.3, 1.0]), state=rng.random() < 0.5)
    kv = rng.choice([1, 2, 3, 4, 8])
    case = dict(op=op, dtype=dtype, heads=kv * rng.choice([1, 2, 3, 4, 8]), kv_heads=kv, dim=rng.choice([32, 64, 128]),
                nseq=_log(rng, 1, 64))
    if op == "rotate":
        return dict(case, tokens=max(case["nseq"], _log(rng, 1, 16384)), spread=1.0, part=case["dim"] // rng.choice([1, 2]),
                    pairs=rng.choice(["half", "interleaved"]), train=rng.random() < 0.5, factor=rng.choice([1.0, 4.0]))
    case.update(form=rng.choice(["int8", "e4m3"]), page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        return dict(case, tokens=max(case["nseq"], _log(rng, 1, 8192)), spread=0.7, past=_log(rng, 1, 8000),
                    pairs=rng.choice(["half", "interleaved"]))
    case["longest"] = _log(rng, 20, 8192 if op == "decode" else 2048)
    if op == "decode":
        case.update(cap=rng.choice([0.0, 30.0]), bias=rng.choice(["none", "slopes", "buckets"]))
    return case


BUCKETS, FAR = 32, 128


def _lengths(case):
    """Token counts of the packed documents: equal ones for spread 0, else a log-normal mix."""
    n, total = case["nseq"], case["tokens"]
    if case["spread"] == 0.0:
        return [total // n + (i < total % n) for i in range(n)]
    r = random.Random(1000 * n + total)
    w = [math.exp(r.gauss(0.0, case["spread"])) for _ in range(n)]
    got = [1 + int((total - n) * x / sum(w)) for x in w]
    got[got.index(max(got))] += total - sum(got)
    return got


def _contexts(case):
    """Cache lengths of a batch, this token included: the longest one and others below it."""
    r = random.Random(31 * case["nseq"] + case["longest"])
    return [case["longest"]] + [r.randint(max(1, case["longest"] // 8), case["longest"])
                                for _ in range(case["nseq"] - 1)]


def _pasts(case):
    r = random.Random(7 * case["nseq"] + case["past"])
    return [r.randint(0, case["past"]) for _ in range(case["nseq"])]


# ---------------------------------------------------------------------------------------- prepare

def _pages(counts, page, gen):
    """A block table over a shuffled pool of pages, some of them in use by nobody."""
    need = [-(-c // page) for c in counts]
    width, pool = max(need) + 1, sum(need) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, pool


def _offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, H = DTYPES[case["dtype"]], case["heads"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def normal(*shape):
        return randn(*shape).to(dtype)

    st = dict(case=case, slopes=None, table=None)
    if case["op"] in ("delta", "step"):
        G, N, P, n = case["groups"], case["key"], case["value"], case["nseq"]
        T = n if case["op"] == "step" else case["tokens"]
        # what a layer has after its projections: activated and normalised queries and keys, writing strengths
        # from a sigmoid, decays from a positive step size and a rate of each head
        for x in "qk":
            st[x] = torch.nn.functional.normalize(torch.nn.functional.silu(randn(T, G, N)), dim=-1).to(dtype)
        st["v"] = normal(T, H, P)
        st["beta"] = randn(T, H).sigmoid()
        rate = 1.0 + 15.0 * torch.rand((H,), generator=gen, device="cuda")
        st["log_a"] = -rate * torch.nn.functional.softplus(randn(T, H) - 4.0)
        st["init"] = 0.3 * randn(n, H, N, P) if case["op"] == "step" or case["state"] else None
        if case["op"] == "delta":
            st["lens"] = _lengths(case)
            st["cu"] = _offsets(st["lens"])
            if case["train"]:
                st["dy"] = normal(T, H, P)
                st["dfinal"] = 0.1 * randn(n, H, N, P) if case["state"] else None
        return st
    Hk, D = case["kv_heads"], case["dim"]
    if case["op"] == "rotate":
        lens = _lengths(case)
        qk = normal(sum(lens), (H + Hk) * D)  # one projection's output: views of one tensor
        st["q"], st["k"] = qk[:, :H * D].unflatten(1, (H, D)), qk[:, H * D:].unflatten(1, (Hk, D))
        if case["train"]:
            st["dq"], st["dk"] = normal(sum(lens), H, D), normal(sum(lens), Hk, D)
        st["lens"], st["cu"] = lens, _offsets(lens)
        # the angles of a context `factor` times as long as the one that was trained on
        st["inv_freq"] = (10000.0 ** (-torch.arange(0, case["part"], 2, dtype=torch.float64) / case["part"])
                          / case["factor"]).float().cuda()
        st["magnitude"] = 0.1 * math.log(case["factor"]) + 1.0
        return st
    form = FORMATS[case["form"]]
    new = _lengths(case) if case["op"] == "append" else None
    lens = [a + b for a, b in zip(new, _pasts(case))] if new else _contexts(case)
    st["lens"], st["new"] = lens, new
    st["block_table"], pool = _pages(lens, case["page"], gen)
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int64).cuda()
    for x in "kv":  # what the cache holds: values of 8 bits and their scales
        st[x + "_cache"] = (randn(pool, case["page"], Hk, D) * 0.3 * TOP[case["form"]]).clamp(-TOP[case["form"]], TOP[case["form"]]).round().to(form)
        st[x + "_scale"] = (0.5 + torch.rand((pool, case["page"], Hk), generator=gen, device="cuda")) * 3.0 / TOP[case["form"]]
    if case["op"] == "append":
        qkv = normal(sum(new), (H + 2 * Hk) * D)
        st["q"] = qkv[:, :H * D].unflatten(1, (H, D))
        st["k"] = qkv[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
        st["v"] = qkv[:, (H + Hk) * D:].unflatten(1, (Hk, D))
        st["cu"] = _offsets(new)
        st["inv_freq"] = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    elif case["op"] == "read":
        st["cu"] = _offsets(lens)
    else:
        st["q"] = normal(case["nseq"], H, D)
        if case["bias"] == "slopes":
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
        if case["bias"] == "buckets":
            st["table"] = randn(BUCKETS, H)
    return st


# -------------------------------------------------------------------------------------------- run

def run(st):
    if own:
        return _run_own(st)
    return {"delta": _plain_delta, "step": _plain_step, "append": _plain_append, "read": _plain_read, "decode": _plain_decode,
            "rotate": _plain_rotate}[st["case"]["op"]](st)


def _run_own(st):
    import ssd_chunked_scan_02_amd as ssd
    c = st["case"]
    if c["op"] == "delta":
        args = (st["q"], st["k"], st["v"], st["log_a"], st["beta"])
        y, final = ssd.ssd_delta_forward(*args, cu_seqlens=st["cu"], init_state=st["init"], final_state=c["state"])
        got = dict(y=y, final=final)
        if c["train"]:
            got.update(ssd.ssd_delta_backward(*args, st["dy"], cu_seqlens=st["cu"], init_state=st["init"],
                                              dfinal=st["dfinal"]))
        return got
    if c["op"] == "step":
        y = ssd.ssd_delta_step(st["init"], st["q"], st["k"], st["v"], st["log_a"], st["beta"])
        return dict(y=y, state=st["init"])
    if c["op"] == "rotate":
        how = dict(cu_seqlens=st["cu"], interleaved=c["pairs"] == "interleaved", magnitude=st["magnitude"])
        q, k = ssd.ssd_rotate(st["q"], st["inv_freq"], k=st["k"], **how)
        if not c["train"]:
            return dict(q=q, k=k)
        dq, dk = ssd.ssd_rotate(st["dq"], st["inv_freq"], k=st["dk"], inverse=True, **how)
        return dict(q=q, k=k, dq=dq, dk=dk)
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["block_table"], st["seq_lens"])
    if c["op"] == "append":
        q = ssd.ssd_kv8_append(st["k"], st["v"], *cache, cu_seqlens=st["cu"], inv_freq=st["inv_freq"],
                               interleaved=c["pairs"] == "interleaved", q=st["q"])
        return dict(q=q, **{x: st[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")})
    if c["op"] == "read":
        k, v = ssd.ssd_kv8_read(*cache, st["cu"], sum(st["lens"]), dtype=DTYPES[c["dtype"]])
        return dict(k=k, v=v)
    return ssd.ssd_kv8_decode(st["q"], *cache, softcap=c["cap"], slopes=st["slopes"], table=st["table"], max_distance=FAR)


CHUNK = 64


def _plain_delta(st):
    c = st["case"]
    args = {x: st[x].float() for x in ("q", "k", "v", "log_a", "beta")}
    if st["init"] is not None:
        args["init"] = st["init"].clone()
    if not c["train"]:
        y, final = _chunked(c, st["cu"], max(st["lens"]), **args)
        return dict(y=y.to(st["v"].dtype), final=final if c["state"] else None)
    leaves = {x: t.detach().requires_grad_(True) for x, t in args.items()}
    with torch.enable_grad():
        y, final = _chunked(c, st["cu"], max(st["lens"]), **leaves)
        target = (y * st["dy"].float()).sum()
        if c["state"]:
            target = target + (final * st["dfinal"]).sum()
        grads = torch.autograd.grad(target, list(leaves.values()))
    got = dict(y=y.detach().to(st["v"].dtype), final=final.detach() if c["state"] else None)
    for x, g in zip(leaves, grads):
        got["d" + x] = g.to(st[x].dtype)
    return got


def _chunked(c, cu, longest, q, k, v, log_a, beta, init=None):
    """y [tokens, H, P] and the final states in fp32, chunk by chunk: the quadratic form inside a chunk, a state between."""
    H, N, P, n = c["heads"], c["key"], c["value"], c["nseq"]
    L = -(-longest // CHUNK) * CHUNK
    pos = torch.arange(L, device=cu.device)
    inside = pos < cu.diff()[:, None]
    at = torch.where(inside, cu[:-1, None] + pos, 0)

    def chunks(x):                                                       # [n, H, chunks, CHUNK, ...], zeros past an end
        x = x[at] * inside.reshape(n, L, *[1] * (x.dim() - 1))
        if x.shape[2] != H:
            x = x.repeat_interleave(H // x.shape[2], 2)
        return x.transpose(1, 2).unflatten(2, (-1, CHUNK)).contiguous()

    q, k, v, log_a, beta = (chunks(x) for x in (q, k, v, log_a, beta))
    g = log_a.double().cumsum(-1)                                        # 64 bits: differences of long sums
    i = torch.arange(CHUNK, device=cu.device)
    apart = (g[..., :, None] - g[..., None, :]).masked_fill(i[:, None] < i, -math.inf).exp()
    kt = k.transpose(-1, -2).contiguous()
    scores = (q @ kt) * apart.float()
    # (I + A) E = V - e^g K S; A is strictly lower, so its inverse is the product of I + (-A)^(2^j); powers lose bits
    a = -((k.double() @ kt.double()) * apart * beta.double()[..., None, :]).masked_fill(i[:, None] <= i, 0.0)
    eye = torch.eye(CHUNK, dtype=torch.float64, device=cu.device)
    inverse = eye + a
    for _ in range(5):
        a = a @ a
        inverse = inverse @ (eye + a)
    inverse, now = inverse.float(), g.exp().float()[..., None]
    left, whole = (g[..., -1:] - g).exp().float()[..., None], g[..., -1].exp().float()[..., None, None]
    s = torch.zeros((n, H, N, P), device=cu.device) if init is None else init
    ys = []
    for j in range(L // CHUNK):
        u = beta[:, :, j, :, None] * (inverse[:, :, j] @ (v[:, :, j] - now[:, :, j] * (k[:, :, j] @ s)))
        ys.append(now[:, :, j] * (q[:, :, j] @ s) + scores[:, :, j] @ u)
        s = whole[:, :, j] * s + kt[:, :, j] @ (left[:, :, j] * u)
    y = torch.stack(ys, 2).flatten(2, 3).transpose(1, 2) * N ** -0.5
    return y[inside], s


def _plain_step(st):
    s, r = st["init"], st["case"]["heads"] // st["case"]["groups"]
    q, k = (st[x].float().repeat_interleave(r, 1) for x in "qk")
    s *= st["log_a"].exp()[..., None, None]
    e = st["v"].float() - (k[..., None] * s).sum(-2)
    s += k[..., None] * (st["beta"][..., None] * e)[..., None, :]
    y = (q[..., None] * s).sum(-2) * st["case"]["key"] ** -0.5
    return dict(y=y.to(st["v"].dtype), state=s)


def _turn(x, cos, sin, pairs, part):
    """The first `part` elements of each head turned, in fp32."""
    x, rest = x.float()[..., :part], x.float()[..., part:]
    if pairs == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = x[..., ::2], x[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _angles(pos, inv_freq):
    angle = pos[:, None].double() * inv_freq.double()
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _plain_rotate(st):
    c, dtype = st["case"], st["q"].dtype
    i = torch.arange(st["q"].shape[0], device="cuda")
    cos, sin = _angles(i - st["cu"][torch.bucketize(i, st["cu"][1:], right=True)], st["inv_freq"])
    m = st["magnitude"]

    def turned(x, sin):
        y = _turn(x, cos * m, sin * m, c["pairs"], c["part"])
        return y.to(dtype)

    got = dict(q=turned(st["q"], sin), k=turned(st["k"], sin))
    if c["train"]:
        got.update(dq=turned(st["dq"], -sin), dk=turned(st["dk"], -sin))
    return got


def _quantise(x, form):
    """Values of 8 bits and a scale per row: the largest one is the type's largest, ties go to even."""
    scale = x.abs().amax(-1) / TOP[form]
    r = x / torch.where(scale > 0, scale, 1.0)[..., None]
    return (r.round() if form == "int8" else r).clamp(-TOP[form], TOP[form]).to(FORMATS[form]), scale


def _plain_append(st):
    c = st["case"]
    i = torch.arange(st["k"].shape[0], device="cuda")
    s = torch.bucketize(i, st["cu"][1:], right=True)
    pos = st["seq_lens"][s] - (st["cu"][s + 1] - i)
    page, off = st["block_table"][s, pos // c["page"]].long(), pos % c["page"]
    cos, sin = _angles(pos, st["inv_freq"])
    for x, t in (("k", _turn(st["k"], cos, sin, c["pairs"], c["dim"])), ("v", st["v"].float())):
        values, scale = _quantise(t, c["form"])
        st[x + "_cache"].view(torch.uint8)[page, off] = values.view(torch.uint8)
        st[x + "_scale"][page, off] = scale
    return dict(q=_turn(st["q"], cos, sin, c["pairs"], c["dim"]).to(st["q"].dtype),
                **{x: st[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")})


def _plain_read(st):
    c, dtype = st["case"], DTYPES[st["case"]["dtype"]]
    i = torch.arange(sum(st["lens"]), device="cuda")
    s = torch.bucketize(i, st["cu"][1:], right=True)
    pos = i - st["cu"][s]
    page, off = st["block_table"][s, pos // c["page"]].long(), pos % c["page"]
    return {x: (st[x + "_cache"].view(torch.uint8)[page, off].view(FORMATS[c["form"]]).float()
                * st[x + "_scale"][page, off][..., None]).to(dtype) for x in "kv"}


def _bucket_of(far):
    """Bucket of a distance: exact up to half the buckets, then spaced evenly in the logarithm up to FAR; borders
    compared in whole numbers."""
    e = BUCKETS // 2
    f, borders = BUCKETS - e, list(range(1, e))
    for k in range(f):  # (d / e)^f >= (FAR / e)^k
        borders.append(next(d for d in range(e, FAR + 1) if d ** f * e ** k >= FAR ** k * e ** f))
    return torch.bucketize(far, torch.tensor(borders, device=far.device), right=True)


def _plain_decode(st):
    c, L = st["case"], max(st["lens"])
    G = c["heads"] // c["kv_heads"]
    pos = torch.arange(L, device="cuda")
    page = st["block_table"][:, pos // c["page"]].clamp(min=0).long()    # [n, L]
    k, v = (st[x + "_cache"].view(torch.uint8)[page, pos % c["page"]].view(FORMATS[c["form"]]).float()
            * st[x + "_scale"][page, pos % c["page"]][..., None] for x in "kv")
    q = st["q"].float().unflatten(1, (-1, G))                           # [n, Hk, G, D]
    sc = (q @ k.permute(0, 2, 3, 1).contiguous()) * c["dim"] ** -0.5    # [n, Hk, G, L]
    if c["cap"]:
        sc = (sc / c["cap"]).tanh() * c["cap"]
    far = (st["seq_lens"][:, None] - 1 - pos).clamp(min=0)
    bias = None
    if st["slopes"] is not None:
        bias = -st["slopes"][:, None, None] * far
    if st["table"] is not None:
        bias = st["table"].t()[:, _bucket_of(far)]
    if bias is not None:
        sc = sc + bias.transpose(0, 1).unflatten(1, (-1, G))
    sc = sc.masked_fill(pos >= st["seq_lens"][:, None, None, None], -math.inf)
    p = (sc - sc.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    return (p @ v.transpose(1, 2).contiguous()).flatten(1, 2).to(st["q"].dtype)


# ------------------------------------------------------------------------------------------- work

def work(case):
    H, e = case["heads"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("delta", "step"):
        G, N, P = case["groups"], case["key"], case["value"]
        states = case["nseq"] * H * N * P * 4
        if case["op"] == "step":
            return dict(bytes=2 * states + case["nseq"] * ((2 * G * N + 2 * H * P) * e + 8 * H), flops=7 * case["nseq"] * H * N * P)
        t, s = case["tokens"], 2 * states if case["state"] else 0
        # the recurrence's own products: key and query by state, key by value, and the decay
        fwd, flops = t * ((2 * G * N + 2 * H * P) * e + 8 * H) + s, 7 * t * H * N * P
        if case["train"]:  # q, k, v, gates, dy in; their gradients out
            return dict(bytes=fwd + t * ((4 * G * N + 3 * H * P) * e + 16 * H) + s, flops=3 * flops)
        return dict(bytes=fwd, flops=flops)
    Hk, D = case["kv_heads"], case["dim"]
    if case["op"] == "rotate":
        n = case["tokens"] * (H + Hk) * D * (2 if case["train"] else 1)
        return dict(bytes=2 * n * e, flops=3 * n)
    if case["op"] == "append":
        return dict(bytes=case["tokens"] * (2 * (H + Hk) * D * e + 2 * Hk * (D + 4)), flops=case["tokens"] * (3 * H + 7 * Hk) * D)
    ctx = sum(_contexts(case))
    if case["op"] == "read":
        return dict(bytes=ctx * 2 * Hk * (D * (1 + e) + 4), flops=2 * ctx * Hk * D)
    return dict(bytes=ctx * 2 * Hk * (D + 4) + 2 * case["nseq"] * H * D * e, flops=4 * D * H * ctx)


# ------------------------------------------------------------------------------------------ exact

def exact(case, seed):
    st = prepare(case, seed)
    return {"delta": _exact_delta, "step": _exact_step, "append": _exact_append, "read": _exact_read, "decode": _exact_decode,
            "rotate": _exact_rotate}[case["op"]](case, st)


def _token(state, q, k, v, log_a, beta, scale):
    """One token of the recurrence: the decayed state, the error of what it says for the key, the next state, y."""
    old = state * torch.exp(log_a)[..., None, None]
    wrong = v - torch.einsum("bhnp,bhn->bhp", old, k)
    new = old + torch.einsum("bhn,bhp->bhnp", k, beta[..., None] * wrong)
    return old, wrong, new, scale * torch.einsum("bhnp,bhn->bhp", new, q)


def _exact_delta(case, st):
    """The recurrence token by token, all sequences beside each other; its adjoint from states kept every `hop` tokens."""
    H, G, N, P, n = case["heads"], case["groups"], case["key"], case["value"], case["nseq"]
    lens, T, scale = st["lens"], max(st["lens"]), 1.0 / math.sqrt(case["key"])
    first = [sum(lens[:i]) for i in range(n)]
    grouped = [h // (H // G) for h in range(H)]

    def by_time(x):  # [T, n, heads, ...]; a token past an end writes nothing and forgets nothing
        out = torch.zeros((T, n) + tuple(x.shape[1:]), dtype=torch.float64, device="cuda")
        for i in range(n):
            out[:lens[i], i] = x[first[i]:first[i] + lens[i]].double()
        return out

    def by_token(x):
        return torch.cat([x[:lens[i], i] for i in range(n)])

    v, la, beta = by_time(st["v"]), by_time(st["log_a"]), by_time(st["beta"])
    q, k = by_time(st["q"])[:, :, grouped], by_time(st["k"])[:, :, grouped]
    state = torch.zeros((n, H, N, P), dtype=torch.float64, device="cuda") if st["init"] is None else st["init"].double()
    hop, kept, y = 32, [], torch.zeros((T, n, H, P), dtype=torch.float64, device="cuda")
    for t in range(T):
        if case["train"] and t % hop == 0:
            kept.append(state)
        _, _, state, y[t] = _token(state, q[t], k[t], v[t], la[t], beta[t], scale)
    out = dict(y=by_token(y), final=state if case["state"] else None)
    if not case["train"]:
        return out
    dy = by_time(st["dy"])
    ds = st["dfinal"].double().clone() if case["state"] else torch.zeros_like(state)
    dq, dk, dv, dla, dbeta = (torch.zeros_like(x) for x in (q, k, v, la, beta))
    for b in reversed(range(len(kept))):
        steps, state = [], kept[b]
        for t in range(b * hop, min(T, b * hop + hop)):
            steps.append(_token(state, q[t], k[t], v[t], la[t], beta[t], scale))
            state = steps[-1][2]
        for t in reversed(range(b * hop, min(T, b * hop + hop))):
            old, wrong, new, _ = steps.pop()
            dq[t] = scale * torch.einsum("bhnp,bhp->bhn", new, dy[t])
            ds = ds + scale * torch.einsum("bhn,bhp->bhnp", q[t], dy[t])
            du = torch.einsum("bhnp,bhn->bhp", ds, k[t])
            dbeta[t] = (du * wrong).sum(-1)
            dv[t] = beta[t][..., None] * du
            dk[t] = torch.einsum("bhnp,bhp->bhn", ds, beta[t][..., None] * wrong) - torch.einsum("bhnp,bhp->bhn", old, dv[t])
            ds = ds - torch.einsum("bhn,bhp->bhnp", k[t], dv[t])
            dla[t] = (ds * old).sum((-1, -2))
            ds = ds * torch.exp(la[t])[..., None, None]
    out.update(dq=by_token(dq).unflatten(1, (G, -1)).sum(2), dk=by_token(dk).unflatten(1, (G, -1)).sum(2), dv=by_token(dv),
               dlog_a=by_token(dla), dbeta=by_token(dbeta))
    if st["init"] is not None:
        out["dinit"] = ds
    return out


def _exact_step(case, st):
    r = case["heads"] // case["groups"]
    q, k = (st[x].double().repeat_interleave(r, 1) for x in "qk")
    _, _, new, y = _token(st["init"].double(), q, k, st["v"].double(), st["log_a"].double(), st["beta"].double(),
                          1.0 / math.sqrt(case["key"]))
    return dict(y=y, state=new)


def _wave(x, pos, inv_freq, pairs, sign=1.0):
    """x [tokens, heads, D] with its pairs as complex numbers times e^(i angle), in 64 bits."""
    part = 2 * inv_freq.numel()
    w = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), sign * torch.outer(pos.double(), inv_freq.double()))[:, None]
    y = x.double().clone()
    head = y[..., :part]
    if pairs == "half":
        z = torch.complex(head[..., :part // 2], head[..., part // 2:]) * w
        y[..., :part] = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.complex(head[..., 0::2], head[..., 1::2]) * w
        y[..., :part] = torch.view_as_real(z).flatten(-2)
    return y, part


def _exact_rotate(case, st):
    pos = torch.cat([torch.arange(n, device="cuda") for n in st["lens"]])
    out = {}
    for x in ("q", "k", "dq", "dk") if case["train"] else ("q", "k"):
        y, part = _wave(st[x], pos, st["inv_freq"], case["pairs"], -1.0 if x[0] == "d" else 1.0)
        y[..., :part] *= st["magnitude"]
        out[x] = y
    return out


def _exact_append(case, st):
    """The rotated queries and the scales; the values of 8 bits have no value in 64."""
    out = dict(q=st["q"].double(), k_scale=st["k_scale"].double(), v_scale=st["v_scale"].double(), k_cache=None, v_cache=None)
    first = 0
    for s, (n, total) in enumerate(zip(st["new"], st["lens"])):
        pos, rows = torch.arange(total - n, total, device="cuda"), slice(first, first + n)
        at = (st["block_table"][s].long()[pos // case["page"]], pos % case["page"])
        out["q"][rows] = _wave(st["q"][rows], pos, st["inv_freq"], case["pairs"])[0]
        out["k_scale"][at] = _wave(st["k"][rows], pos, st["inv_freq"], case["pairs"])[0].abs().amax(-1) / TOP[case["form"]]
        out["v_scale"][at] = st["v"][rows].double().abs().amax(-1) / TOP[case["form"]]
        first += n
    return out


def _held(case, st, s, n):
    pages = st["block_table"][s, :-(-n // case["page"])].long()
    return [(st[x + "_cache"].double()[pages] * st[x + "_scale"][pages].double()[..., None]).flatten(0, 1)[:n] for x in "kv"]


def _exact_read(case, st):
    got = [_held(case, st, s, n) for s, n in enumerate(st["lens"])]
    return dict(k=torch.cat([x[0] for x in got]), v=torch.cat([x[1] for x in got]))


def _exact_decode(case, st):
    y = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    half, far_top = BUCKETS // 2, FAR
    lut = []
    for d in range(far_top + 1):  # the largest k with (FAR / half)^k <= (d / half)^(BUCKETS - half)
        k = 0
        while d >= half and half + k + 1 < BUCKETS and far_top ** (k + 1) * half ** half <= d ** half * half ** (k + 1):
            k += 1
        lut.append(d if d < half else half + k)
    lut = torch.tensor(lut, device="cuda")
    for s, n in enumerate(st["lens"]):
        k, v = _held(case, st, s, n)
        back = torch.arange(n - 1, -1, -1, device="cuda")
        for h in range(case["heads"]):
            g = h // (case["heads"] // case["kv_heads"])
            z = torch.mv(k[:, g].contiguous(), st["q"][s, h].double()) / math.sqrt(case["dim"])
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if st["slopes"] is not None:
                z = z - st["slopes"][h].double() * back
            if st["table"] is not None:
                z = z + st["table"].double()[lut[back.clamp(max=far_top)], h]
            y[s, h] = torch.mv(v[:, g].t().contiguous(), torch.softmax(z, 0))
    return y
