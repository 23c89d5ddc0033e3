"""The cache-side operators of a verification step, as measured cases.

A model that verifies drafts against a paged key/value cache does three
things around the projections of a layer, and these are the operators here:

  qk      norm of every query and key head, then the position rotation
          (specfold_qk_norm_rope)
  append  keys and values of the step's rows into the page pools, the keys
          normed and rotated on the way where the model asks for it
          (specfold_kv_append)
  tree    attention of the drafted rows over cache and tree
          (specfold_tree_attention)

``run`` computes them by elementary torch operations, or, with ``own`` true,
by the library's calls.  Lengths within a batch follow from the case alone
(``lengths``), values, pages and trees from the seed.
"""
import math

import numpy as np
import torch

own = False

PAD = -2          # parent of a padding row: sees nothing, its output is zeros
TAIL = 3          # rows behind the last sequence: capacity that a step leaves unused
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a 7B-like model (28 query heads on 4 key heads): the step of plain decoding, all latency
        dict(name="qk one token", op="qk", dtype="bf16", rows=1, heads=28, kv=4, dim=128, norm=True, theta=1e6,
             start=2047, layout="fused"),
        # the rows of a long prompt, cut raggedly, 3B-like heads: all bandwidth
        dict(name="qk prompt", op="qk", dtype="bf16", rows=16381, heads=24, kv=8, dim=128, norm=True, theta=1e4,
             start=24000, layout="fused"),
        # a batch of drafted trees in the tiny fp32 configuration's head shape, outputs head by head
        dict(name="qk trees f32", op="qk", dtype="f32", rows=777, heads=4, kv=2, dim=64, norm=True, theta=1e4,
             start=500, layout="heads"),
        # one token into the cache: latency
        dict(name="append one token", op="append", dtype="bf16", seqs=1, rows=1, kv=4, dim=128, ctx=2047, page=16,
             norm=True, theta=1e6, layout="fused", gather=False),
        # the accepted rows of 61 drafted trees written to their final places (rows picked from the step's)
        dict(name="append accepted", op="append", dtype="bf16", seqs=61, rows=33, kv=8, dim=128, ctx=1024, page=32,
             norm=False, theta=1e4, layout="split", gather=True),
        # prompts of eight sequences filling their pages
        dict(name="append prompts", op="append", dtype="bf16", seqs=8, rows=2041, kv=8, dim=128, ctx=777, page=64,
             norm=True, theta=1e4, layout="fused", gather=False),
        # plain decoding of one short sequence: the smallest call, latency
        dict(name="tree one token", op="tree", dtype="bf16", seqs=1, nodes=1, heads=28, kv=4, dim=128, ctx=511,
             page=16, layout="fused", pad=False),
        # plain decoding of a batch: all cache bandwidth
        dict(name="tree decode batch", op="tree", dtype="bf16", seqs=64, nodes=1, heads=28, kv=4, dim=128, ctx=8000,
             page=16, layout="fused", pad=False),
        # one long sequence with a 61-node tree: the cache has to be split over the whole GPU
        dict(name="tree long context", op="tree", dtype="bf16", seqs=1, nodes=61, heads=24, kv=8, dim=128, ctx=40000,
             page=64, layout="split", pad=False),
        # a batch padded to a common tree size, as a captured graph has it
        dict(name="tree padded batch", op="tree", dtype="bf16", seqs=16, nodes=33, heads=28, kv=4, dim=128, ctx=8192,
             page=16, layout="fused", pad=True),
        # the widest step: large trees over a large batch, where arithmetic bounds it too
        dict(name="tree wide batch", op="tree", dtype="bf16", seqs=32, nodes=128, heads=24, kv=8, dim=128, ctx=8192,
             page=64, layout="split", pad=False),
        # the tiny fp32 configuration's heads, pages stored head by head
        dict(name="tree f32", op="tree", dtype="f32", seqs=7, nodes=16, heads=4, kv=2, dim=64, ctx=1111, page=24,
             layout="heads", pad=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, kv = rng.choice([(28, 4), (24, 8), (32, 8), (16, 16), (12, 2), (20, 1), (4, 2), (7, 7)])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    op = rng.choice(["qk", "append", "tree", "tree"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128, 256])
    layout = rng.choice(["fused", "split", "heads"])
    theta = rng.choice([1e4, 5e5, 1e6])
    if op == "qk":
        rows = spread(1, min(16381, 16381 * 32 * 256 // ((heads + kv) * dim * SIZE[dtype])))
        return dict(op="qk", dtype=dtype, rows=rows, heads=heads, kv=kv, dim=dim, norm=rng.random() < 0.7,
                    theta=theta, start=spread(1, 100000) - 1, layout=layout)
    if op == "append":
        seqs = spread(1, 64)
        rows = spread(1, max(1, min(2041, 8 * 2041 * 8 * 256 // (seqs * kv * dim * SIZE[dtype]))))
        return dict(op="append", dtype=dtype, seqs=seqs, rows=rows, kv=kv, dim=dim, ctx=spread(1, 1500) - 1,
                    page=page, norm=rng.random() < 0.5, theta=theta, layout=layout, gather=rng.random() < 0.3)
    seqs = spread(1, 64)
    nodes = rng.choice([1, 1, spread(2, 128), spread(2, 128)])
    if dtype == "f32":
        seqs, nodes = min(seqs, 16), min(nodes, 64)
    # no more cache than the widest listed batch reads, nor more arithmetic (fp32: a sixteenth)
    most = min(40000, 32 * 8192 * 8 * 256 // (seqs * kv * dim * SIZE[dtype]),
               32 * 128 * 24 * 8192 * 128 // ((1 if dtype == "bf16" else 16) * seqs * nodes * heads * dim))
    return dict(op="tree", dtype=dtype, seqs=seqs, nodes=nodes, heads=heads, kv=kv, dim=dim,
                ctx=spread(1, max(2, most)) - 1, page=page, layout=layout, pad=rng.random() < 0.3)


def lengths(case):
    """Cache length and row count of every sequence of a batch: the first has
    the case's own, the others a spread of shorter ones (the golden ratio's
    multiples), so that a batch is ragged."""
    s = np.arange(case["seqs"])
    part = (s * 0.6180339887498949) % 1.0
    ctx = np.where(s == 0, case["ctx"], np.floor(case["ctx"] * (0.4 + 0.6 * part))).astype(np.int64)
    most = case["nodes"] if case["op"] == "tree" else case["rows"]
    rows = np.where(s == 0, most, 1 + np.floor((most - 1) * (0.3 + 0.7 * ((part * 7.0) % 1.0)))).astype(np.int64)
    return ctx, rows


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "qk":
        n = case["rows"] * (case["heads"] + case["kv"]) * case["dim"]
        return {"bytes": 2 * n * e + 4 * case["rows"], "flops": 8 * n}
    ctx, rows = lengths(case)
    if case["op"] == "append":
        n = int(rows.sum()) * case["kv"] * case["dim"]
        return {"bytes": 4 * n * e + 4 * int(rows.sum()), "flops": 8 * n}
    q = int(rows.sum()) * case["heads"] * case["dim"]
    cache = int((ctx + rows).sum()) * case["kv"] * case["dim"] * 2
    # every row sees its whole context and at least itself
    return {"bytes": (2 * q + cache) * e + 8 * int(rows.sum()),
            "flops": 4 * case["heads"] * case["dim"] * int((rows * (ctx + 1)).sum())}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, device="cuda", dtype=torch.float32, generator=gen).mul_(scale).to(dtype)


def _pools(case, tokens, gen):
    """Key and value pools [tokens, kv, dim] in one of the layouts that caches
    have: K and V of a token side by side, two tensors, or head by head."""
    kv, dim, dt = case["kv"], case["dim"], DTYPES[case["dtype"]]
    if case["layout"] == "fused":
        pool = torch.randn((tokens, 2, kv, dim), device="cuda", dtype=dt, generator=gen)
        return pool[:, 0], pool[:, 1]
    if case["layout"] == "split":
        return tuple(torch.randn((tokens, kv, dim), device="cuda", dtype=dt, generator=gen) for _ in range(2))
    return tuple(torch.randn((kv, tokens, dim), device="cuda", dtype=dt, generator=gen).transpose(0, 1) for _ in range(2))


def _table(need, page, rs):
    """Block tables over a shuffled pool: a sequence's pages lie anywhere."""
    pages = -(-need // page)
    total = int(pages.sum()) + 2
    order = rs.permutation(total)
    table = np.zeros((len(need), max(1, int(pages.max()))), np.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n]
        at += int(n)
    return table, total


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _gains(case, gen, scale=1.0):
    dt = DTYPES[case["dtype"]]
    return (scale * (1.0 + 0.2 * torch.randn(case["dim"], device="cuda", generator=gen))).to(dt)


def prepare(case, seed):
    gen, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    dt, dim, kv = DTYPES[case["dtype"]], case["dim"], case["kv"]
    st = {"case": case, "eps": 1e-6}
    if case["op"] == "qk":
        rows, heads = case["rows"], case["heads"]
        # the fused projection's output [rows, queries | keys | values]
        x = _randn((rows, heads + 2 * kv, dim), dt, gen, 2.0)
        st["q"], st["k"] = x[:, :heads], x[:, heads:heads + kv]
        if case["layout"] == "heads":
            st["q_out"] = torch.empty((heads, rows, dim), device="cuda", dtype=dt).transpose(0, 1)
            st["k_out"] = torch.empty((kv, rows, dim), device="cuda", dtype=dt).transpose(0, 1)
        else:
            st["q_out"] = torch.empty((rows, heads, dim), device="cuda", dtype=dt)
            st["k_out"] = torch.empty((rows, kv, dim), device="cuda", dtype=dt)
        st["gq"] = _gains(case, gen, 1.5) if case["norm"] else None
        st["gk"] = _gains(case, gen) if case["norm"] else None
        step = np.arange(rows) if case["rows"] > 1024 else rs.randint(0, 8, rows)   # a prompt, or depths in a tree
        st["positions"] = _dev((case["start"] + step).astype(np.int32))
        return st
    ctx, rows = lengths(case)
    table, pages = _table(ctx + rows, case["page"], rs)
    st["k_pool"], st["v_pool"] = _pools(case, pages * case["page"], gen)
    st["table"], st["ctx"] = _dev(table), _dev(ctx.astype(np.int32))
    if case["op"] == "append":
        start = np.concatenate([[0], np.cumsum(rows)])
        total = int(start[-1])
        cap = total + TAIL
        src = cap if not case["gather"] else 2 * cap
        x = _randn((src, 2, kv, dim), dt, gen, 2.0)
        st["k"], st["v"] = x[:, 0], x[:, 1]
        st["gk"] = _gains(case, gen) if case["norm"] else None
        st["rows"] = _dev(np.sort(rs.permutation(src)[:cap]).astype(np.int32)) if case["gather"] else None
        st["positions"] = None
        if not case["gather"] and case["rows"] <= 256:     # drafted rows sit at their depth, not at their slot
            pos = np.concatenate([c + rs.randint(0, 8, r) for c, r in zip(ctx, rows)] + [np.zeros(TAIL)])
            st["positions"] = _dev(pos.astype(np.int32))
    else:
        # trees: a row's parent is one of the eight rows before it, or the last cached token
        tree = []
        for r in rows:
            i = np.arange(r)
            tree.append(np.where(i == 0, -1, np.maximum(i - rs.randint(1, 9, r), -1)))
            if case["pad"]:
                tree.append(np.full(case["nodes"] - r, PAD))
        held = np.full_like(rows, case["nodes"]) if case["pad"] else rows
        if case["pad"]:      # the padding rows have slots in the cache as well
            table, pages = _table(ctx + held, case["page"], rs)
            st["k_pool"], st["v_pool"] = _pools(case, pages * case["page"], gen)
            st["table"] = _dev(table)
        start = np.concatenate([[0], np.cumsum(held)])
        total = int(start[-1])
        st["parent"] = _dev(np.concatenate(tree + [np.full(TAIL, PAD)]).astype(np.int32))
        st["q"] = _randn((total + TAIL, case["heads"], dim), dt, gen, 1.5)
        st["o"] = torch.zeros((total + TAIL, case["heads"], dim), device="cuda", dtype=dt)
    st["row_start"] = _dev(start.astype(np.int32))
    st["total"] = total
    if own:
        from diffusion_branch_speculative_gb300 import binding
        st["cache"] = binding.PagedCache(st["k_pool"], st["v_pool"], st["table"], case["page"])
        if case["op"] == "tree":
            n = binding.tree_attention_workspace_size(binding.dtype_code(dt), case["heads"], kv, dim, case["nodes"])
            st["ws"] = binding.alloc_workspace(n)
    return st


# ------------------------------------------------------------ plain forms --

def _norm_rope(x, gain, eps, positions, theta):
    """x [rows, heads, dim] in 32 bits: norm of every head, then the rotation
    of (x[j], x[j + dim/2]) by position * theta^(-2j/dim); the angles, which
    far positions make large, in 64 bits."""
    y = x.float()
    if gain is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * gain.float()
    half = x.shape[-1] // 2
    j = torch.arange(half, device=x.device, dtype=torch.float64)
    angle = positions.double()[:, None] * theta ** (-j / half)
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = y[..., :half], y[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _slots(table, page, seq, at):
    return table[seq, at // page].long() * page + at % page


def _plain_append(st):
    case, page = st["case"], st["case"]["page"]
    t = torch.arange(st["total"], device="cuda")
    seq = torch.searchsorted(st["row_start"], t.to(torch.int32), right=True) - 1
    at = st["ctx"][seq].long() + t - st["row_start"][seq].long()
    src = t if st["rows"] is None else st["rows"][: st["total"]].long()
    pos = at if st["positions"] is None else st["positions"][: st["total"]]
    slot = _slots(st["table"], page, seq, at)
    k = _norm_rope(st["k"][src], st["gk"], st["eps"], pos, case["theta"])
    st["k_pool"][slot] = k.to(st["k_pool"].dtype)
    st["v_pool"][slot] = st["v"][src]
    return {"k": st["k_pool"], "v": st["v_pool"]}


def _plain_tree(st):
    case, page = st["case"], st["case"]["page"]
    dim, kv, g = case["dim"], case["kv"], case["heads"] // case["kv"]
    start, ctx = st["row_start"].long(), st["ctx"].long()
    count, first = start[1:] - start[:-1], start[:-1]
    S, N, L = len(ctx), case["nodes"], int(st["table"].shape[1]) * page
    i = torch.arange(N, device="cuda")
    row = (first[:, None] + i).clamp(max=st["total"] + TAIL - 1)
    parent = torch.where(i < count[:, None], st["parent"][row].long(), PAD)
    there = parent != PAD
    # a row sees itself and its ancestors: the powers of (1 + child-to-parent)
    step = (parent[:, :, None] == i) | (torch.eye(N, device="cuda", dtype=torch.bool) & there[:, :, None])
    sees = torch.linalg.matrix_power(step.double(), N) > 0
    t = torch.arange(L, device="cuda")
    length = (ctx + count)[:, None]
    slot = _slots(st["table"], page, torch.arange(S, device="cuda")[:, None], t[None].expand(S, L))
    live = t < length
    k = st["k_pool"][slot].float() * live[:, :, None, None]
    v = st["v_pool"][slot].float() * live[:, :, None, None]
    node = (t - ctx[:, None]).clamp(0, N - 1)
    visible = torch.where((t < ctx[:, None])[:, None], there[:, :, None],
                          torch.gather(sees, 2, node[:, None].expand(S, N, L)) & live[:, None])
    q = st["q"][row].float().view(S, N, kv, g, dim).permute(0, 2, 3, 1, 4).reshape(S, kv, g * N, dim)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(dim)
    del k
    score = score.view(S, kv, g, N, L).masked_fill_(~visible[:, None, None], -math.inf)
    most = score.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = score.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, kv, g * N, L), v.permute(0, 2, 1, 3)).view(S, kv, g, N, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(S, N, kv * g, dim)
    held = i < count[:, None]
    st["o"][row[held]] = o[held].to(st["o"].dtype)
    return st["o"]


def run(st):
    case = st["case"]
    if own:
        from diffusion_branch_speculative_gb300 import binding
        if case["op"] == "qk":
            binding.specfold_qk_norm_rope(st["q"], st["k"], st["q_out"], st["k_out"], st["gq"], st["gk"], st["eps"],
                                          st["positions"], case["theta"])
            return {"q": st["q_out"], "k": st["k_out"]}
        if case["op"] == "append":
            binding.specfold_kv_append(st["k"], st["v"], st["cache"], st["row_start"], st["ctx"], gk=st["gk"],
                                       eps=st["eps"], positions=st["positions"], rope_theta=case["theta"],
                                       rows=st["rows"])
            return {"k": st["k_pool"], "v": st["v_pool"]}
        binding.specfold_tree_attention(st["q"], st["cache"], st["parent"], st["row_start"], st["ctx"],
                                        case["nodes"], st["o"], st["ws"])
        return st["o"]
    if case["op"] == "qk":
        st["q_out"].copy_(_norm_rope(st["q"], st["gq"], st["eps"], st["positions"], case["theta"]))
        st["k_out"].copy_(_norm_rope(st["k"], st["gk"], st["eps"], st["positions"], case["theta"]))
        return {"q": st["q_out"], "k": st["k_out"]}
    if case["op"] == "append":
        return _plain_append(st)
    return _plain_tree(st)


# ---------------------------------------------------- the definition, exact --

def _rotated(x, gain, eps, pos, theta):
    """Complex form: (x[j] + i x[j + dim/2]) times e^(i pos theta^(-2j/dim))."""
    x = x.to(torch.float64)
    dim = x.shape[-1]
    if gain is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / dim + eps) * gain.to(torch.float64)
    freq = torch.tensor([theta ** (-2.0 * j / dim) for j in range(dim // 2)], dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(freq)[None].expand(len(pos), -1).contiguous(), pos.to(torch.float64)[:, None] * freq)
    z = torch.complex(x[..., : dim // 2].contiguous(), x[..., dim // 2:].contiguous()) * turn[:, None]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "qk":
        return {"q": _rotated(st["q"], st["gq"], st["eps"], st["positions"], case["theta"]),
                "k": _rotated(st["k"], st["gk"], st["eps"], st["positions"], case["theta"])}
    start, ctx = st["row_start"].tolist(), st["ctx"].tolist()
    page, table = case["page"], st["table"].cpu().numpy().astype(np.int64)

    def slots(s, n):
        t = np.arange(n)
        return _dev(table[s, t // page] * page + t % page)

    if case["op"] == "append":
        k_pool, v_pool = st["k_pool"].to(torch.float64), st["v_pool"].to(torch.float64)
        for s in range(case["seqs"]):
            a, b = start[s], start[s + 1]
            to = slots(s, ctx[s] + b - a)[ctx[s]:]
            src = torch.arange(a, b, device="cuda") if st["rows"] is None else st["rows"][a:b].long()
            pos = torch.arange(ctx[s], ctx[s] + b - a, device="cuda") if st["positions"] is None else st["positions"][a:b]
            k_pool.index_copy_(0, to, _rotated(st["k"].index_select(0, src), st["gk"], st["eps"], pos, case["theta"]))
            v_pool.index_copy_(0, to, st["v"].index_select(0, src).to(torch.float64))
        return {"k": k_pool, "v": v_pool}
    out = torch.zeros_like(st["o"], dtype=torch.float64)
    parent = st["parent"].cpu().numpy()
    g = case["heads"] // case["kv"]
    for s in range(case["seqs"]):
        a, n, c = start[s], start[s + 1] - start[s], ctx[s]
        sees = np.zeros((n, c + n), bool)
        for i in range(n):
            j = i
            if parent[a + i] != PAD:
                sees[i, :c] = True
                while j >= 0:
                    sees[i, c + j] = True
                    j = int(parent[a + j])
        at = slots(s, c + n)
        k = st["k_pool"][at].to(torch.float64).transpose(0, 1).repeat_interleave(g, 0)
        v = st["v_pool"][at].to(torch.float64).transpose(0, 1).repeat_interleave(g, 0)
        live = _dev(sees.any(1).nonzero()[0])
        if len(live) == 0:
            continue
        q = st["q"][a + live].to(torch.float64).transpose(0, 1)
        w = torch.bmm(q, k.transpose(1, 2)) * case["dim"] ** -0.5
        w = w.masked_fill(~_dev(sees)[live][None], -math.inf)
        out[a + live] = torch.bmm(torch.softmax(w, -1), v).transpose(0, 1)
    return out
