"""The operators that thin out a paged cache, and positions of several axes, as
measured cases.

Prompts with images and video fill a cache with long runs of tokens, placed by
time, height and width; a decoder that keeps only the tokens it attends to adds
up their weights, chooses, and closes the gaps.  The operators here:

  qk       norm of every query and key head, rotation by several positions a row
           (specfold_qk_norm_rope_axes)
  append   keys and values into the page pools, keys rotated that way
           (specfold_kv_append_axes)
  weigh    the attention weight that cached tokens get from a batch of rows, per
           key/value head (specfold_kv_weigh)
  select   the tokens of largest weight, beside the first and the latest ones
           (specfold_kv_select)
  compact  the kept tokens moved to the front of their sequences' pages, in place
           (specfold_kv_compact)

``run`` computes them by elementary torch operations, or, with ``own`` true,
by the library's calls.  Lengths within a batch follow from the case alone
(``lengths``), values, pages and kept tokens from the seed.
"""
import math

import numpy as np
import torch

own = False

TAIL = 3          # rows behind the last sequence: capacity that a step leaves unused
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a 7B-like model with time, height and width in blocks of its pairs: all latency
        dict(name="qk one token", op="qk", dtype="bf16", rows=1, heads=28, kv=4, dim=128, axes=3, order="blocks",
             own_freq=False, norm=False, theta=1e6, layout="fused"),
        # the rows of a long video prompt, 3B-like heads, the axes' pairs in turn: all bandwidth
        dict(name="qk video prompt", op="qk", dtype="bf16", rows=16381, heads=24, kv=8, dim=128, axes=3, order="turns",
             own_freq=False, norm=True, theta=5e6, layout="fused"),
        # images' patches by height and width, each axis with frequencies of its own, the tiny fp32 configuration's heads
        dict(name="append patches f32", op="append", dtype="f32", seqs=5, rows=333, kv=2, dim=64, axes=2, order="blocks",
             own_freq=True, ctx=200, page=24, norm=False, theta=1e4, layout="heads", gather=False),
        # several prompts with images at once, 3B-like heads
        dict(name="append prompts", op="append", dtype="bf16", seqs=8, rows=2041, kv=8, dim=128, axes=3, order="turns",
             own_freq=False, ctx=100, page=64, norm=True, theta=5e6, layout="split", gather=False),
        # a single sequence's step of decoding, 7B-like heads: all latency
        dict(name="weigh one token", op="weigh", dtype="bf16", seqs=1, rows=1, heads=28, kv=4, dim=128, ctx=2047, page=16,
             layout="fused", decay=1.0, gather=False),
        # a batch's step of decoding: the keys once
        dict(name="weigh decoding", op="weigh", dtype="bf16", seqs=64, rows=1, heads=28, kv=4, dim=128, ctx=8000, page=16,
             layout="fused", decay=0.98, gather=False),
        # the last rows of long prompts look back over them, 3B-like heads: arithmetic
        dict(name="weigh prompts' ends", op="weigh", dtype="bf16", seqs=4, rows=32, heads=24, kv=8, dim=128, ctx=32700,
             page=64, layout="split", decay=0.0, gather=False),
        # the tiny fp32 configuration's heads, the accepted rows of a verification step picked by index
        dict(name="weigh f32", op="weigh", dtype="f32", seqs=7, rows=5, heads=4, kv=2, dim=64, ctx=1111, page=24,
             layout="heads", decay=1.0, gather=True),
        # a budget overrun by a step's rows, one sequence
        dict(name="select one sequence", op="select", seqs=1, kv=4, ctx=2080, keep=2048, sinks=4, recent=64),
        # long prompts to a small budget
        dict(name="select long prompts", op="select", seqs=3, kv=8, ctx=131071, keep=4096, sinks=4, recent=512),
        # the same overrun over a whole batch
        dict(name="compact step", op="compact", dtype="bf16", seqs=64, kv=4, dim=128, ctx=2080, keep=2048, page=16,
             layout="fused"),
        # a few long prompts' kept tokens
        dict(name="compact prompts", op="compact", dtype="bf16", seqs=3, kv=8, dim=128, ctx=32700, keep=4096, page=64,
             layout="split"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, kv = rng.choice([(28, 4), (24, 8), (32, 8), (16, 16), (12, 2), (20, 1), (4, 2), (7, 7)])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    op = rng.choice(["qk", "append", "weigh", "weigh", "select", "compact"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128, 256])
    layout = rng.choice(["fused", "split", "heads"])
    rope = dict(axes=rng.choice([1, 2, 3, 3, 4]), order=rng.choice(["blocks", "turns"]), own_freq=rng.random() < 0.3,
                theta=rng.choice([1e4, 1e6, 5e6]))
    if op == "qk":
        rows = spread(1, min(16381, 16381 * 32 * 256 // ((heads + kv) * dim * SIZE[dtype])))
        return dict(op="qk", dtype=dtype, rows=rows, heads=heads, kv=kv, dim=dim, norm=rng.random() < 0.5, layout=layout,
                    **rope)
    if op == "append":
        seqs = spread(1, 64)
        rows = spread(1, max(1, min(2041, 8 * 2041 * 8 * 256 // (seqs * kv * dim * SIZE[dtype]))))
        return dict(op="append", dtype=dtype, seqs=seqs, rows=rows, kv=kv, dim=dim, ctx=spread(1, 1500) - 1, page=page,
                    norm=rng.random() < 0.5, layout=layout, gather=rng.random() < 0.3, **rope)
    if op == "weigh":
        seqs = spread(1, 64)
        rows = rng.choice([1, 1, spread(2, 64), spread(2, 64)])
        if dtype == "f32":
            seqs, rows = min(seqs, 16), min(rows, 16)
        # no more keys than the listed batch of decoding, nor more arithmetic than the prompts' ends (fp32: a sixteenth)
        most = min(40000, 64 * 8000 * 4 * 256 // (seqs * kv * dim * SIZE[dtype]),
                   4 * 32 * 24 * 32700 * 128 // ((1 if dtype == "bf16" else 16) * seqs * rows * heads * dim))
        return dict(op="weigh", dtype=dtype, seqs=seqs, rows=rows, heads=heads, kv=kv, dim=dim,
                    ctx=spread(1, max(2, most)) - 1, page=page, layout=layout, decay=rng.choice([0.0, 0.98, 1.0]),
                    gather=rng.random() < 0.3)
    seqs = spread(1, 64)
    keep = spread(1, 4096)
    if op == "select":
        ctx = spread(1, max(1, min(131071, 3 * 8 * 131071 // (seqs * kv))))
        sinks = rng.choice([0, min(4, keep // 2)])
        return dict(op="select", seqs=seqs, kv=kv, ctx=ctx, keep=keep, sinks=sinks,
                    recent=rng.choice([0, keep // 8, keep - sinks]))
    keep = max(1, min(keep, 64 * 2048 * 4 * 256 // (seqs * kv * dim * SIZE[dtype])))
    ctx = keep + spread(1, max(1, min(32700, 64 * 2080 * 4 * 256 // (seqs * kv * dim * SIZE[dtype])) - keep + 1)) - 1
    return dict(op="compact", dtype=dtype, seqs=seqs, kv=kv, dim=dim, ctx=ctx, keep=keep, page=page, layout=layout)


def lengths(case):
    """Cache length and row count of every sequence of a batch: the first has
    the case's own, the others a spread of shorter ones (the golden ratio's
    multiples), so that a batch is ragged."""
    s = np.arange(case["seqs"])
    part = (s * 0.6180339887498949) % 1.0
    low = 0.4
    if case["op"] == "compact":     # what is kept varies little from sequence to sequence: most are over the budget
        low = 1.0 - 0.6 * (case["ctx"] - case["keep"]) / max(1, case["ctx"])
    ctx = np.where(s == 0, case["ctx"], np.floor(case["ctx"] * (low + (1 - low) * part))).astype(np.int64)
    most = case.get("rows", 0)
    rows = np.where(s == 0, most, 1 + np.floor((most - 1) * (0.3 + 0.7 * ((part * 7.0) % 1.0)))).astype(np.int64)
    return ctx, rows


def work(case):
    if case["op"] == "qk":
        n = case["rows"] * (case["heads"] + case["kv"]) * case["dim"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 4 * case["axes"] * case["rows"], "flops": 8 * n}
    ctx, rows = lengths(case)
    if case["op"] == "append":
        n = int(rows.sum()) * case["kv"] * case["dim"]
        return {"bytes": 4 * n * SIZE[case["dtype"]] + 4 * case["axes"] * int(rows.sum()), "flops": 8 * n}
    if case["op"] == "weigh":
        e, held = SIZE[case["dtype"]], int((ctx + rows).sum()) * case["kv"]
        # keys and queries, the weights' old values where they count, the new ones
        return {"bytes": held * case["dim"] * e + int(rows.sum()) * case["heads"] * case["dim"] * e
                + held * (4 if case["decay"] == 0.0 else 8),
                "flops": 2 * case["heads"] * case["dim"] * int((rows * (ctx + 1)).sum())}
    kept = np.minimum(ctx, case["keep"])
    if case["op"] == "select":
        return {"bytes": 4 * case["kv"] * int((ctx + kept).sum()), "flops": case["kv"] * int(ctx.sum())}
    moved = int(np.where(ctx > kept, kept, 0).sum()) * case["kv"]
    return {"bytes": moved * (4 * case["dim"] * SIZE[case["dtype"]] + 4 + 8) + 1, "flops": 0}


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


def _pairs(case):
    """Rotation pairs of every axis: time has fewer of three, as such models have them."""
    half, n = case["dim"] // 2, case["axes"]
    if n == 3:
        return [half // 4, half * 3 // 8, half * 3 // 8]
    return [half // n + (1 if a < half % n else 0) for a in range(n)]


def _axis_of(case):
    """The axis of every pair: the axes' pairs one block after the other, or in
    turn, an axis that has had its share left out."""
    pairs = _pairs(case)
    if case["order"] == "blocks":
        return [a for a, n in enumerate(pairs) for _ in range(n)]
    left, got = list(pairs), []
    while len(got) < sum(pairs):
        for a in range(len(pairs)):
            if left[a]:
                left[a] -= 1
                got.append(a)
    return got


def _exponents(case):
    """Exponent of 1 / theta for every pair: its place's among all, or its
    place's among its axis's own."""
    axis, half = _axis_of(case), case["dim"] // 2
    if not case["own_freq"]:
        return [j / half for j in range(half)]
    seen, pairs, got = [0] * case["axes"], _pairs(case), []
    for a in axis:
        got.append(seen[a] / pairs[a])
        seen[a] += 1
    return got


def _positions(case, count, rs):
    """Positions [axes, count] of text with pictures in it: where all axes run
    alike, and grids of rows and columns at one time."""
    out = np.zeros((case["axes"], count), np.int64)
    at, t = 0, int(rs.randint(0, 2000))
    while at < count:
        n = min(count - at, int(rs.randint(1, 400)))
        i = np.arange(n)
        if rs.rand() < 0.5:
            out[:, at:at + n] = t + i
            t += n
        else:
            wide = int(rs.randint(4, 40))
            grid = [i // (wide * wide), i // wide % wide, i % wide, i % 3]
            for a in range(case["axes"]):
                out[a, at:at + n] = t + grid[(a + 4 - case["axes"]) % 4 if case["axes"] < 3 else a]
            t += wide
        at += n
    return out.astype(np.int32)


def prepare(case, seed):
    gen, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    st = {"case": case, "eps": 1e-6}
    if "axes" in case:
        st["axis"] = torch.tensor(_axis_of(case), device="cuda")
        st["frequency"] = torch.tensor(_exponents(case), device="cuda", dtype=torch.float64).neg_().mul_(math.log(case["theta"])).exp_()
    if case["op"] == "qk":
        dt, dim, kv, rows, heads = DTYPES[case["dtype"]], case["dim"], case["kv"], case["rows"], case["heads"]
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
        st["positions"] = _dev(_positions(case, rows, rs))
        _plan(st)
        return st
    ctx, rows = lengths(case)
    if case["op"] in ("select", "compact"):
        most = int(ctx.max())
        # what tokens have gathered: most next to nothing, some of them exactly that, a few nearly all
        w = torch.randn((case["seqs"], case["kv"], most), device="cuda", generator=gen).mul_(2.5).exp_()
        w *= torch.rand(w.shape, device="cuda", generator=gen) > 0.125
        st["weights"], st["lengths"] = w, _dev(ctx.astype(np.int32))
        kept = np.minimum(ctx, case["keep"])
        if case["op"] == "select":
            st["kept"] = torch.full((case["seqs"], case["kv"], case["keep"]), -1, device="cuda", dtype=torch.int32)
            st["new_len"] = torch.zeros(case["seqs"], device="cuda", dtype=torch.int32)
            return st
        st["new_len"] = _dev(kept.astype(np.int32))
        st["kept"] = torch.zeros((case["seqs"], case["kv"], max(1, int(kept.max()))), device="cuda", dtype=torch.int32)
        for s in range(case["seqs"]):
            chosen = torch.rand((case["kv"], int(ctx[s])), device="cuda", generator=gen).argsort(-1)[:, : int(kept[s])]
            st["kept"][s, :, : int(kept[s])] = chosen.sort(-1).values.to(torch.int32)
        rows = np.zeros_like(ctx)
    dt, dim, kv = DTYPES[case["dtype"]], case["dim"], case["kv"]
    table, pages = _table(ctx + rows, case["page"], rs)
    st["k_pool"], st["v_pool"] = _pools(case, pages * case["page"], gen)
    st["table"], st["ctx"] = _dev(table), _dev(ctx.astype(np.int32))
    start = np.concatenate([[0], np.cumsum(rows)])
    total = int(start[-1])
    st["row_start"], st["total"] = _dev(start.astype(np.int32)), total
    cap = total + TAIL
    gather = case.get("gather", False)
    src = 2 * cap if gather else cap
    st["rows"] = _dev(np.sort(rs.permutation(src)[:cap]).astype(np.int32)) if gather else None
    if case["op"] == "append":
        x = _randn((src, 2, kv, dim), dt, gen, 2.0)
        st["k"], st["v"] = x[:, 0], x[:, 1]
        st["gk"] = _gains(case, gen) if case["norm"] else None
        st["positions"] = _dev(_positions(case, cap, rs))
    elif case["op"] == "weigh":
        st["q"] = _randn((src, case["heads"], dim), dt, gen, 1.5)
        most = int((ctx + rows).max())
        # what a few such batches gave before
        st["weights"] = torch.rand((case["seqs"], kv, most), device="cuda", generator=gen)
        st["weights"] *= 4.0 * case["rows"] * case["heads"] / (kv * most)
    _plan(st)
    return st


def _plan(st):
    """What a program that uses the library keeps: its cache, its axes, its workspace."""
    if own:
        from diffusion_branch_speculative_gb300 import binding
        case = st["case"]
        if "axes" in case:
            st["plan"] = binding.RopeAxes(case["theta"], _pairs(case), in_turn=case["order"] == "turns",
                                          own_frequencies=case["own_freq"])
        if "table" in st:
            st["cache"] = binding.PagedCache(st["k_pool"], st["v_pool"], st["table"], case["page"])
        if case["op"] == "weigh":
            w = st["weights"]
            st["ws"] = binding.alloc_workspace(binding.kv_weigh_workspace_size(
                binding.dtype_code(DTYPES[case["dtype"]]), st["total"] + TAIL, case["rows"], case["heads"], case["kv"],
                case["dim"], w.shape[0], w.shape[2]))


# ------------------------------------------------------------ plain forms --

def _norm_rope(x, gain, eps, positions, st):
    """x [rows, heads, dim] in 32 bits: norm of every head, then the rotation
    of (x[j], x[j + dim/2]) by its axis's position times its frequency; the
    angles, which far positions make large, in 64 bits."""
    y = x.float()
    if gain is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * gain.float()
    half = x.shape[-1] // 2
    angle = positions[st["axis"]].double().transpose(0, 1) * st["frequency"]
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = y[..., :half], y[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _slots(table, page, seq, at):
    return table[seq, at // page].long() * page + at % page


def _plain_append(st):
    t = torch.arange(st["total"], device="cuda")
    seq = torch.searchsorted(st["row_start"], t.to(torch.int32), right=True) - 1
    at = st["ctx"][seq].long() + t - st["row_start"][seq].long()
    src = t if st["rows"] is None else st["rows"][: st["total"]].long()
    slot = _slots(st["table"], st["case"]["page"], seq, at)
    k = _norm_rope(st["k"][src], st["gk"], st["eps"], st["positions"][:, : st["total"]], st)
    st["k_pool"][slot] = k.to(st["k_pool"].dtype)
    st["v_pool"][slot] = st["v"][src]
    return {"k": st["k_pool"], "v": st["v_pool"]}


def _plain_weigh(st):
    case, w = st["case"], st["weights"]
    dim, kv, g, N = case["dim"], case["kv"], case["heads"] // case["kv"], case["rows"]
    start, ctx = st["row_start"].long(), st["ctx"].long()
    count, first = start[1:] - start[:-1], start[:-1]
    S, L = len(ctx), w.shape[2]
    i = torch.arange(N, device="cuda")
    row = (first[:, None] + i).clamp(max=st["total"] + TAIL - 1)
    if st["rows"] is not None:
        row = st["rows"].long()[row]
    held = i < count[:, None]
    t = torch.arange(L, device="cuda").clamp(max=st["table"].shape[1] * case["page"] - 1)
    slot = _slots(st["table"], case["page"], torch.arange(S, device="cuda")[:, None], t[None].expand(S, L))
    t = torch.arange(L, device="cuda")
    k = st["k_pool"][slot].float()
    q = st["q"][row].float().view(S, N, kv, g, dim).permute(0, 2, 3, 1, 4).reshape(S, kv, g * N, dim)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).div_(math.sqrt(dim)).view(S, kv, g, N, L)
    del k
    sees = t <= (ctx[:, None] + i)[:, :, None]                      # [S, N, L]
    score.masked_fill_(~sees[:, None, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    score.div_(score.sum(-1, keepdim=True)).mul_(held[:, None, None, :, None])
    got = score.sum((2, 3))
    old = torch.where(t < ctx[:, None], case["decay"], 0.0)[:, None] * w
    w.copy_(torch.where((t < (ctx + count)[:, None])[:, None], old + got, w))
    return w


def _plain_select(st):
    case, w = st["case"], st["weights"]
    t, length = torch.arange(w.shape[2], device="cuda"), st["lengths"].long()[:, None]
    key = torch.where((t < case["sinks"]) | (t >= length - case["recent"]), math.inf, 0.0)[:, None] + w
    key = torch.where((t < length)[:, None], key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., : case["keep"]]
    kept = torch.minimum(length, torch.tensor(case["keep"], device="cuda"))[:, None]
    there = torch.arange(order.shape[-1], device="cuda") < kept
    order = torch.where(there, order, w.shape[2]).sort(-1).values
    n = order.shape[-1]
    st["kept"][..., :n] = torch.where(there, order.to(torch.int32), st["kept"][..., :n])
    st["new_len"].copy_(kept[:, 0, 0])
    return {"kept": st["kept"], "len": st["new_len"]}


def _plain_compact(st):
    case, w = st["case"], st["weights"]
    S, kv, n = st["kept"].shape
    seq = torch.arange(S, device="cuda")[:, None, None].expand(S, kv, n)
    head = torch.arange(kv, device="cuda")[None, :, None].expand(S, kv, n)
    i = torch.arange(n, device="cuda").expand(S, kv, n)
    live = i < st["new_len"].long()[:, None, None]
    seq, head, to, src = seq[live], head[live], i[live], st["kept"].long()[live]
    a, b = _slots(st["table"], case["page"], seq, to), _slots(st["table"], case["page"], seq, src)
    st["k_pool"][a, head] = st["k_pool"][b, head]
    st["v_pool"][a, head] = st["v_pool"][b, head]
    w[seq, head, to] = w[seq, head, src]
    return {"k": st["k_pool"], "v": st["v_pool"], "weights": w}


def run(st):
    case = st["case"]
    if own:
        from diffusion_branch_speculative_gb300 import binding
        if case["op"] == "qk":
            binding.specfold_qk_norm_rope_axes(st["q"], st["k"], st["q_out"], st["k_out"], st["plan"], st["positions"],
                                               gq=st["gq"], gk=st["gk"], eps=st["eps"])
            return {"q": st["q_out"], "k": st["k_out"]}
        if case["op"] == "append":
            binding.specfold_kv_append_axes(st["k"], st["v"], st["cache"], st["row_start"], st["ctx"], st["plan"],
                                            st["positions"], gk=st["gk"], eps=st["eps"], rows=st["rows"])
            return {"k": st["k_pool"], "v": st["v_pool"]}
        if case["op"] == "weigh":
            binding.specfold_kv_weigh(st["q"], st["cache"], st["row_start"], st["ctx"], case["rows"], st["weights"],
                                      st["ws"], decay=case["decay"], rows=st["rows"])
            return st["weights"]
        if case["op"] == "select":
            binding.specfold_kv_select(st["weights"], st["lengths"], case["keep"], st["kept"], st["new_len"],
                                       sinks=case["sinks"], recent=case["recent"])
            return {"kept": st["kept"], "len": st["new_len"]}
        binding.specfold_kv_compact(st["cache"], st["kept"], st["lengths"], st["new_len"], weights=st["weights"])
        return {"k": st["k_pool"], "v": st["v_pool"], "weights": st["weights"]}
    if case["op"] == "qk":
        st["q_out"].copy_(_norm_rope(st["q"], st["gq"], st["eps"], st["positions"], st))
        st["k_out"].copy_(_norm_rope(st["k"], st["gk"], st["eps"], st["positions"], st))
        return {"q": st["q_out"], "k": st["k_out"]}
    return {"append": _plain_append, "weigh": _plain_weigh, "select": _plain_select, "compact": _plain_compact}[case["op"]](st)


# ---------------------------------------------------- the definition, exact --

def _rotated(x, gain, eps, pos, case):
    """Complex form: (x[j] + i x[j + dim/2]) times e^(i pos theta^-exponent)."""
    x = x.to(torch.float64)
    dim = x.shape[-1]
    if gain is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / dim + eps) * gain.to(torch.float64)
    half, n, pairs = dim // 2, case["axes"], _pairs(case)
    if case["order"] == "blocks":
        axis = np.repeat(np.arange(n), pairs)
    else:       # the j-th of an axis comes in round j, rounds by axis
        axis = np.array([a for _, a in sorted((j, a) for a in range(n) for j in range(pairs[a]))])
    place = np.arange(half) / half
    if case["own_freq"]:
        place = np.array([np.sum(axis[:j] == axis[j]) / pairs[axis[j]] for j in range(half)])
    freq = _dev(np.power(float(case["theta"]), -place))
    angle = pos.to(torch.float64).index_select(0, _dev(axis)).T * freq
    turn = torch.polar(torch.ones_like(angle), angle)
    z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn[:, None]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "qk":
        return {"q": _rotated(st["q"], st["gq"], st["eps"], st["positions"], case),
                "k": _rotated(st["k"], st["gk"], st["eps"], st["positions"], case)}
    if case["op"] == "select":
        w, kept = st["weights"].cpu().numpy().astype(np.float64), st["kept"].cpu().numpy()
        n, sinks, recent = st["lengths"].cpu().numpy(), case["sinks"], case["recent"]
        for s in range(case["seqs"]):
            for h in range(case["kv"]):
                chosen = np.arange(n[s])
                if n[s] > case["keep"]:
                    middle = np.arange(sinks, n[s] - recent)
                    best = np.argsort(-w[s, h, middle], kind="stable")[: case["keep"] - sinks - recent]
                    chosen = np.concatenate([np.arange(sinks), np.sort(middle[best]), np.arange(n[s] - recent, n[s])])
                kept[s, h, : len(chosen)] = chosen
        return {"kept": _dev(kept), "len": _dev(np.minimum(n, case["keep"]).astype(np.int32))}
    page, table = case["page"], st["table"].cpu().numpy().astype(np.int64)

    def slots(s, tokens):
        return _dev(table[s, tokens // page] * page + tokens % page)

    if case["op"] == "compact":
        k_pool, v_pool = st["k_pool"].to(torch.float64), st["v_pool"].to(torch.float64)
        w, kept, n = st["weights"].to(torch.float64), st["kept"].cpu().numpy().astype(np.int64), st["new_len"].tolist()
        for s in range(case["seqs"]):
            to = slots(s, np.arange(n[s]))
            for h in range(case["kv"]):
                src = slots(s, kept[s, h, : n[s]])
                k_pool[to, h] = st["k_pool"][src, h].to(torch.float64)
                v_pool[to, h] = st["v_pool"][src, h].to(torch.float64)
                w[s, h, : n[s]] = st["weights"][s, h, _dev(kept[s, h, : n[s]])].to(torch.float64)
        return {"k": k_pool, "v": v_pool, "weights": w}
    start, ctx = st["row_start"].tolist(), st["ctx"].tolist()
    picked = torch.arange(st["total"] + TAIL, device="cuda") if st["rows"] is None else st["rows"].long()
    if case["op"] == "append":
        k_pool, v_pool = st["k_pool"].to(torch.float64), st["v_pool"].to(torch.float64)
        for s in range(case["seqs"]):
            a, b = start[s], start[s + 1]
            to, src = slots(s, np.arange(ctx[s], ctx[s] + b - a)), picked[a:b]
            k_pool.index_copy_(0, to, _rotated(st["k"].index_select(0, src), st["gk"], st["eps"], st["positions"][:, a:b], case))
            v_pool.index_copy_(0, to, st["v"].index_select(0, src).to(torch.float64))
        return {"k": k_pool, "v": v_pool}
    w, g = st["weights"].to(torch.float64), case["heads"] // case["kv"]
    for s in range(case["seqs"]):
        a, n, c = start[s], start[s + 1] - start[s], ctx[s]
        k = st["k_pool"][slots(s, np.arange(c + n))].to(torch.float64).permute(1, 2, 0)
        q = st["q"].index_select(0, picked[a:a + n]).to(torch.float64).transpose(0, 1)
        past = torch.arange(c + n, device="cuda")[None] > c + torch.arange(n, device="cuda")[:, None]
        w[s, :, :c] *= case["decay"]
        w[s, :, c:c + n] = 0.0
        for h in range(case["heads"]):
            p = torch.matmul(q[h], k[h // g]) * case["dim"] ** -0.5
            w[s, h // g, : c + n] += torch.softmax(p.masked_fill(past, -math.inf), -1).sum(0)
    return w
