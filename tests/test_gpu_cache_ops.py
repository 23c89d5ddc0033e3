"""Norm with rotation, paged append and tree attention on the GPU against the
float64 oracle (oracle/cache_oracle.py), element by element.

Bounds.  One rounding to the storage type is off by at most
u = finfo(type).eps / 2 of the value.  In 32-bit arithmetic (unit e = 2^-24):
  * a normed and rotated element y0 cos - y1 sin: the mean of squares sums
    hd/16 * 2 terms a lane and log2(hd/16) shuffles (relative 20 e, halved by the
    root), root, division and three products 6 e, the angle (32 bits of a half
    turn: pi 2^-25 rad) and the sine's own error 2^-22: together under 2e-6 of
    |y0| + |y1|; the frequencies' 64-bit rounding adds 2 pi 2^-49 rad a position.
  * attention: a score's sum of hd products is off by hd e * sum |q k| scale
    (times log2 e and 2^-22 for the exponential), which moves a weight by that
    share; numerator and denominator each: 2 (hd e score + 2^-21) of the
    softmax-weighted |v|, and a sum over the keys adds e a term in a chain no
    longer than 4096 + 64.  bf16 rounds the weights too: u of the weighted |v|.
"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from diffusion_branch_speculative_gb300 import binding
    binding.lib()
    return binding


def half_step(dt):
    return torch.finfo(DT[dt]).eps / 2


def randn(rng, shape, dt, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda().to(DT[dt])


def host(t):
    return t.double().cpu().numpy()


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ----------------------------------------------------- norm and rotation --

def rot_bound(dt, ref, size, positions):
    far = np.abs(np.asarray(positions, np.float64))[:, None, None] * (2 * np.pi * 2.0 ** -49)
    return half_step(dt) * np.abs(ref) + (2e-6 + far) * size * (1 + half_step(dt)) + 1e-30


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T,n_q,n_kv", [(1, 28, 4), (1, 1, 1), (2, 4, 2), (33, 7, 7), (301, 24, 8), (2500, 3, 1)])
@pytest.mark.parametrize("form", ["both", "queries", "keys", "rotate", "norm", "copy"])
def test_qk_norm_rope(B, dt, hd, T, n_q, n_kv, form):
    rng = np.random.default_rng(T * 131 + n_q * 7 + hd)
    x = randn(rng, (T, n_q + 2 * n_kv, hd), dt, 2.0)
    before = x.clone()
    q, k = x[:, :n_q], x[:, n_q:n_q + n_kv]
    gq = randn(rng, (hd,), dt) if form in ("both", "queries", "norm") else None
    gk = randn(rng, (hd,), dt) if form in ("both", "keys", "norm") else None
    theta = 0.0 if form in ("norm", "copy") else 1e4
    pos = rng.integers(0, 1 << 20, T)
    # queries token-major, keys head-major, both inside a larger buffer
    qo = torch.full((T, n_q + 1, hd), 7.0, device="cuda", dtype=DT[dt])
    ko = torch.full((n_kv, T + 1, hd), 7.0, device="cuda", dtype=DT[dt])
    B.specfold_qk_norm_rope(q, k, qo[:, :n_q], ko[:, :T].transpose(0, 1), gq, gk, 1e-5, ints(pos), theta)
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    assert (qo[:, n_q] == 7.0).all() and (ko[:, T] == 7.0).all()
    for got, src, g in ((qo[:, :n_q], q, gq), (ko[:, :T].transpose(0, 1), k, gk)):
        ref, size = orc.norm_rotate(host(src), None if g is None else host(g), 1e-5, pos, theta)
        err = np.abs(host(got) - ref)
        assert (err <= rot_bound(dt, ref, size, pos)).all(), err.max()
        if form == "copy":
            assert torch.equal(got, src)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_qk_in_place_equals_out_of_place(B, dt):
    rng = np.random.default_rng(5)
    x = randn(rng, (77, 12, 128), dt)
    g, pos = randn(rng, (128,), dt), ints(rng.integers(0, 5000, 77))
    qo, ko = torch.empty_like(x[:, :8]), torch.empty_like(x[:, 8:10])
    B.specfold_qk_norm_rope(x[:, :8], x[:, 8:10], qo, ko, g, g, 1e-6, pos, 1e6)
    v = x[:, 10:].clone()
    B.specfold_qk_norm_rope(x[:, :8], x[:, 8:10], x[:, :8], x[:, 8:10], g, g, 1e-6, pos, 1e6)
    torch.cuda.synchronize()
    assert torch.equal(x[:, :8], qo) and torch.equal(x[:, 8:10], ko) and torch.equal(x[:, 10:], v)


def test_qk_one_side_only_and_no_rows(B):
    rng = np.random.default_rng(6)
    q, pos = randn(rng, (5, 4, 64), "f32"), ints(range(5))
    a, b = torch.empty_like(q), torch.empty_like(q)
    B.specfold_qk_norm_rope(q, None, a, None, positions=pos, rope_theta=1e4)
    B.specfold_qk_norm_rope(None, q, None, b, positions=pos, rope_theta=1e4)
    B.specfold_qk_norm_rope(q[:0], None, a[:0], None, positions=pos[:0], rope_theta=1e4)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("theta", [1.0, 1e4, 1e6, 0.5])
def test_qk_far_positions(B, hd, theta):
    pos = np.array([0, 1, -1, 1 << 20, 131071, (1 << 31) - 1, -(1 << 31), 123456789])
    rng = np.random.default_rng(7)
    q = randn(rng, (len(pos), 3, hd), "f32")
    o = torch.empty_like(q)
    B.specfold_qk_norm_rope(q, None, o, None, positions=ints(pos), rope_theta=theta)
    ref, size = orc.norm_rotate(host(q), None, 0.0, pos, theta)
    # a base below one turns faster the higher the pair: its frequencies' share of the bound grows with them
    far = max(1.0, 1.0 / theta)
    assert (np.abs(host(o) - ref) <= rot_bound("f32", ref, size, pos * far)).all()


def test_qk_zero_rows_and_infinite_rows(B):
    q = torch.zeros(3, 2, 64, device="cuda")
    q[1, 0, 5] = float("inf")
    q[2, 1, 63] = float("nan")
    o = torch.empty_like(q)
    g = torch.ones(64, device="cuda")
    B.specfold_qk_norm_rope(q, None, o, None, gq=g, eps=1e-6, positions=ints([0, 0, 9]), rope_theta=1e4)
    torch.cuda.synchronize()
    assert (o[0] == 0).all() and (o[1, 1] == 0).all() and (o[2, 0] == 0).all()   # other heads untouched by them
    assert torch.isnan(o[1, 0]).any() and torch.isnan(o[2, 1]).all()


# ---------------------------------------------------------------- append --

def make_cache(B, rng, dt, hd, n_kv, page, need, layout, spare=2, widen=0):
    """A PagedCache over shuffled pages whose sequences hold `need` tokens."""
    pages = [max(1, -(-int(n) // page)) for n in need]
    total = sum(pages) + spare
    order = rng.permutation(total)
    table = np.full((len(need), max(pages) + widen), total + 5, np.int32)   # entries past a length are never used
    used = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[used:used + n]
        used += n
    tokens = total * page
    if layout == "fused":
        f = randn(rng, (tokens, 2, n_kv, hd), dt)
        kp, vp = f[:, 0], f[:, 1]
    elif layout == "heads":
        kp, vp = (randn(rng, (n_kv, tokens, hd), dt).transpose(0, 1) for _ in range(2))
    else:
        kp, vp = (randn(rng, (tokens, n_kv, hd), dt) for _ in range(2))
    wide = torch.full((table.shape[0], table.shape[1] + 3), -9, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = ints(table)
    return B.PagedCache(kp, vp, wide[:, :table.shape[1]], page), table


def check_append(B, cache, table, before, args, dt, T):
    K, V, start, ctx, gk, pos, theta, rows = args
    kp, vp, size = orc.append(before[0], before[1], table, cache.page_size, host(K), host(V), start, ctx,
                              None if gk is None else host(gk), 1e-6, pos, theta, rows)
    got_k, got_v = host(cache.k_pool), host(cache.v_pool)
    assert np.array_equal(got_v, vp)
    bound = np.zeros_like(kp)
    for at, sz in size.items():
        bound[at] = half_step(dt) * np.abs(kp[at]) + 2.1e-6 * sz
    assert (np.abs(got_k - kp) <= bound).all()     # zero off the written tokens
    return size


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hd,n_kv", [(64, 2), (128, 4), (128, 7)])
@pytest.mark.parametrize("page", [8, 24, 64])
@pytest.mark.parametrize("layout", ["fused", "split", "heads"])
@pytest.mark.parametrize("form", ["plain", "normed", "rotated", "placed", "picked"])
def test_kv_append(B, dt, hd, n_kv, page, layout, form):
    rng = np.random.default_rng(page + hd + n_kv)
    counts, ctx = [3, 0, 1, 41, 0, 2], [0, 5, 63, 130, 9, 23]
    start = np.concatenate([[0], np.cumsum(counts)])
    n = int(start[-1])
    T = n + 4                                           # rows behind the last sequence
    src = 2 * T if form == "picked" else T
    x = randn(rng, (src, 2 * n_kv + 1, hd), dt)
    K, V = x[:, :n_kv], x[:, n_kv + 1:]
    cache, table = make_cache(B, rng, dt, hd, n_kv, page, np.array(ctx) + counts, layout)
    gk = randn(rng, (hd,), dt) if form == "normed" else None
    theta = 0.0 if form == "plain" else 5e5
    pos = rng.integers(0, 300, T) if form == "placed" else None
    rows = rng.permutation(src)[:T] if form == "picked" else None
    before = host(cache.k_pool), host(cache.v_pool)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.specfold_kv_append(K, V, cache, ints(start), ints(ctx), gk=gk, positions=None if pos is None else ints(pos),
                         rope_theta=theta, rows=None if rows is None else ints(rows), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    size = check_append(B, cache, table, before, (K, V, start, ctx, gk, pos, theta, rows), dt, T)
    assert len(size) == n


def test_kv_append_many_sequences(B):
    rng = np.random.default_rng(3)
    S = 1024
    counts, ctx = rng.integers(0, 3, S), rng.integers(0, 20, S)
    start = np.concatenate([[0], np.cumsum(counts)])
    cache, table = make_cache(B, rng, "f32", 64, 1, 8, ctx + counts, "split")
    K, V = randn(rng, (int(start[-1]), 1, 64), "f32"), randn(rng, (int(start[-1]), 1, 64), "f32")
    before = host(cache.k_pool), host(cache.v_pool)
    B.specfold_kv_append(K, V, cache, ints(start), ints(ctx), rope_theta=1e4)
    torch.cuda.synchronize()
    check_append(B, cache, table, before, (K, V, start, ctx, None, None, 1e4, None), "f32", len(K))


def test_kv_append_drops_what_it_cannot_place(B):
    rng = np.random.default_rng(4)
    cache, table = make_cache(B, rng, "bf16", 64, 2, 8, [16, 16, 16], "fused")
    table[1, 1] = -1                                    # no such page
    table[2, 0] = 10 ** 6
    cache.block_table.copy_(ints(table))
    K, V = randn(rng, (9, 2, 64), "bf16"), randn(rng, (9, 2, 64), "bf16")
    before = host(cache.k_pool), host(cache.v_pool)
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    start, ctx = [0, 3, 6, 9], [14, 6, 3]               # the third token of sequence 0 lies past its table
    B.specfold_kv_append(K, V, cache, ints(start), ints(ctx), status=status[:1])
    assert B.specfold_get_status(status) == B.DEV_BAD_PAGE
    size = check_append(B, cache, table, before, (K, V, start, ctx, None, None, 0.0, None), "bf16", 9)
    assert len(size) == 4
    # picked rows out of range, then a batch whose entries are wrong
    before = host(cache.k_pool), host(cache.v_pool)
    rows = [0, -1, 2, 3, 9, 5, 0, 0, 0]
    B.specfold_kv_append(K, V, cache, ints([0, 3, 5, 5]), ints([2, 0, 0]), rows=ints(rows), status=status[:1])
    assert B.specfold_get_status(status) == B.DEV_BAD_SEQ
    check_append(B, cache, table, before, (K, V, [0, 3, 5, 5], [2, 0, 0], None, None, 0.0, rows), "bf16", 9)
    for bad_start, bad_ctx in (([0, 3, 2, 2], [0, 0, 0]), ([0, 3, 6, 12], [0, 0, 0]), ([-4, -1, 0, 0], [0, 0, 0]),
                               ([0, 0, 0, 1], [0, 0, -5])):
        keep = cache.k_pool.clone(), cache.v_pool.clone()
        B.specfold_kv_append(K, V, cache, ints(bad_start), ints(bad_ctx), status=status[:1])
        assert B.specfold_get_status(status) & B.DEV_BAD_SEQ
        written = int((cache.k_pool != keep[0]).any(-1).any(-1).sum())
        assert written <= 3                             # the valid sequence's rows at most


def test_kv_append_no_rows(B):
    rng = np.random.default_rng(8)
    cache, _ = make_cache(B, rng, "bf16", 64, 2, 8, [16], "split")
    keep = cache.k_pool.clone()
    K = randn(rng, (6, 2, 64), "bf16")
    B.specfold_kv_append(K, K, cache, ints([0, 0]), ints([0]))        # a batch without rows
    B.specfold_kv_append(K[:0], K[:0], cache, ints([0, 0]), ints([0]))
    torch.cuda.synchronize()
    assert torch.equal(cache.k_pool, keep)


# -------------------------------------------------------- tree attention --

def random_tree(rng, n, kind):
    i = np.arange(n)
    if kind == "chain":
        return np.maximum(i - 1, -1)
    if kind == "flat":
        return np.full(n, -1)
    p = np.maximum(i - rng.integers(1, 9, n), -1)
    if kind == "padded":
        p[rng.random(n) < 0.3] = -2
        for j in range(n):                              # no row below a padding row
            if p[j] >= 0 and p[p[j]] == -2:
                p[j] = -1
    return p


def tree_case(B, rng, dt, hd, n_q, n_kv, page, layout, counts, ctx, kind, extra=3):
    counts, ctx = np.asarray(counts), np.asarray(ctx)
    start = np.concatenate([[0], np.cumsum(counts)])
    T = int(start[-1]) + extra
    cache, table = make_cache(B, rng, dt, hd, n_kv, page, ctx + counts, layout)
    parent = None
    if kind != "none":
        parent = np.concatenate([random_tree(rng, int(n), kind) for n in counts] + [np.full(extra, 77)])
    wide = randn(rng, (T, n_q + 2, hd), dt, 1.5)
    q = wide[:, 1:n_q + 1]
    return dict(cache=cache, table=table, start=start, ctx=ctx, parent=parent, q=q, T=T,
                nodes=max(1, int(counts.max())))


def run_tree(B, c, o=None, ws=None, scale=0.0, nodes=None):
    q, cache = c["q"], c["cache"]
    nodes = nodes or c["nodes"]
    if o is None:
        o = torch.full(q.shape, 7.0, device="cuda", dtype=q.dtype)
    if ws is None:
        ws = B.alloc_workspace(B.tree_attention_workspace_size(B.dtype_code(q.dtype), q.shape[1], cache.n_kv,
                                                               q.shape[2], nodes))
    B.specfold_tree_attention(q, cache, None if c["parent"] is None else ints(c["parent"]), ints(c["start"]),
                              ints(c["ctx"]), nodes, o, ws, scale)
    return o, ws


def check_tree(B, c, o, dt, scale=0.0):
    hd = c["q"].shape[2]
    ref, spread, score = orc.tree_attention(host(c["q"]), host(c["cache"].k_pool), host(c["cache"].v_pool), c["table"],
                                            c["cache"].page_size, c["parent"], c["start"], c["ctx"], scale)
    got = host(o)
    free = np.isnan(ref)
    assert (got[free] == 7.0).all()                     # rows of no sequence stay as they were
    share = 2 * (hd * E * score * 1.45 + 2.0 ** -21) + 4160 * E
    u = half_step(dt)
    bound = (u * np.abs(ref) + ((u if dt == "bf16" else 0.0) + share) * spread * (1 + u)) + 1e-30
    err = np.abs(got - ref)
    ok = (err <= bound) | free
    assert ok.all(), (float(np.nanmax(err / bound)), np.argwhere(~ok)[:5])


GEOMETRY = [(1, 1, 64, 16, "split"), (28, 4, 128, 16, "fused"), (24, 8, 128, 24, "heads"), (4, 2, 64, 8, "fused"),
            (20, 1, 128, 64, "split"), (7, 7, 64, 128, "heads"), (32, 2, 64, 256, "fused"), (64, 1, 128, 32, "fused")]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,n_kv,hd,page,layout", GEOMETRY)
@pytest.mark.parametrize("counts,ctx", [([1], [0]), ([1], [1]), ([1], [700]), ([5], [0]), ([2, 0, 1, 9], [15, 4, 16, 333]),
                                        ([1] * 9, [0, 1, 15, 16, 17, 63, 64, 65, 200]), ([33, 64, 3], [130, 1, 250])])
@pytest.mark.parametrize("kind", ["tree", "padded", "none"])
def test_tree_attention(B, dt, n_q, n_kv, hd, page, layout, counts, ctx, kind):
    rng = np.random.default_rng(n_q * 1009 + sum(counts) * 31 + sum(ctx))
    c = tree_case(B, rng, dt, hd, n_q, n_kv, page, layout, counts, ctx, kind)
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0
    check_tree(B, c, o, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["chain", "flat", "tree"])
@pytest.mark.parametrize("n_q,n_kv,hd", [(4, 2, 64), (14, 2, 128)])
def test_tree_largest(B, dt, kind, n_q, n_kv, hd):
    rng = np.random.default_rng(11)
    c = tree_case(B, rng, dt, hd, n_q, n_kv, 16, "fused", [256, 1, 200], [77, 500, 0], kind)
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0
    check_tree(B, c, o, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [1, 4, 40])
def test_tree_long_context(B, dt, nodes):
    rng = np.random.default_rng(12)
    c = tree_case(B, rng, dt, 64, 4, 2, 32, "split", [nodes, 1], [20011, 300], "tree")
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    check_tree(B, c, o, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_tree_many_sequences(B, dt):
    rng = np.random.default_rng(13)
    c = tree_case(B, rng, dt, 64, 2, 1, 8, "split", rng.integers(0, 4, 1024), rng.integers(0, 70, 1024), "tree")
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    check_tree(B, c, o, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.01])
def test_tree_scale(B, dt, scale):
    rng = np.random.default_rng(14)
    c = tree_case(B, rng, dt, 128, 8, 2, 16, "fused", [7, 3], [90, 40], "tree")
    c["q"].mul_(0.3)
    o, _ = run_tree(B, c, scale=scale)
    torch.cuda.synchronize()
    check_tree(B, c, o, dt, scale)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nodes,g", [(5, 2), (30, 4), (70, 4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3e38])
def test_tree_unseen_values_change_nothing(B, dt, nodes, g, bad):
    """Stale pool tokens, padding rows' and other branches' keys and values."""
    rng = np.random.default_rng(15)
    c = tree_case(B, rng, dt, 128, 2 * g, 2, 16, "fused", [nodes, 3], [37, 16], "tree")
    par = c["parent"]
    par[2], par[3:nodes] = -2, np.where(par[3:nodes] == 2, 1, par[3:nodes])
    lone = nodes - 1                                    # a leaf: seen by itself alone
    clean, ws = run_tree(B, c)
    cache, table, page = c["cache"], c["table"], 16
    live = set()
    for s in range(2):
        for t in range(int(c["ctx"][s]) + int(c["start"][s + 1] - c["start"][s])):
            live.add(int(table[s, t // page]) * page + t % page)
    stale = torch.tensor(sorted(set(range(cache.k_pool.shape[0])) - live), device="cuda")
    cache.k_pool[stale], cache.v_pool[stale] = bad, bad
    for node in (2, lone):
        t = 37 + node
        at = int(table[0, t // page]) * page + t % page
        cache.k_pool[at], cache.v_pool[at] = bad, bad
    o, _ = run_tree(B, c, ws=ws)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0
    same = [t for t in range(c["T"]) if t != lone]
    assert torch.equal(o[same], clean[same])
    assert (o[2] == 0).all()
    if bad != bad:
        assert torch.isnan(o[lone]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [3, 60])
def test_tree_infinite_value_reaches_its_descendants_only(B, dt, nodes):
    rng = np.random.default_rng(16)
    c = tree_case(B, rng, dt, 64, 4, 2, 8, "split", [nodes], [21], "flat")
    c["parent"][2] = 1
    at = int(c["table"][0, 22 // 8]) * 8 + 22 % 8       # row 1's token
    clean, ws = run_tree(B, c)
    c["cache"].v_pool[at, :, 9] = float("inf")
    o, _ = run_tree(B, c, ws=ws)
    torch.cuda.synchronize()
    rows = [t for t in range(c["T"]) if t not in (1, 2)]
    assert torch.equal(o[rows], clean[rows])
    assert (o[1:3, :, 9] == float("inf")).all()
    rest = [d for d in range(64) if d != 9]
    assert torch.equal(o[1:3][..., rest], clean[1:3][..., rest])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [4, 50])
def test_tree_reports_and_survives_bad_entries(B, dt, nodes):
    rng = np.random.default_rng(17)
    c = tree_case(B, rng, dt, 64, 4, 2, 16, "fused", [nodes, 2, 3], [40, 8, 30], "tree")
    good, ws = run_tree(B, c)
    # parents out of range count as roots
    c["parent"][0], c["parent"][2], c["parent"][3] = 0, 9, -7
    o, _ = run_tree(B, c, ws=ws)
    assert B.specfold_get_status(ws) == B.DEV_BAD_PARENT
    check_tree(B, c, o, dt)
    c["parent"][0], c["parent"][2], c["parent"][3] = -1, -1, -1
    # pages outside the pool read as zeros
    keep = c["table"].copy()
    c["table"][0, 1], c["table"][2, 0] = -3, 10 ** 6
    c["cache"].block_table.copy_(ints(c["table"]))
    o, _ = run_tree(B, c, ws=ws)
    assert B.specfold_get_status(ws) == B.DEV_BAD_PAGE
    check_tree(B, c, o, dt)
    c["table"][:] = keep
    c["cache"].block_table.copy_(ints(keep))
    # tokens past the table: the same
    long_ctx = dict(c, ctx=c["ctx"] + np.array([0, 0, 16 * keep.shape[1]]))
    o, _ = run_tree(B, long_ctx, ws=ws)
    assert B.specfold_get_status(ws) == B.DEV_BAD_PAGE
    check_tree(B, long_ctx, o, dt)
    # invalid sequences are left out, the others computed
    o0, _ = run_tree(B, c, ws=ws)
    assert B.specfold_get_status(ws) == 0
    for change in (dict(ctx=c["ctx"] * np.array([1, -1, 1])), dict(start=c["start"] + np.array([0, 0, -1, 10 ** 6])),
                   dict(ctx=np.array([40, 2 ** 31 - 1, 30]))):
        o, _ = run_tree(B, dict(c, **change), ws=ws)
        assert B.specfold_get_status(ws) & B.DEV_BAD_SEQ
        assert torch.equal(o[:nodes], o0[:nodes])
    o, _ = run_tree(B, c, ws=ws, nodes=nodes - 1)       # more rows than the caller's bound
    assert B.specfold_get_status(ws) == B.DEV_BAD_SEQ
    assert (o[:nodes] == 7.0).all() and torch.allclose(o[nodes:nodes + 5].float(), o0[nodes:nodes + 5].float(), atol=0.05)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [1, 6, 48])
def test_tree_repeats_bit_for_bit_and_in_place(B, dt, nodes):
    rng = np.random.default_rng(18)
    c = tree_case(B, rng, dt, 128, 8, 2, 16, "fused", [nodes, 1, nodes], [900, 33, 5000], "tree")
    a, ws = run_tree(B, c)
    for _ in range(5):
        b, _ = run_tree(B, c, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    q = c["q"].clone()
    c["q"] = q
    run_tree(B, c, o=q, ws=ws)                          # o may be q
    torch.cuda.synchronize()
    n = int(c["start"][-1])
    assert torch.equal(q[:n], a[:n])


@pytest.mark.parametrize("nodes", [1, 20])
def test_tree_two_streams(B, nodes):
    """Two calls at once, a workspace each, on streams of their own."""
    rng = np.random.default_rng(19)
    cs = [tree_case(B, rng, "bf16", 128, 8, 2, 16, "fused", [nodes, nodes], [3000 + 500 * i, 100], "tree") for i in range(2)]
    ref = [run_tree(B, c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[] for _ in cs]
    for _ in range(10):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                outs[i].append(run_tree(B, c, ws=ref[i][1])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, ref[i][0]) for o in outs[i])
        assert B.specfold_get_status(ref[i][1]) == 0


GUARD = 4096


def guarded(nbytes):
    buf = torch.full((nbytes + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf, buf[GUARD:GUARD + nbytes]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [1, 7, 65])
def test_guards_intact(B, dt, nodes):
    """Nothing is written outside outputs, workspace and the rows' own tokens."""
    rng = np.random.default_rng(20)
    c = tree_case(B, rng, dt, 128, 8, 2, 24, "split", [nodes, 2], [1500, 31], "tree", extra=0)
    cache = c["cache"]
    nws = B.tree_attention_workspace_size(B.dtype_code(DT[dt]), 8, 2, 128, c["nodes"])
    wbuf, ws = guarded(nws)
    ws.zero_()
    obuf, oin = guarded(c["q"].numel() * c["q"].element_size())
    o = oin.view(DT[dt]).view(c["q"].shape)
    keep = cache.k_pool.clone(), cache.v_pool.clone(), c["q"].clone()
    run_tree(B, c, o=o, ws=ws)
    torch.cuda.synchronize()
    for buf in (wbuf, obuf):
        assert (buf[:GUARD] == 0xA5).all() and (buf[-GUARD:] == 0xA5).all()
    assert torch.equal(cache.k_pool, keep[0]) and torch.equal(cache.v_pool, keep[1]) and torch.equal(c["q"], keep[2])
    check_tree(B, c, o, dt)


def far_cache(B, rng, n_kv, hd, page, need, tokens):
    """A cache whose sequences' pages lie at the end of a pool of `tokens`
    tokens; the rest of the pool is never touched."""
    kp, vp = (torch.empty((tokens, n_kv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = [-(-int(n) // page) for n in need]
    table = np.zeros((len(need), max(pages)), np.int32)
    at = tokens // page
    for s, n in enumerate(pages):
        for i in range(n):
            at -= 1
            table[s, i] = at
            kp[at * page:(at + 1) * page] = randn(rng, (page, n_kv, hd), "bf16")
            vp[at * page:(at + 1) * page] = randn(rng, (page, n_kv, hd), "bf16")
    return B.PagedCache(kp, vp, ints(table), page), table


@pytest.mark.parametrize("nodes,n_q", [(3, 8), (40, 16)])
def test_pools_past_two_to_the_31_elements(B, nodes, n_q):
    """Append and attention at element offsets that 32 bits do not hold."""
    rng = np.random.default_rng(22)
    n_kv, hd, page, tokens = 4, 128, 16, 4_300_000 // 16 * 16   # 2.2e9 elements a pool
    counts, ctx = np.array([nodes, 2]), np.array([100, 33])
    start = np.concatenate([[0], np.cumsum(counts)])
    cache, table = far_cache(B, rng, n_kv, hd, page, ctx + counts, tokens)
    T = int(start[-1])
    K, V, q = randn(rng, (T, n_kv, hd), "bf16"), randn(rng, (T, n_kv, hd), "bf16"), randn(rng, (T, n_q, hd), "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.specfold_kv_append(K, V, cache, ints(start), ints(ctx), status=status)
    # the oracle on the used pages alone
    used = table[table > 0]
    slots = torch.from_numpy((used[:, None].astype(np.int64) * page + np.arange(page)).reshape(-1)).cuda()
    small = np.zeros_like(table)
    small[table > 0] = np.arange(len(used))
    kp, vp = cache.k_pool[slots], cache.v_pool[slots]
    for s in range(2):
        for i in range(int(counts[s])):
            t = int(ctx[s]) + i
            at = int(small[s, t // page]) * page + t % page
            assert torch.equal(kp[at], K[int(start[s]) + i]) and torch.equal(vp[at], V[int(start[s]) + i])
    assert int(status) == 0
    c = dict(cache=cache, table=table, start=start, ctx=ctx, parent=None, q=q, T=T, nodes=nodes)
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0

    class Small:
        k_pool, v_pool, page_size = kp, vp, page
    check_tree(B, dict(c, cache=Small, table=small), o, "bf16")


def test_a_batch_too_long_for_one_call_is_refused(B):
    """Sequences whose blocks no 32-bit count holds (tables that name one page
    over and over): nothing is computed, and the status says so."""
    rng = np.random.default_rng(23)
    page = 1 << 19
    kp = torch.zeros((page, 4, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((2, 4096), dtype=torch.int32, device="cuda")
    cache = B.PagedCache(kp, kp, table, page)
    c = dict(cache=cache, start=[0, 1, 2], ctx=[2 ** 31 - 600, 2 ** 31 - 600], parent=None, q=randn(rng, (2, 8, 64), "bf16"),
             nodes=1)
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == B.DEV_BAD_SEQ
    assert (o == 7.0).all()


@pytest.mark.parametrize("dt,nodes", [("bf16", 1), ("bf16", 4), ("bf16", 60), ("f32", 9)])
def test_tree_grows_like_a_sequence(B, dt, nodes):
    """Rows one by one, each appended and attended alone, give what the chain
    gives at once (another split of the keys: rounding apart)."""
    rng = np.random.default_rng(24)
    c = tree_case(B, rng, dt, 64, 4, 2, 8, "fused", [nodes], [45], "none", extra=0)
    whole, _ = run_tree(B, c)
    for i in range(nodes):
        one = dict(c, q=c["q"][i:i + 1], start=[0, 1], ctx=[45 + i], nodes=1)
        o, _ = run_tree(B, one)
        torch.cuda.synchronize()
        assert torch.allclose(o[0].float(), whole[i].float(), rtol=0.03, atol=0.03 if dt == "bf16" else 1e-4)


# ------------------------------------------------------------- a whole step --

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("captured", [False, True])
def test_decoding_steps_together(B, dt, captured):
    """Three steps of a batch as a decoder runs them: norm and rotation,
    append, attention over cache and tree, and the accepted rows committed by a
    second append; eager, or one captured graph replayed with lengths, trees
    and inputs changed in place."""
    rng = np.random.default_rng(21)
    n_q, n_kv, hd, page, S, N, theta = 8, 2, 64, 16, 3, 9, 1e4
    T = S * N
    cap = 80
    cache, table = make_cache(B, rng, dt, hd, n_kv, page, [cap] * S, "fused")
    x = torch.zeros(T, n_q + 2 * n_kv, hd, device="cuda", dtype=DT[dt])
    qr = torch.zeros(T, n_q, hd, device="cuda", dtype=DT[dt])
    o = torch.full((T, n_q, hd), 7.0, device="cuda", dtype=DT[dt])
    gq, gk = randn(rng, (hd,), dt), randn(rng, (hd,), dt)
    start, ctx, parent, pos = ints(np.zeros(S + 1)), ints(np.zeros(S)), ints(np.zeros(T)), ints(np.zeros(T))
    take, tstart, status = ints(np.zeros(T)), ints(np.zeros(S + 1)), torch.zeros(64, dtype=torch.int32, device="cuda")
    ws = B.alloc_workspace(B.tree_attention_workspace_size(B.dtype_code(DT[dt]), n_q, n_kv, hd, N))
    q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]

    def verify():
        B.specfold_qk_norm_rope(q, None, qr, None, gq, None, 1e-6, pos, theta)
        B.specfold_kv_append(k, v, cache, start, ctx, gk=gk, positions=pos, rope_theta=theta, status=status[:1])
        B.specfold_tree_attention(qr, cache, parent, start, ctx, N, o, ws)

    def commit():
        B.specfold_kv_append(k, v, cache, tstart, ctx, gk=gk, rope_theta=theta, rows=take, status=status[:1])

    graphs = None
    if captured:
        verify(), commit()                              # every launch once before the capture
        torch.cuda.synchronize()
        graphs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        for g, f in zip(graphs, (verify, commit)):
            with torch.cuda.graph(g):
                f()
    length = np.array([0, 21, 40])
    for _ in range(3):
        counts = rng.integers(1, N + 1, S)
        st = np.concatenate([[0], np.cumsum(counts)])
        par = np.concatenate([random_tree(rng, int(n), "tree") for n in counts] + [np.zeros(T - st[-1], int)])
        depth = np.zeros(T, int)
        for s in range(S):
            for i in range(counts[s]):
                p = par[st[s] + i]
                depth[st[s] + i] = 0 if p < 0 else depth[st[s] + p] + 1
        at = depth + np.concatenate([np.repeat(length, counts), np.zeros(T - st[-1], int)])
        # the accepted path: the last row's ancestors, oldest first
        picked, tst = [], [0]
        for s in range(S):
            path, i = [], int(counts[s]) - 1
            while i >= 0:
                path.append(int(st[s]) + i)
                i = int(par[st[s] + i])
            picked += path[::-1]
            tst.append(len(picked))
        x.copy_(randn(rng, tuple(x.shape), dt))
        for dst, val in ((start, st), (ctx, length), (parent, par), (pos, at), (tstart, tst),
                         (take, picked + [0] * (T - len(picked)))):
            dst.copy_(ints(val))
        o.fill_(7.0)
        before = host(cache.k_pool), host(cache.v_pool)
        (graphs[0].replay if captured else verify)()
        torch.cuda.synchronize()
        check_append(B, cache, table, before, (k, v, st, length, gk, at, theta, None), dt, T)
        ref, size = orc.norm_rotate(host(q), host(gq), 1e-6, at, theta)
        assert (np.abs(host(qr) - ref) <= rot_bound(dt, ref, size, at)).all()
        check_tree(B, dict(q=qr, cache=cache, table=table, start=st, ctx=length, parent=par), o, dt)
        before = host(cache.k_pool), host(cache.v_pool)
        (graphs[1].replay if captured else commit)()
        torch.cuda.synchronize()
        check_append(B, cache, table, before, (k, v, tst, length, gk, None, theta, picked), dt, T)
        length = length + np.diff(tst)
        assert B.specfold_get_status(ws) == 0 and int(status[0]) == 0
    # what the steps left is what the framework's own paged prefix view reads
    pk = B.PagedPrefix(cache.k_pool, cache.block_table[2], page, int(length[2]))
    assert pk.view().num_pages == cache.k_pool.shape[0] // page


# ------------------------------------------------------------------- edges --

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,n_kv,hd", [(128, 1, 128), (127, 1, 64), (218, 2, 128), (96, 1, 64)])
@pytest.mark.parametrize("counts,ctx", [([1], [300]), ([3, 1, 2], [129, 0, 40])])
def test_tree_widest_groups(B, dt, n_q, n_kv, hd, counts, ctx):
    rng = np.random.default_rng(31)
    c = tree_case(B, rng, dt, hd, n_q, n_kv, 40, "fused", counts, ctx, "tree")
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0
    check_tree(B, c, o, dt)


@pytest.mark.parametrize("nodes,hd", [(4, 128), (5, 128), (8, 128), (9, 128), (4, 64), (5, 64), (8, 64), (9, 64)])
@pytest.mark.parametrize("page", [8, 1000])
def test_tree_on_both_sides_of_the_rules(B, nodes, hd, page):
    """Rows of a head group just within and just past 16 and 32."""
    rng = np.random.default_rng(32)
    c = tree_case(B, rng, "bf16", hd, 8, 2, page, "heads", [nodes, 1, nodes], [999, 2000, 31], "padded")
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0
    check_tree(B, c, o, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [2, 40])
def test_sequences_that_share_one_table(B, dt, nodes):
    """One table row for all sequences (stride 0): the same cache, read by each
    to its own length."""
    rng = np.random.default_rng(33)
    c = tree_case(B, rng, dt, 64, 4, 2, 16, "split", [nodes] * 5, [400, 3, 17, 128, 64], "tree")
    one = c["cache"].block_table[:1].expand(5, -1)
    c["cache"] = B.PagedCache(c["cache"].k_pool, c["cache"].v_pool, one, 16)
    c["table"] = np.repeat(c["table"][:1], 5, axis=0)
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0
    check_tree(B, c, o, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_append_takes_a_row_many_times(B, dt):
    rng = np.random.default_rng(34)
    T = 70
    x = randn(rng, (9, 3, 64), dt)
    cache, table = make_cache(B, rng, dt, 64, 3, 8, [100, 20], "fused")
    rows, start, ctx = np.repeat([8, 0, 8, 3, 3], 14), [0, 55, 70], [45, 5]
    before = host(cache.k_pool), host(cache.v_pool)
    B.specfold_kv_append(x, x, cache, ints(start), ints(ctx), rope_theta=1e4, rows=ints(rows))
    torch.cuda.synchronize()
    assert len(check_append(B, cache, table, before, (x, x, start, ctx, None, None, 1e4, rows), dt, T)) == T


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_calls_on_a_stream_of_their_own(B, dt):
    """stream= takes the work off the current stream, and the order on that
    stream is the calls'."""
    rng = np.random.default_rng(35)
    c = tree_case(B, rng, dt, 64, 4, 2, 16, "fused", [6, 2], [500, 90], "tree", extra=0)
    cache, T = c["cache"], c["T"]
    k = randn(rng, (T, 2, 64), dt)
    g = randn(rng, (64,), dt)
    pos, start, ctx, par = (ints(v) for v in (np.arange(T), c["start"], c["ctx"], c["parent"]))
    keep = cache.k_pool.clone(), cache.v_pool.clone()
    ws = B.alloc_workspace(B.tree_attention_workspace_size(B.dtype_code(DT[dt]), 4, 2, 64, 6))

    def step(stream):
        cache.k_pool.copy_(keep[0]), cache.v_pool.copy_(keep[1])
        qr, o = torch.zeros(T, 4, 64, device="cuda", dtype=DT[dt]), torch.zeros(T, 4, 64, device="cuda", dtype=DT[dt])
        torch.cuda.synchronize()
        for _ in range(3):
            B.specfold_qk_norm_rope(c["q"], None, qr, None, g, None, 1e-6, pos, 1e4, stream=stream)
            B.specfold_kv_append(k, k, cache, start, ctx, gk=g, rope_theta=1e4, stream=stream)
            B.specfold_tree_attention(qr, cache, par, start, ctx, 6, o, ws, stream=stream)
        torch.cuda.synchronize()
        return qr, o, cache.k_pool.clone(), cache.v_pool.clone()

    here, there = step(None), step(torch.cuda.Stream())
    assert all(torch.equal(a, b) for a, b in zip(here, there))


def test_append_then_a_layer_that_reads_the_prefix(B):
    """The verification layer right behind the append that writes its paged
    prefix, no wait between: the same result as with one."""
    from diffusion_branch_speculative_gb300 import synth
    from tests.gpu_cases import DeviceInputs
    inp = synth.make_layer_inputs(synth.small_workload(d=512, n_q=8, n_kv=2, hd=128, F=384, P=500, L=12,
                                                       levels=(1, 3, 4)), seed=8)
    dev = DeviceInputs(inp)
    nb, L, _ = inp.H.shape
    P, page = 500, 16
    pages = -(-P // page)
    pk, pv = (torch.zeros(pages * page, 2, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = ints(np.random.default_rng(36).permutation(pages)[None])
    cache = B.PagedCache(pk, pv, table, page)
    start, ctx = ints([0, P]), ints([0])
    ws = B.alloc_workspace(B.workspace_size(dev.dims, nb, L))
    cw = B.make_weights(dev.W)

    def layer(wait):
        pk.zero_(), pv.zero_()
        out = torch.empty_like(dev.H)
        B.specfold_kv_append(dev.pk, dev.pv, cache, start, ctx)
        if wait:
            torch.cuda.synchronize()
        B.specfold_layer_forward(dev.dims, cw, dev.H, dev.parent, B.PagedPrefix(pk, table[0], page, P),
                                 B.PagedPrefix(pv, table[0], page, P), P, 0.05, out, ws)
        return out

    ref = layer(True)
    plain = torch.empty_like(dev.H)
    B.specfold_layer_forward(dev.dims, cw, dev.H, dev.parent, dev.pk, dev.pv, P, 0.05, plain, ws)
    outs = [layer(False) for _ in range(20)]
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0
    assert torch.equal(ref, plain)
    assert all(torch.equal(o, ref) for o in outs)
