"""Tree attention's tcgen05 form over runs of many pieces: a block of the grid
that goes through several sequences, heads and tiles, through rings of tiles
that wrap, and through scores that rise from block to block.

The oracle is float64 torch, a sequence at a time; the bounds are
test_gpu_cache_ops.py's.  How many units or key blocks a thread block of the
grid gets is held to by counting alone: there is one an SM, so with k times as
many units as SMs some of them has k or more, however the work is cut.
"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from tests.test_gpu_cache_ops import B, E, half_step, run_tree, tree_case

pytestmark = pytest.mark.gpu
TILE, KEYS = 256, 128      # rows and keys of the form's tiles


def grid():
    return torch.cuda.get_device_properties(0).multi_processor_count


def units(c):
    g = c["q"].shape[1] // c["cache"].n_kv
    counts = np.diff(c["start"])
    return int((-(-counts * g // TILE)).sum()) * c["cache"].n_kv


def blocks(c):
    """Key blocks of all units."""
    g = c["q"].shape[1] // c["cache"].n_kv
    counts = np.diff(c["start"])
    return int((-(-counts * g // TILE) * -(-(np.asarray(c["ctx"]) + counts) // KEYS)).sum()) * c["cache"].n_kv


def takes_the_form(c):
    g = c["q"].shape[1] // c["cache"].n_kv
    return c["nodes"] * g > (16 if c["q"].shape[2] == 128 else 32)


def check(c, o):
    """Every row of every sequence; non-finite values of visible tokens included."""
    q, cache, page = c["q"], c["cache"], c["cache"].page_size
    hd, n_kv = q.shape[2], cache.n_kv
    g = q.shape[1] // n_kv
    u = half_step("bf16")
    seen_rows = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    worst = 0.0
    for s in range(len(c["ctx"])):
        a, n, ctx = int(c["start"][s]), int(c["start"][s + 1] - c["start"][s]), int(c["ctx"][s])
        if n == 0:
            continue
        seen_rows[a:a + n] = True
        sees = orc.ancestors(None if c["parent"] is None else c["parent"][a:a + n], n)
        t = np.arange(ctx + n)
        at = torch.from_numpy(c["table"][s][t // page].astype(np.int64) * page + t % page).cuda()
        vis = torch.from_numpy(np.concatenate([np.repeat(sees.any(1)[:, None], ctx, 1), sees], 1)).cuda()   # [n, L]
        k = cache.k_pool[at].double().transpose(0, 1)                                     # [n_kv, L, hd]
        v = cache.v_pool[at].double().transpose(0, 1)
        qs = q[a:a + n].double().view(n, n_kv, g, hd).permute(1, 2, 0, 3)                  # [n_kv, g, n, hd]
        w = torch.einsum("hgid,htd->hgit", qs, k) * hd ** -0.5
        size = torch.einsum("hgid,htd->hgit", qs.abs(), k.abs()).masked_fill(~vis, 0.0).amax() * hd ** -0.5
        w = w.masked_fill(~vis, -np.inf)
        live = vis.any(1)
        w = torch.where(live[:, None], torch.softmax(w, -1), 0.0)
        fin = torch.where(torch.isfinite(v), v, 0.0)
        ref = torch.einsum("hgit,htd->hgid", w, fin)
        spread = torch.einsum("hgit,htd->hgid", w, fin.abs())
        share = 2 * (hd * E * float(size) * 1.45 + 2.0 ** -21) + 4160 * E
        bound = u * ref.abs() + (u + share) * spread * (1 + u) + 1e-30
        vf = vis.double()
        plus, minus, nan = (torch.einsum("it,htd->hid", vf, m.double())[:, None] > 0
                            for m in (v == np.inf, v == -np.inf, torch.isnan(v)))
        got = o[a:a + n].double().view(n, n_kv, g, hd).permute(1, 2, 0, 3)
        odd = (plus | minus | nan).expand_as(got)
        err = torch.where(odd, 0.0, (got - ref).abs() / bound)
        worst = max(worst, float(err.nan_to_num(nan=np.inf).max()))
        want = torch.where(nan | (plus & minus), np.nan, torch.where(plus, np.inf, -np.inf)).expand_as(got)
        assert ((got == want) | (torch.isnan(got) & torch.isnan(want)))[odd].all(), s
        assert worst <= 1.0, (s, worst)
    assert (o[~seen_rows] == 7.0).all()


def run(B, c):
    assert takes_the_form(c)
    o, ws = run_tree(B, c)
    torch.cuda.synchronize()
    assert B.specfold_get_status(ws) == 0
    check(c, o)
    again, _ = run_tree(B, c, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), again.view(torch.int16))
    return o


# rows of a sequence: one tile for both lanes (up to 128 rows of 8 heads), a tile
# of two lanes, two tiles of either kind
MIXED = [1, 2, 5, 16, 17, 20, 32, 33, 40, 49, 64]


@pytest.mark.parametrize("n_q,n_kv,hd,page,layout", [(8, 1, 128, 16, "fused"), (16, 2, 64, 8, "heads"),
                                                     (8, 1, 64, 64, "split"), (24, 3, 128, 24, "split")])
@pytest.mark.parametrize("kind", ["tree", "padded", "none"])
def test_many_short_sequences(B, n_q, n_kv, hd, page, layout, kind):
    """Units of one to three blocks, several a thread block, tiles of one and of
    two lanes in turn, sequences without rows among them."""
    rng = np.random.default_rng(51)
    S = 900 // n_kv
    counts = np.where(rng.random(S) < 0.1, 0, rng.choice(MIXED, S))
    counts[0] = max(MIXED)
    c = tree_case(B, rng, "bf16", hd, n_q, n_kv, page, layout, counts, rng.integers(0, 260, S), kind)
    assert units(c) >= 5 * grid()
    run(B, c)


@pytest.mark.parametrize("hd", [64, 128])
def test_the_most_sequences(B, hd):
    rng = np.random.default_rng(52)
    counts, ctx = rng.choice([0, 1, 3, 8, 9, 40], 1024), rng.integers(0, 200, 1024)
    counts[5] = 40
    c = tree_case(B, rng, "bf16", hd, 16, 1, 16, "split", counts, ctx, "tree")
    assert units(c) >= 6 * grid()
    run(B, c)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nodes", [[5, 5, 4, 5, 5, 3, 5, 5], [40, 33, 20, 36, 17, 40, 3, 40]])
@pytest.mark.parametrize("heads", [(8, 1), (14, 2)])
def test_long_contexts(B, hd, nodes, heads):
    """Twelve blocks and more a thread block: both rings go round several times."""
    rng = np.random.default_rng(53)
    n_q, n_kv = heads
    need = 12 * grid() * KEYS // (len(nodes) * n_kv) + 500
    ctx = need + rng.integers(0, 900, len(nodes))
    c = tree_case(B, rng, "bf16", hd, n_q, n_kv, 32, "split", nodes, ctx, "tree")
    assert blocks(c) >= 12 * grid()
    run(B, c)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nodes", [6, 24])
@pytest.mark.parametrize("order", ["rising", "falling", "shuffled"])
def test_scores_that_step_from_block_to_block(B, hd, nodes, order):
    """A block's scores lie 6 to 7 (9 to 10 in powers of two) above the last one's,
    or below, or anywhere: the accumulators are rescaled in place between blocks,
    in both lanes.  Dimension 0 of the keys is the block's level and of the
    queries sqrt(hd), so that scores are the level and some."""
    rng = np.random.default_rng(54)
    S, n_kv, g = 5, 2, 8
    per = 16 * grid() // (S * n_kv) + 3
    ctx = per * KEYS + rng.integers(0, 100, S)
    c = tree_case(B, rng, "bf16", hd, n_kv * g, n_kv, 64, "split", [nodes] * S, ctx, "tree")
    c["q"].mul_(0.3)
    c["q"][..., 0] = hd ** 0.5
    cache, table = c["cache"], c["table"]
    for s in range(S):
        t = np.arange(int(ctx[s]) + nodes)
        level = 6.5 * (t // KEYS % 12)                  # up to 71.5, then again from 0
        if order == "falling":
            level = level[::-1].copy()
        if order == "shuffled":
            level = rng.permutation(12)[t // KEYS % 12] * 6.5
        at = torch.from_numpy(table[s][t // 64].astype(np.int64) * 64 + t % 64).cuda()
        cache.k_pool[at, :, 0] = torch.from_numpy(level).cuda().bfloat16()[:, None]
    assert blocks(c) >= 16 * grid()
    run(B, c)


@pytest.mark.parametrize("n_q,hd", [(8, 128), (16, 64)])
def test_values_that_are_not_finite_in_many_units(B, n_q, hd):
    """Infinities and NaN among the tree's values, in most of the units that a
    thread block goes through: each reaches the rows that see it and no other."""
    rng = np.random.default_rng(55)
    S = 1000
    counts, ctx = rng.choice(MIXED, S), rng.integers(0, 300, S)
    counts[0] = max(MIXED)
    c = tree_case(B, rng, "bf16", hd, n_q, 1, 8, "fused", counts, ctx, "padded")
    assert units(c) >= 6 * grid()
    odd = np.array([np.inf, -np.inf, np.nan])
    at, dim, val = [], [], []
    for s in range(S):
        for _ in range(int(rng.integers(0, 4))):
            t = int(ctx[s]) + int(rng.integers(counts[s]))
            at.append(int(c["table"][s, t // 8]) * 8 + t % 8)
            dim.append(int(rng.integers(hd)))
            val.append(rng.choice(odd))
    c["cache"].v_pool[torch.tensor(at).cuda(), 0, torch.tensor(dim).cuda()] = torch.tensor(val).cuda().bfloat16()
    run(B, c)
