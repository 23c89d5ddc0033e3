"""Tree attention over lengths that count: batches just inside and just past
the header's limit, and lines of work that 32 bits do not hold.

Contexts of 10^5 to 10^7 tokens come from tables that name one page over and
over.  That page's keys are zeros (a score of 0 for every row); eight marked
pages, spread from the first to the last, score 6 to 9 and carry a value of 16
in a dimension of their own, so that each is some 7 % of a row's weight and a
stretch of the cache that is left out, or gone over twice, shows.  The oracle
is then a closed form in 64 bits: every page times how often the table has it.

Bounds: a score as in test_gpu_cache_ops.py; the output sums one product of 16
keys after the other, each off by at most 2^-22 of the sum (17 terms, cut and not
rounded, at 24 bits), the weights' sum one block after the other.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache_ops import B, E, half_step, ints

pytestmark = pytest.mark.gpu
MARKS = 8
PAGE, HD = 64, 64


def marked_cache(B, rng, n_kv, pages, n_seqs, tail):
    """`pages` pages of context, the same for all sequences (a table stride of
    0), and behind them `tail` pages of their own tokens.  Returns the cache and
    the pages' multiplicities."""
    gen = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 30)))
    total = 1 + MARKS + tail
    # head by head: rows of one head a stretch of memory, which stays in L2
    kp, vp = torch.zeros((2, n_kv, total * PAGE, HD), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    vp[:PAGE] = 0.5 * torch.randn((PAGE, n_kv, HD), device="cuda", generator=gen).bfloat16()
    table = np.zeros(pages + tail, np.int32)
    at = np.unique(np.concatenate([[0, pages - 1], rng.choice(np.arange(1, pages - 1), MARKS - 2, replace=False)]))
    assert len(at) == MARKS
    for m in range(MARKS):
        rows = slice((1 + m) * PAGE, (2 + m) * PAGE)
        kp[rows, :, 0] = 8.0
        vp[rows, :, m] = 16.0
        table[at[m]] = 1 + m
    table[pages:] = 1 + MARKS + np.arange(tail)
    own = slice((1 + MARKS) * PAGE, None)
    kp[own] = torch.randn((tail * PAGE, n_kv, HD), device="cuda", generator=gen).bfloat16()
    vp[own] = torch.randn((tail * PAGE, n_kv, HD), device="cuda", generator=gen).bfloat16()
    cache = B.PagedCache(kp, vp, ints(table)[None].expand(n_seqs, -1), PAGE)
    return cache, np.bincount(table[:pages], minlength=1 + MARKS)


def expected(cache, times, q, n, heads):
    """Rows [n, heads, HD] of one sequence, a chain of n, by key/value head `heads`
    (one a query head): (o, spread)."""
    kp, vp = cache.k_pool[:, heads].double(), cache.v_pool[:, heads].double()      # [tokens, heads, HD]
    own = (1 + MARKS) * PAGE
    tokens = own + n
    w = torch.einsum("ihd,thd->iht", q.double(), kp[:tokens]) / np.sqrt(HD)
    count = torch.from_numpy(np.concatenate([np.repeat(times, PAGE), np.ones(n)])).cuda()
    i, j = torch.arange(n, device="cuda"), torch.arange(tokens, device="cuda") - own
    w = w + torch.log(count)
    w = w.masked_fill((j[None] > i[:, None])[:, None], -np.inf)
    w = torch.softmax(w, -1)
    return torch.einsum("iht,thd->ihd", w, vp[:tokens]), torch.einsum("iht,thd->ihd", w, vp[:tokens].abs())


def check(cache, times, q, o, start, g, blocks, kinds, rng):
    """Sampled sequences and heads against the closed form; blocks: of a chain of
    sums, kinds: (products of 16 keys a block, sums of weights a block)."""
    score = 16.0       # sum |q k| scale: 8 * 9 / 8 of a marked page
    share = 2 * (HD * E * score * 1.45 + 2.0 ** -21) + blocks * (kinds[0] * 2.0 ** -22 + kinds[1] * E)
    u = half_step("bf16")
    n_q, n_seqs = q.shape[1], len(start) - 1
    for s in sorted({0, n_seqs - 1, int(rng.integers(n_seqs))}):
        a, n = int(start[s]), int(start[s + 1] - start[s])
        heads = torch.from_numpy(np.unique(np.concatenate([[0, n_q - 1], rng.integers(0, n_q, 30)]))).cuda()
        ref, spread = expected(cache, times, q[a:a + n][:, heads], n, heads // g)
        got = o[a:a + n][:, heads].double()
        bound = u * ref.abs() + (u + share) * spread * (1 + u)
        assert (ref[..., :MARKS] > 0.3).all()          # a marked page left out shows
        assert float(bound[..., :MARKS].max()) < 0.1
        err = (got - ref).abs()
        assert (err <= bound).all(), float((err / bound).max())


def queries(rng, T, n_q, pages):
    """A marked page scores log(pages) - 1.9 to - 1.4: a share of 0.15 to 0.25 of all other pages'."""
    gen = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 30)))
    q = torch.randn((T, n_q, HD), device="cuda", generator=gen, dtype=torch.bfloat16)
    q[..., 0] = (np.log(pages) - 1.9 + 0.5 * torch.rand((T, n_q), device="cuda", generator=gen)).bfloat16()
    return q


def call(B, cache, q, start, ctx, nodes):
    o = torch.full_like(q, 7.0)
    ws = B.alloc_workspace(B.tree_attention_workspace_size(B.BF16, q.shape[1], cache.n_kv, HD, nodes))
    B.specfold_tree_attention(q, cache, None, ints(start), ints(ctx), nodes, o, ws)
    torch.cuda.synchronize()
    return o, B.specfold_get_status(ws)


def test_one_long_sequence_of_many_heads_is_computed(B):
    """2.5 10^7 blocks, a quarter of the limit, all of one sequence."""
    rng = np.random.default_rng(41)
    n_kv, g, nodes, pages = 4096, 16, 3, 12208
    cache, times = marked_cache(B, rng, n_kv, pages, 1, 1)
    q = queries(rng, nodes, n_kv * g, pages)
    o, status = call(B, cache, q, [0, nodes], [pages * PAGE], nodes)
    assert status == 0
    check(cache, times, q, o, [0, nodes], g, pages * PAGE // 128, (8, 36), rng)


def test_the_limit_is_the_header_s(B):
    """10^8 blocks of 64 keys, head by head, are computed, one more a head is refused."""
    rng = np.random.default_rng(42)
    n_kv, n_seqs, pages = 50, 1000, 2000
    cache, times = marked_cache(B, rng, n_kv, pages - 1, n_seqs, 2)
    q = queries(rng, n_seqs, n_kv, pages)
    start, ctx = np.arange(n_seqs + 1), np.full(n_seqs, (pages - 1) * PAGE)
    o, status = call(B, cache, q, start, ctx, 1)
    assert status == 0
    check(cache, times, q, o, start, 1, pages // 4, (4, 36), rng)
    ctx[rng.integers(n_seqs)] += PAGE
    o, status = call(B, cache, q, start, ctx, 1)
    assert status == B.DEV_BAD_SEQ
    assert (o == 7.0).all()


def test_a_line_of_work_past_32_bits(B):
    """10^8 blocks of 128 keys, each for ten tiles of 256 rows: 5 10^9 places."""
    rng = np.random.default_rng(43)
    n_kv, g, nodes, n_seqs, pages = 256, 64, 40, 32, 2 * 12206
    cache, times = marked_cache(B, rng, n_kv, pages, n_seqs, 1)
    blocks = (pages * PAGE + nodes - 1) // 128 + 1
    assert blocks * n_kv * n_seqs <= 10 ** 8 and blocks * n_kv * n_seqs * (nodes * g // 256) * 5 > 2 ** 32
    start = np.arange(n_seqs + 1) * nodes
    q = queries(rng, n_seqs * nodes, n_kv * g, pages)
    o, status = call(B, cache, q, start, np.full(n_seqs, pages * PAGE), nodes)
    assert status == 0
    check(cache, times, q, o, start, g, blocks, (8, 36), rng)
    marks = o[..., :MARKS]
    assert (marks > 0.2).all() and (marks < 3.0).all()  # every row and head has every marked page
