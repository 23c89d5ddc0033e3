"""Edges of the operators that thin out a paged cache, on the GPU against the
float64 oracle: what is invalid or not finite reaches no further than the header
says.  Bounds as in test_gpu_evict_ops.py."""
import warnings

import numpy as np
import pytest
import torch

from oracle import evict_oracle as orc
from tests.test_gpu_cache_ops import host, ints, make_cache
from tests.test_gpu_evict_ops import B, Weigh, chosen, word  # noqa: F401 (B is the fixture)

pytestmark = pytest.mark.gpu

# rows of a sequence, group, head size, the longest context: one launch of one and two tiles of rows, two launches
# with the scores kept, products computed twice with one and several tiles of rows (fp32: one and several tiles)
FORMS = [(3, 2, 128, 200), (3, 4, 64, 700), (3, 5, 128, 20000), (2, 2, 64, 40000), (30, 4, 128, 300), (70, 8, 64, 500)]


def batch(B, dt, form):
    rows, g, hd, longest = form
    rng = np.random.default_rng(rows * g + hd)
    return Weigh(B, rng, dt, hd, 2 * g, 2, 16, "split", [rows] * 3, [longest, 33, 130], pick=True)


# ------------------------------------------------------------------ weigh --

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("what", ["nan query", "infinite query", "infinite key", "minus infinite key"])
def test_rows_without_a_source_weigh_nothing_whatever_there_is(B, dt, form, what):
    b = batch(B, dt, form)
    rows = form[0]
    pick = np.where(b.rows == 0, 1, b.rows)     # no row of the batch takes the source's first
    pick[[0, rows - 1]] = -1, len(b.q)          # of sequence 0 the first and the last
    pick[rows:2 * rows] = 2 ** 31 - 1           # of sequence 1 all
    b.rows = pick
    b.at = b.at[0], b.at[1], ints(pick)
    if "query" in what:
        b.q[0] = float("nan") if "nan" in what else float("inf")
    else:                                       # a token that only rows without a source see
        for s in (0, 1):
            t = int(b.ctx[s]) + rows - 1
            b.cache.k_pool[int(b.table[s, t // 16]) * 16 + t % 16] = float("inf") if what[0] == "i" else -float("inf")
    before = host(b.w)
    b.call(0.5)
    torch.cuda.synchronize()
    assert B.specfold_get_status(b.ws) == B.DEV_BAD_SEQ
    got = host(b.w)
    assert np.isfinite(got).all()
    assert np.array_equal(got[1, :, :33], 0.5 * before[1, :, :33]) and (got[1, :, 33:33 + rows] == 0).all()
    b.check(before, got, 0.5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 1])
def test_a_row_without_a_softmax_spoils_what_it_sees_alone(B, dt, form, what, at):
    """Scores that are NaN, or all of them infinite: the weights of the tokens that the row sees are NaN, those of the
    rows behind it are not."""
    b = batch(B, dt, form)
    rows, g = form[:2]
    b.q[:, :, 0].abs_()
    b.cache.k_pool[:, :, 0].abs_().add_(0.5)    # an infinity keeps its sign, and comes with no zero
    before = host(b.w)
    _, bound = b.bound(before, 0.75)            # with finite queries: of at least the sums that are left
    b.q[int(b.rows[at]), g - 1, 0] = what       # a row of sequence 0, the last of its first group's heads
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        ref = orc.weigh(host(b.q), host(b.cache.k_pool), b.table, 16, b.start, b.ctx, before, 0.75, b.rows)[0]
    spoilt = np.isnan(ref)
    n = int(b.ctx[0]) + at + 1
    assert spoilt[0, 0, :n].all() and spoilt.sum() == n
    b.call(0.75)
    torch.cuda.synchronize()
    got = host(b.w)
    assert np.array_equal(np.isnan(got), spoilt)
    err = np.abs(got - ref)[~spoilt]
    assert (err <= bound[~spoilt]).all(), err.max()
    assert B.specfold_get_status(b.ws) == 0


@pytest.mark.parametrize("rows,n_q,n_kv,ctx", [(48, 24, 2, 12011), (256, 4, 1, 5003)])
def test_fp32_many_rows_over_a_long_context(B, rows, n_q, n_kv, ctx):
    """Many tiles of rows, each cut over many blocks."""
    b = Weigh(B, np.random.default_rng(rows), "f32", 64, n_q, n_kv, 64, "split", [rows, 1], [ctx, 700])
    before = host(b.w)
    b.call(0.5)
    b.check(before, host(b.w), 0.5)


# ---------------------------------------------------------------- compact --

@pytest.mark.parametrize("sets", [1, 3])
@pytest.mark.parametrize("lengths,keep", [([100, 100, 70], 60), ([9000, 300, 8000], 2000)])
def test_a_token_that_stays_keeps_its_weight(B, sets, lengths, keep):
    """A move from or to a page outside the pool, or past the table: neither keys and values nor the weight."""
    rng = np.random.default_rng(keep + sets)
    cache, table = make_cache(B, rng, "bf16", 64, 3, 8, lengths, "split")
    kept = np.zeros((3, sets, keep), np.int64)
    for s, n in enumerate(lengths):
        for u in range(sets):
            kept[s, u, :min(n, keep)] = chosen(rng, n, min(n, keep))
    kept[2, 0, [20, 21]] = 5, -1                    # entries that move nothing
    bad = table.copy()
    bad[0, 2], bad[0, 9], bad[1, 1] = -3, 10 ** 6, cache.k_pool.shape[0] // 8
    cache.block_table.copy_(ints(bad))
    w = torch.rand(3, sets, max(lengths) + 2, device="cuda")
    before = [host(cache.k_pool), host(cache.v_pool), host(w)]
    n = [min(x, keep) for x in lengths]
    status = word()
    B.specfold_kv_compact(cache, ints(kept), ints(lengths), ints(n), weights=w, status=status)
    torch.cuda.synchronize()
    assert int(status) == B.DEV_BAD_PAGE | B.DEV_BAD_SEQ
    # the definition, a token at a time
    want = [x.copy() for x in before]
    pages = cache.k_pool.shape[0] // 8
    for s in range(3):
        for h in range(3):
            u = h if sets > 1 else 0
            for i in range(n[s]):
                t = int(kept[s, u, i])
                if not i <= t < lengths[s] or not all(0 <= bad[s, x // 8] < pages for x in (i, t)):
                    continue
                to, of = (int(bad[s, x // 8]) * 8 + x % 8 for x in (i, t))
                want[0][to, h], want[1][to, h] = before[0][of, h], before[1][of, h]
                if h < sets:
                    want[2][s, u, i] = before[2][s, u, t]
    for got, ref in zip((cache.k_pool, cache.v_pool, w), want):
        assert np.array_equal(host(got), ref)


# -------------------------------------------------------- binding refusals --

def test_lists_and_weights_of_other_dimensions_are_refused(B):
    cache, _ = make_cache(B, np.random.default_rng(0), "f32", 64, 2, 8, [16], "split")
    n, new, kept, w = ints([16]), ints([4]), ints([[[1, 2, 3, 4]] * 2]), torch.rand(1, 2, 16, device="cuda")
    for bad in (kept[0, 0], kept[0], kept[None]):
        with pytest.raises(ValueError, match="kept"):
            B.specfold_kv_compact(cache, bad, n, new)
        with pytest.raises(ValueError, match="kept"):
            B.specfold_kv_select(w, n, 4, bad, new)
    for bad in (w[0, 0], w[0], w[None]):
        with pytest.raises(ValueError):
            B.specfold_kv_select(bad, n, 4, kept, new)
        with pytest.raises(ValueError, match="weights"):
            B.specfold_kv_compact(cache, kept, n, new, weights=bad)
