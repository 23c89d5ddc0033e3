"""Positions with several axes and the operators that thin out a paged cache, on
the GPU against the float64 oracle (oracle/evict_oracle.py), element by element.

Bounds, with e = 2^-24 and u = finfo(type).eps / 2:
  * rotation: test_gpu_cache_ops.rot_bound, for the same arithmetic.
  * a weight p = 2^(x - m) / l.  x, the score in log2 units, is off by hd e times
    the sum of |q k| scale log2 e, one rounding of it, and log2 e's own (all below
    2 hd e of that sum); m is one of the x as computed, so that only x's own error
    counts, 2^(x - m) has 2^-22 of its own: p's numerator is off by
    d = 2 hd e score + 2^-21 of itself.  l sums such numerators: d again, and e a
    term in a chain no longer than 4096 + 64; one division.  The sum over the rows
    and the group's heads: e a term.  The old weight times decay and the last sum: 2 e
    of either.
  * what is chosen, and what is moved, is equal.
"""
import numpy as np
import pytest
import torch

from oracle import evict_oracle as orc
from tests.test_gpu_cache_ops import DT, E, far_cache, half_step, host, ints, make_cache, randn, rot_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from diffusion_branch_speculative_gb300 import binding
    binding.lib()
    return binding


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------- several axes --

AXES = [(64, [16, 8, 8], False, False), (64, [11, 0, 21], True, False), (128, [16, 24, 24], True, False),
        (128, [16, 24, 24], False, False), (128, [20, 14, 14, 16], True, True), (128, [32, 32], False, True),
        (64, [32], False, True), (128, [1, 63], True, True)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hd,pairs,turn,own", AXES)
@pytest.mark.parametrize("T,n_q,n_kv", [(1, 28, 4), (2, 1, 1), (33, 7, 7), (301, 24, 8), (2500, 3, 1)])
@pytest.mark.parametrize("normed", [False, True])
def test_qk_norm_rope_axes(B, dt, hd, pairs, turn, own, T, n_q, n_kv, normed):
    rng = np.random.default_rng(T + n_q + hd + len(pairs))
    x = randn(rng, (T, n_q + 2 * n_kv, hd), dt, 2.0)
    before = x.clone()
    q, k = x[:, :n_q], x[:, n_q:n_q + n_kv]
    gq, gk = (randn(rng, (hd,), dt), randn(rng, (hd,), dt)) if normed else (None, None)
    pos = rng.integers(0, 1 << 20, (len(pairs), T))
    qo = torch.full((T, n_q + 1, hd), 7.0, device="cuda", dtype=DT[dt])
    ko = torch.full((n_kv, T + 1, hd), 7.0, device="cuda", dtype=DT[dt])
    # rows of positions side by side, or axes
    p = ints(pos) if T % 2 else ints(pos.T).t()
    B.specfold_qk_norm_rope_axes(q, k, qo[:, :n_q], ko[:, :T].transpose(0, 1), B.RopeAxes(1e4, pairs, turn, own), p,
                                 gq=gq, gk=gk, eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(x, before) and (qo[:, n_q] == 7.0).all() and (ko[:, T] == 7.0).all()
    for got, src, g in ((qo[:, :n_q], q, gq), (ko[:, :T].transpose(0, 1), k, gk)):
        ref, size = orc.norm_rotate_axes(host(src), None if g is None else host(g), 1e-5, pos, pairs, turn, 1e4, own)
        err = np.abs(host(got) - ref)
        assert (err <= rot_bound(dt, ref, size, pos.max(0))).all(), err.max()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_axes_alike_are_the_single_position(B, dt):
    rng = np.random.default_rng(3)
    x, g = randn(rng, (77, 12, 128), dt), randn(rng, (128,), dt)
    pos = ints(rng.integers(-1000, 1 << 30, 77))
    a, b = torch.empty_like(x[:, :8]), torch.empty_like(x[:, 8:])
    B.specfold_qk_norm_rope(x[:, :8], x[:, 8:], a, b, g, g, 1e-6, pos, 1e6)
    for pairs, turn in (([64], False), ([16, 24, 24], True), ([10, 20, 30, 4], False)):
        c, d = torch.empty_like(a), torch.empty_like(b)
        axes = B.RopeAxes(1e6, pairs, in_turn=turn)
        B.specfold_qk_norm_rope_axes(x[:, :8], x[:, 8:], c, d, axes, pos[None].expand(len(pairs), -1), gq=g, gk=g)
        # frequencies of the one are powers by steps, of the other pow: the angles differ by less than 2^-12 of a
        # turn's 32-bit step even at 2^30, the results by a rounding
        for y, z in ((a, c), (b, d)):
            size = host(y[..., :64]).__abs__() + host(y[..., 64:]).__abs__()
            bound = 2 * half_step(dt) * np.abs(host(y)) + 4e-6 * np.concatenate([size] * 2, -1) * 2 + 1e-30
            assert (np.abs(host(y) - host(z)) <= bound).all()


def test_axes_far_positions_and_in_place(B):
    pos = np.array([[0, 1, -1, 1 << 20, (1 << 31) - 1, -(1 << 31)], [5, -(1 << 31), (1 << 31) - 1, 77, -3, 0]])
    rng = np.random.default_rng(4)
    q = randn(rng, (6, 3, 128), "f32")
    ref, size = orc.norm_rotate_axes(host(q), None, 0.0, pos, [30, 34], True, 5e6, True)
    B.specfold_qk_norm_rope_axes(q, None, q, None, B.RopeAxes(5e6, [30, 34], True, True), ints(pos))
    assert (np.abs(host(q) - ref) <= rot_bound("f32", ref, size, np.abs(pos).max(0))).all()
    B.specfold_qk_norm_rope_axes(q[:0], None, q[:0], None, B.RopeAxes(5e6, [30, 34]), ints(pos)[:, :0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hd,pairs,turn,own", AXES[::2])
@pytest.mark.parametrize("page,layout,form", [(8, "fused", "plain"), (24, "heads", "normed"), (64, "split", "picked")])
def test_kv_append_axes(B, dt, hd, pairs, turn, own, page, layout, form):
    rng = np.random.default_rng(page + hd)
    counts, ctx, n_kv = [3, 0, 1, 41, 0, 2], [0, 5, 63, 130, 9, 23], 3
    start = np.concatenate([[0], np.cumsum(counts)])
    T = int(start[-1]) + 4
    src = 2 * T if form == "picked" else T
    x = randn(rng, (src, 2 * n_kv + 1, hd), dt)
    K, V = x[:, :n_kv], x[:, n_kv + 1:]
    cache, table = make_cache(B, rng, dt, hd, n_kv, page, np.array(ctx) + counts, layout)
    gk = randn(rng, (hd,), dt) if form == "normed" else None
    pos = rng.integers(0, 30000, (len(pairs), T))
    rows = rng.permutation(src)[:T] if form == "picked" else None
    kp, vp = host(cache.k_pool), host(cache.v_pool)
    bound, status = np.zeros_like(kp), word()
    from oracle.cache_oracle import slot_of
    for s, c in enumerate(ctx):
        for t in range(start[s], start[s + 1]):
            at = slot_of(table, page, kp.shape[0] // page, s, c + t - start[s])
            r = t if rows is None else rows[t]
            y, size = orc.norm_rotate_axes(host(K[r])[None], None if gk is None else host(gk), 1e-6, pos[:, t:t + 1],
                                           pairs, turn, 5e5, own)
            kp[at], vp[at] = y[0], host(V[r])
            bound[at] = half_step(dt) * np.abs(y[0]) + 2.1e-6 * size[0]
    B.specfold_kv_append_axes(K, V, cache, ints(start), ints(ctx), B.RopeAxes(5e5, pairs, turn, own), ints(pos), gk=gk,
                              rows=None if rows is None else ints(rows), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert np.array_equal(host(cache.v_pool), vp)
    assert (np.abs(host(cache.k_pool) - kp) <= bound).all()


# -------------------------------------------------------------- weigh --

class Weigh:
    """A batch to weigh: its cache, queries, weights and a call."""

    def __init__(self, B, rng, dt, hd, n_q, n_kv, page, layout, counts, ctx, pick=False, tail=3, slack=5, qscale=1.5):
        self.B, self.dt, self.counts, self.ctx = B, dt, np.array(counts), np.array(ctx)
        self.start = np.concatenate([[0], np.cumsum(counts)])
        self.T = int(self.start[-1]) + tail
        self.cache, self.table = make_cache(B, rng, dt, hd, n_kv, page, self.ctx + self.counts, layout, widen=1)
        src = 2 * self.T if pick else self.T
        self.q = randn(rng, (src, n_q + 1, hd), dt, qscale)[:, :n_q]
        self.rows = rng.permutation(src)[:self.T] if pick else None
        self.max_rows = max(1, int(self.counts.max()))
        self.tokens = int((self.ctx + self.counts).max()) + slack
        self.w = torch.from_numpy(rng.random((len(ctx), n_kv, self.tokens + 2)).astype(np.float32)).cuda()[:, :, 1:-1]
        self.n_q, self.n_kv, self.hd = n_q, n_kv, hd
        n = B.kv_weigh_workspace_size(B.dtype_code(DT[dt]), self.T, self.max_rows, n_q, n_kv, hd, len(ctx), self.tokens)
        assert n > 0
        self.ws = B.alloc_workspace(n)
        self.at = ints(self.start), ints(self.ctx), None if self.rows is None else ints(self.rows)

    def call(self, decay=1.0, scale=0.0, w=None, stream=None):
        start, ctx, rows = self.at
        self.B.specfold_kv_weigh(self.q, self.cache, start, ctx, self.max_rows, self.w if w is None else w, self.ws,
                                 decay=decay, scale=scale, rows=rows, stream=stream)

    def bound(self, before, decay, scale=0.0):
        """The oracle's weights and how far a call's may be off."""
        ref, new, score = orc.weigh(host(self.q), host(self.cache.k_pool), self.table, self.cache.page_size, self.start,
                                    self.ctx, before, decay, self.rows, scale)
        terms = int(self.counts.max()) * self.n_q // self.n_kv
        d = 2 * self.hd * E * score + 2.0 ** -21
        return ref, (2 * d + (min(int(self.ctx.max()) + 300, 4160) + terms + 4) * E) * new + 3 * E * np.abs(ref) + 1e-37

    def check(self, before, got, decay, scale=0.0):
        ref, bound = self.bound(before, decay, scale)
        err = np.abs(got - ref)
        assert (err <= bound).all(), (err.max(), (err / bound).max())


GEOMETRY = [(28, 4, 128, 16, "fused"), (24, 8, 128, 64, "split"), (4, 2, 64, 24, "heads"), (7, 7, 64, 8, "fused"),
            (12, 1, 128, 32, "heads"), (20, 1, 64, 256, "split")]
BATCHES = [([1], [0]), ([1], [1]), ([1], [700]), ([5], [0]), ([2, 0, 1, 9], [15, 4, 16, 333]),
           ([1, 1, 1, 1, 1], [127, 128, 129, 0, 1023]), ([40, 33, 1], [250, 0, 1100])]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,n_kv,hd,page,layout", GEOMETRY)
@pytest.mark.parametrize("counts,ctx", BATCHES)
@pytest.mark.parametrize("decay,pick", [(0.0, False), (1.0, True), (0.75, False)])
def test_kv_weigh(B, dt, n_q, n_kv, hd, page, layout, counts, ctx, decay, pick):
    rng = np.random.default_rng(sum(ctx) + sum(counts) + n_q + hd)
    b = Weigh(B, rng, dt, hd, n_q, n_kv, page, layout, counts, ctx, pick)
    if decay == 0.0:
        b.w.fill_(float("nan"))     # not read
    before = host(b.w)
    b.call(decay)
    torch.cuda.synchronize()
    assert B.specfold_get_status(b.ws) == 0
    got = host(b.w)
    if decay == 0.0:
        for s in range(len(ctx)):
            n = ctx[s] + counts[s] if counts[s] else 0
            assert np.isnan(got[s, :, n:]).all() and not np.isnan(got[s, :, :n]).any()
        before, got = np.nan_to_num(before), np.nan_to_num(got)
    b.check(before, got, decay)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,n_kv,hd", [(128, 1, 128), (127, 1, 64), (218, 2, 128), (96, 1, 64)])
@pytest.mark.parametrize("counts,ctx", [([1], [300]), ([3, 1, 2], [129, 0, 40]), ([17], [65])])
def test_kv_weigh_widest_groups(B, dt, n_q, n_kv, hd, counts, ctx):
    b = Weigh(B, np.random.default_rng(n_q + hd), dt, hd, n_q, n_kv, 16, "split", counts, ctx)
    before = host(b.w)
    b.call(0.5)
    b.check(before, host(b.w), 0.5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,n_kv,hd", [(4, 2, 64), (14, 2, 128)])
@pytest.mark.parametrize("rows", [2, 3, 4, 5, 8, 16, 18, 19, 36, 37, 73, 256])
def test_kv_weigh_row_counts(B, dt, n_q, n_kv, hd, rows):
    b = Weigh(B, np.random.default_rng(rows), dt, hd, n_q, n_kv, 16, "fused", [rows, 1, max(1, rows // 2)], [90, 5, 260])
    before = host(b.w)
    b.call(1.0)
    b.check(before, host(b.w), 1.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n_q", [(1, 8), (6, 8), (48, 24)])
def test_kv_weigh_long_context(B, dt, rows, n_q):
    if dt == "f32":
        rows = min(rows, 6)
    b = Weigh(B, np.random.default_rng(rows), dt, 128, n_q, 2, 64, "split", [rows], [20011])
    before = host(b.w)
    b.call(1.0)
    b.check(before, host(b.w), 1.0)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("longest", [7000, 12000, 16385, 26011, 32767])
@pytest.mark.parametrize("rows,g", [(1, 7), (2, 4), (3, 5)])
def test_kv_weigh_long_decoding(B, hd, longest, rows, g):
    """Few rows of sequences whose slices take more and more warps of a cluster, most of them empty."""
    b = Weigh(B, np.random.default_rng(longest), "bf16", hd, 4 * g, 4, 16, "split", [rows, 1, rows, 0, 1, rows],
              [longest - rows, 100, longest // 2, 7, 0, 4095])
    before = host(b.w)
    b.call(0.5)
    b.check(before, host(b.w), 0.5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,g,hd", [(64, 8, 64), (57, 9, 128), (256, 5, 64), (40, 40, 64)])
def test_kv_weigh_groups_of_rows(B, dt, rows, g, hd):
    b = Weigh(B, np.random.default_rng(rows), dt, hd, g, 1, 16, "split", [rows, 1, 7], [70, 3, 130])
    before = host(b.w)
    b.call(0.75)
    b.check(before, host(b.w), 0.75)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("counts", [[40, 17, 5, 90], [3, 200, 33, 16], [65, 64, 63, 32], [16, 8, 15, 7]])
def test_kv_weigh_runs_of_many_blocks(B, hd, counts):
    """Of one, two and more tiles of rows a head group, a run of blocks passing from one to the next."""
    b = Weigh(B, np.random.default_rng(hd), "bf16", hd, 64, 8, 16, "split", counts, [9000, 7011, 6100, 10007])
    before = host(b.w)
    b.call(0.5)
    b.check(before, host(b.w), 0.5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_kv_weigh_rows_in_parts(B, dt):
    """Rows weighed a part at a time, each behind the tokens of the parts before."""
    b = Weigh(B, np.random.default_rng(3), dt, 64, 4, 2, 16, "fused", [30, 12], [100, 9])
    before = host(b.w)
    got = b.w.clone()
    for lo, hi in ((0, 5), (5, 12), (12, 30)):
        n = [min(hi, c) - min(lo, c) for c in b.counts]
        rows = ints(np.concatenate([b.start[s] + np.arange(min(lo, b.counts[s]), min(hi, b.counts[s])) for s in range(2)]))
        ctx = ints(b.ctx + np.minimum(lo, b.counts))
        B.specfold_kv_weigh(b.q, b.cache, ints(np.concatenate([[0], np.cumsum(n)])), ctx, b.max_rows, got, b.ws,
                            decay=0.5 if lo == 0 else 1.0, rows=rows)
    ref, bound = b.bound(before, 0.5)
    assert (np.abs(host(got) - ref) <= 2 * bound).all()     # two more roundings of the sums


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_kv_weigh_many_sequences(B, dt):
    rng = np.random.default_rng(8)
    counts, ctx = rng.integers(0, 4, 1024), rng.integers(0, 40, 1024)
    b = Weigh(B, rng, dt, 64, 4, 2, 8, "fused", counts, ctx)
    before = host(b.w)
    b.call(1.0)
    b.check(before, host(b.w), 1.0)
    assert B.specfold_get_status(b.ws) == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.01])
@pytest.mark.parametrize("rows", [2, 50])
def test_kv_weigh_scale(B, dt, scale, rows):
    b = Weigh(B, np.random.default_rng(9), dt, 128, 8, 2, 16, "fused", [rows, 1], [300, 77], qscale=0.5)
    before = host(b.w)
    b.call(1.0, scale=scale)
    b.check(before, host(b.w), 1.0, scale)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,g", [(1, 7), (5, 2), (70, 4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), -3e38])
def test_kv_weigh_unseen_keys_change_nothing(B, dt, rows, g, bad):
    b = Weigh(B, np.random.default_rng(rows), dt, 128, 2 * g, 2, 16, "split", [rows, rows], [45, 130])
    w0 = b.w.clone()
    b.call(1.0)
    ref = b.w.clone()
    # every pool token that no sequence holds, the pages' ends among them
    pool = b.cache.k_pool
    held = torch.zeros(pool.shape[0], dtype=torch.bool)
    for s in range(2):
        t = np.arange(b.ctx[s] + b.counts[s])
        held[b.table[s, t // 16] * 16 + t % 16] = True
    pool[~held.cuda()] = bad
    b.w.copy_(w0)
    b.call(1.0)
    torch.cuda.synchronize()
    assert torch.equal(b.w, ref)
    # the last row's key is seen by that row alone
    at = b.table[0, (45 + rows - 1) // 16] * 16 + (45 + rows - 1) % 16
    if rows > 1:
        b.q.copy_(b.q.abs())
        b.w.copy_(w0)
        b.call(1.0)
        ref = b.w.clone()
        pool[at] = -float("inf") if bad == bad else bad
        b.w.copy_(w0)
        b.call(1.0)
        torch.cuda.synchronize()
        got = host(b.w)[0]
        if bad != bad:
            assert np.isnan(got[:, :45 + rows]).all()
        else:       # a score of minus infinity: a weight of zero, and the others' as they are
            assert (got[:, 45 + rows - 1] == 0).all() and np.isfinite(got).all()
            assert abs((got[:, :45] - host(w0)[0, :, :45]).sum() + got[:, 45:45 + rows].sum() - 2 * g * rows) < 1e-2
        assert torch.equal(b.w[1], ref[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 60])
def test_kv_weigh_reports_and_survives_bad_entries(B, dt, rows):
    rng = np.random.default_rng(rows)
    b = Weigh(B, rng, dt, 64, 4, 2, 16, "fused", [rows] * 3, [70, 33, 90])
    before = host(b.w)

    def run(start=None, ctx=None, table=None, picked=None, w=None):
        b.w.copy_(torch.from_numpy(before.astype(np.float32)))
        if table is not None:
            b.cache.block_table.copy_(ints(table))
        B.specfold_kv_weigh(b.q, b.cache, ints(b.start if start is None else start), ints(b.ctx if ctx is None else ctx),
                            b.max_rows, b.w if w is None else w, b.ws, rows=None if picked is None else ints(picked))
        torch.cuda.synchronize()
        b.cache.block_table.copy_(ints(b.table))
        return B.specfold_get_status(b.ws), host(b.w)

    ok, good = run()
    assert ok == 0
    # without one of its sequences a batch is cut elsewhere, and sums come in another order: either
    # result is within the bound of the exact one, so they differ by twice that at most
    apart = 2 * b.bound(before, 1.0)[1]
    for ctx in ([70, -1, 90], [70, 2 ** 31 - 1, 90], [70, b.tokens - rows + 1, 90]):
        st, got = run(ctx=ctx)
        assert st == B.DEV_BAD_SEQ and np.array_equal(got[1], before[1])
        assert (np.abs(got - good)[[0, 2]] <= apart[[0, 2]]).all()
    for start in ([0, rows, 3 * rows, 2 * rows], [0, rows, 2 * rows, b.T + 1], [-1, rows, 2 * rows, 3 * rows]):
        st, got = run(start=start)
        assert st & B.DEV_BAD_SEQ
    # a page outside the pool, and a token past the table: keys of zeros
    t = b.table.copy()
    t[0, 1] = 10 ** 6
    st, got = run(table=t)
    assert st == B.DEV_BAD_PAGE and np.array_equal(got[1:], good[1:])
    zero = b.cache.k_pool.clone()
    page = b.table[0, 1]
    b.cache.k_pool[page * 16:page * 16 + 16] = 0
    st, want = run()
    b.cache.k_pool.copy_(zero)
    assert st == 0 and np.array_equal(got[0], want[0])
    # a picked row outside the source weighs nothing
    pick = np.arange(b.T)
    pick[0] = b.T
    st, got = run(picked=pick)
    assert st == B.DEV_BAD_SEQ and np.array_equal(got[1:], good[1:])
    gain = got[0, :, :70].sum() - before[0, :, :70].sum() + got[0, :, 70:70 + rows].sum()
    assert abs(gain - 4 * (rows - 1)) < 1e-2


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 6, 48])
def test_kv_weigh_repeats_bit_for_bit(B, dt, rows):
    b = Weigh(B, np.random.default_rng(rows), dt, 128, 8, 2, 16, "split", [rows, 1, rows], [3000, 7, 411])
    got = []
    for _ in range(5):
        w = torch.zeros_like(b.w)
        b.call(1.0, w=w)
        got.append(w)
    torch.cuda.synchronize()
    assert all(torch.equal(x, got[0]) for x in got)


@pytest.mark.parametrize("longest", [7000, 14000, 28000])
@pytest.mark.parametrize("rows", [2, 4])
@pytest.mark.parametrize("n_kv", [4, 16])
def test_kv_weigh_long_decoding_edges(B, n_kv, longest, rows):
    """Clusters of few and many warps: the same bits again, unseen keys, a bad page, a bad row, a bad length."""
    b = Weigh(B, np.random.default_rng(longest), "bf16", 64, 4 * n_kv, n_kv, 16, "split", [rows] * 6,
              [longest, 33, longest // 3, 0, 5000, longest - 700])
    # One launch keeps nothing in the workspace and cuts no sequence by the others' lengths.  Two do:
    # without one of its sequences the others' sums come in another order, and either result is
    # within the bound of the exact one.
    apart = None
    if B.kv_weigh_workspace_size(B.BF16, b.T, rows, 4 * n_kv, n_kv, 64, 6, b.tokens) != 256:
        apart = 2 * b.bound(host(b.w), 1.0)[1]
    w0 = b.w.clone()

    def run(ctx=None, picked=None):
        b.w.copy_(w0)
        B.specfold_kv_weigh(b.q, b.cache, b.at[0], b.at[1] if ctx is None else ints(ctx), rows, b.w, b.ws,
                            rows=None if picked is None else ints(picked))
        torch.cuda.synchronize()
        return B.specfold_get_status(b.ws), b.w.clone()

    ok, good = run()
    assert ok == 0 and torch.equal(run()[1], good)
    held = torch.zeros(b.cache.k_pool.shape[0], dtype=torch.bool)
    for s in range(6):
        t = np.arange(b.ctx[s] + rows)
        held[b.table[s, t // 16] * 16 + t % 16] = True
    b.cache.k_pool[~held.cuda()] = float("nan")
    st, got = run()
    assert st == 0 and torch.equal(got, good)
    # sequence 2 is longer than its weights: no other one's change
    st, got = run(ctx=[longest, 33, b.tokens, 0, 5000, longest - 700])
    assert st == B.DEV_BAD_SEQ and torch.equal(got[2], w0[2])
    others = [0, 1, 3, 4, 5]
    if apart is None:
        assert torch.equal(got[others], good[others])
    else:
        assert (np.abs(host(got) - host(good))[others] <= apart[others]).all()
    # a picked row outside the source weighs nothing
    pick = np.arange(b.T)
    pick[0] = -1
    st, got = run(picked=pick)
    assert st == B.DEV_BAD_SEQ and torch.equal(got[1:], good[1:])
    gain = (got[0] - w0[0])[:, :longest].double().sum() + got[0, :, longest:longest + rows].double().sum()
    assert abs(float(gain) - 4 * n_kv * (rows - 1)) < 1e-2
    # a page outside the pool reads as zeros
    table = b.cache.block_table.clone()
    b.cache.block_table[4, 100] = -3
    st, got = run()
    b.cache.block_table.copy_(table)
    assert st == B.DEV_BAD_PAGE and torch.equal(got[[0, 1, 2, 3, 5]], good[[0, 1, 2, 3, 5]])
    page = b.table[4, 100]
    b.cache.k_pool[page * 16:page * 16 + 16] = 0
    st, want = run()
    assert st == 0 and torch.equal(got, want)


# ------------------------------------------------------------- select --

def run_select(B, w, lengths, keep, sinks=0, recent=0, cap=None):
    S, U = w.shape[:2]
    kept = torch.full((S, U, (cap or keep) + 2), -7, dtype=torch.int32, device="cuda")
    new_len, status = ints([99] * S), word()
    B.specfold_kv_select(w, ints(lengths), keep, kept[:, :, 1:-1], new_len, sinks, recent, status)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), new_len.cpu().numpy(), int(status)


def check_select(B, w, lengths, keep, sinks=0, recent=0, cap=None):
    kept, new_len, status = run_select(B, w, lengths, keep, sinks, recent, cap)
    ref = orc.select(w.cpu().numpy(), lengths, keep, sinks, recent)
    for s, sets in enumerate(ref):
        n = 0 if sets is None else min(int(lengths[s]), keep)
        assert new_len[s] == (-1 if sets is None else n)
        for u in range(w.shape[1]):
            if n:
                assert np.array_equal(kept[s, u, 1:n + 1], sets[u]), (s, u)
            assert (kept[s, u, n + 1:] == -7).all() and kept[s, u, 0] == -7
    assert status == (B.DEV_BAD_SEQ if None in ref else 0)


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (50, 0, 0), (50, 4, 16), (50, 10, 40),
                                               (64, 0, 64), (513, 3, 30)])
@pytest.mark.parametrize("kind", ["spread", "few values", "equal", "signs"])
def test_kv_select(B, keep, sinks, recent, kind):
    rng = np.random.default_rng(keep + sinks)
    lengths = [0, 1, keep - 1, keep, keep + 1, 700, 1337, 1400]
    w = np.exp(3 * rng.standard_normal((len(lengths), 3, 1400))).astype(np.float32)
    if kind == "few values":
        w = rng.integers(0, 4, w.shape).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "signs":
        w = rng.standard_normal(w.shape).astype(np.float32)
        odd = rng.integers(0, 12, w.shape)
        for i, v in enumerate((np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45)):
            w[odd == i] = v
    check_select(B, torch.from_numpy(w).cuda(), lengths, keep, sinks, recent)


@pytest.mark.parametrize("tokens", [5000, 16384, 16385, 40001, 131071, 300000, 700001])
@pytest.mark.parametrize("S,U", [(1, 1), (3, 2)])
def test_kv_select_long(B, tokens, S, U):
    rng = np.random.default_rng(tokens)
    w = np.exp(2 * rng.standard_normal((S, U, tokens))).astype(np.float32)
    w[:, :, rng.integers(0, tokens, tokens // 3)] = 0.0
    lengths = [tokens, tokens * 2 // 3, 4097][:S]
    for keep, sinks, recent in ((4096, 4, 512), (1, 0, 0), (tokens * 4 // 5, 0, 100)):
        kept, new_len, status = run_select(B, torch.from_numpy(w).cuda(), lengths, keep, sinks, recent)
        assert status == 0
        for s, n in enumerate(lengths):
            assert new_len[s] == min(n, keep)
            for u in range(U):
                got = kept[s, u, 1:new_len[s] + 1]
                if n <= keep:
                    assert np.array_equal(got, np.arange(n))
                    continue
                mid = np.arange(sinks, n - recent)
                best = np.sort(mid[np.argsort(-w[s, u, mid], kind="stable")[: keep - sinks - recent]])
                assert np.array_equal(got, np.concatenate([np.arange(sinks), best, np.arange(n - recent, n)]))


@pytest.mark.parametrize("tokens,S,U", [(26011, 40, 5), (60007, 40, 5), (110003, 26, 6)])
def test_kv_select_many_long(B, tokens, S, U):
    """More sets than SMs, of more keys than two blocks of an SM hold."""
    rng = np.random.default_rng(tokens)
    w = torch.from_numpy(rng.random((S, U, tokens), dtype=np.float32) ** 4).cuda()
    lengths = rng.integers(1, tokens + 1, S)
    lengths[:3] = [tokens, 2048, 2049]
    check_select(B, w, lengths, 2048, 4, 64)


def test_kv_select_many_and_strided(B):
    rng = np.random.default_rng(1)
    S, U = 1024, 3
    big = torch.from_numpy(rng.random((U, S, 77)).astype(np.float32)).cuda()
    w = big.transpose(0, 1)[:, :, 3:70]
    check_select(B, w, rng.integers(0, 68, S), 20, 2, 5, cap=31)
    # one row of weights for every set
    check_select(B, w[:5, :1].expand(5, 4, 67), [67, 30, 20, 21, 0], 20)


def test_kv_select_bad_lengths(B):
    w = torch.rand(4, 2, 50, device="cuda")
    check_select(B, w, [50, 51, -1, 30], 10, 1, 1)
    check_select(B, w, [2 ** 31 - 1, -2 ** 31, 50, 10], 10)


# ------------------------------------------------------------ compact --

def chosen(rng, n, keep, first=0):
    """`keep` of n tokens, ascending, the first ones among them."""
    rest = np.sort(rng.choice(np.arange(first, n), keep - first, replace=False))
    return np.concatenate([np.arange(first), rest])


def run_compact(B, rng, dt, hd, n_kv, page, layout, lengths, keep, sets, weights=True, first=0):
    cache, table = make_cache(B, rng, dt, hd, n_kv, page, lengths, layout)
    n = np.minimum(lengths, keep)
    kept = np.full((len(lengths), sets, max(1, int(n.max())) + 3), -5)
    for s in range(len(lengths)):
        for u in range(sets):
            kept[s, u, :n[s]] = chosen(rng, lengths[s], n[s], min(first, n[s]))
    w = torch.rand(len(lengths), sets, max(1, max(lengths)) + 2, device="cuda")
    before = [x.float().cpu().numpy() for x in (cache.k_pool, cache.v_pool, w)]
    bits = cache.k_pool.clone(), cache.v_pool.clone()
    status = word()
    B.specfold_kv_compact(cache, ints(kept), ints(lengths), ints(n), weights=w if weights else None, status=status)
    torch.cuda.synchronize()
    kp, vp, wr = orc.compact(before[0], before[1], table, page, kept, lengths, n, before[2])
    assert np.array_equal(cache.k_pool.float().cpu().numpy(), kp)
    assert np.array_equal(cache.v_pool.float().cpu().numpy(), vp)
    assert np.array_equal(w.cpu().numpy(), wr if weights else before[2])
    assert int(status) == 0
    return bits


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hd,n_kv", [(64, 2), (128, 4), (128, 7)])
@pytest.mark.parametrize("page,layout", [(8, "fused"), (24, "split"), (64, "heads")])
@pytest.mark.parametrize("keep,first", [(1, 0), (63, 0), (64, 3), (65, 65), (257, 100)])
@pytest.mark.parametrize("one_set", [False, True])
def test_kv_compact(B, dt, hd, n_kv, page, layout, keep, first, one_set):
    rng = np.random.default_rng(keep + page)
    lengths = np.array([0, 1, keep, keep + 1, keep + 200, 300, 64])
    run_compact(B, rng, dt, hd, n_kv, page, layout, lengths, keep, 1 if one_set else n_kv, first=first)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,keep", [([5000], 4999), ([5000], 4097), ([9000, 300, 8000], 2000), ([33000], 1000),
                                          ([2080] * 40, 2048)])
def test_kv_compact_long(B, dt, lengths, keep):
    run_compact(B, np.random.default_rng(keep), dt, 128, 2, 16, "fused", np.array(lengths), keep, 2, weights=len(lengths) > 1)


def test_kv_compact_many_sequences(B):
    rng = np.random.default_rng(2)
    run_compact(B, rng, "bf16", 64, 1, 8, "split", rng.integers(0, 90, 1024), 40, 1)


def test_kv_compact_moves_bits(B):
    rng = np.random.default_rng(3)
    cache, table = make_cache(B, rng, "bf16", 64, 1, 8, [40], "split")
    nan = torch.tensor([0x7fc1, -63, 0x7f80, 1], dtype=torch.int16, device="cuda").view(torch.bfloat16)
    at = table[0, 30 // 8] * 8 + 30 % 8
    cache.k_pool[at, 0, :4] = nan
    B.specfold_kv_compact(cache, ints([[[30]]]), ints([40]), ints([1]))
    to = table[0, 0] * 8
    assert torch.equal(cache.k_pool[to, 0, :4].view(torch.int16), nan.view(torch.int16))


def test_kv_compact_bad_entries(B):
    rng = np.random.default_rng(4)
    cache, table = make_cache(B, rng, "f32", 64, 2, 8, [100] * 3, "split")
    k0, v0 = cache.k_pool.clone(), cache.v_pool.clone()
    good = np.stack([np.stack([chosen(rng, 100, 60) for _ in range(2)]) for _ in range(3)])

    def run(kept=good, lengths=(100,) * 3, n=(60,) * 3, tab=None, w=None):
        cache.k_pool.copy_(k0)
        cache.v_pool.copy_(v0)
        if tab is not None:
            cache.block_table.copy_(ints(tab))
        status = word()
        B.specfold_kv_compact(cache, ints(kept), ints(lengths), ints(n), weights=w, status=status)
        torch.cuda.synchronize()
        cache.block_table.copy_(ints(table))
        return int(status), host(cache.k_pool), host(cache.v_pool)

    ref_k, ref_v, _ = orc.compact(host(k0), host(v0), table, 8, good, [100] * 3, [60] * 3)
    st, k, v = run()
    assert st == 0 and np.array_equal(k, ref_k) and np.array_equal(v, ref_v)
    tokens = lambda s: table[s, np.arange(100) // 8] * 8 + np.arange(100) % 8
    # the whole sequence is left alone, the others are moved
    for lengths, n in (((100, -1, 100), (60, -1, 60)), ((100, 50, 100), (60, 60, 60)), ((100, 100, 100), (60, 61, 60)),
                       ((100, 100, 100), (60, -1, 60))):
        st, k, v = run(lengths=lengths, n=n)
        assert st == B.DEV_BAD_SEQ
        assert np.array_equal(k[tokens(1)], host(k0)[tokens(1)]) and np.array_equal(k[tokens(2)], ref_k[tokens(2)])
    # more tokens than weights
    st, k, v = run(w=torch.rand(3, 2, 99, device="cuda"))
    assert st == B.DEV_BAD_SEQ and np.array_equal(k, host(k0))
    # an entry outside [i, length) moves nothing; any other takes the token that was there, in whatever order
    at = tokens(1)
    for i, x in ((0, -1), (20, 19), (59, 100), (59, 2 ** 31 - 1), (33, -2 ** 31), (20, 20), (20, 99), (0, 59)):
        bad = good.copy()
        bad[1, 1, i] = x
        st, k, v = run(kept=bad)
        wrong = not i <= x < 100
        assert st == (B.DEV_BAD_SEQ if wrong else 0)
        want_k, want_v = ref_k.copy(), ref_v.copy()
        want_k[at[i], 1] = host(k0)[at[i if wrong else x], 1]
        want_v[at[i], 1] = host(v0)[at[i if wrong else x], 1]
        assert np.array_equal(k, want_k) and np.array_equal(v, want_v)
    # a page outside the pool: tokens that would leave or enter it stay
    tab = table.copy()
    tab[1, 2], tab[1, 9] = -3, 10 ** 6
    st, k, v = run(tab=tab)
    want_k, want_v, _ = orc.compact(host(k0), host(v0), tab, 8, good, [100] * 3, [60] * 3)
    assert st == B.DEV_BAD_PAGE and np.array_equal(k, want_k) and np.array_equal(v, want_v)


# ------------------------------------------------ where calls can go wrong --

@pytest.mark.parametrize("rows,n_q", [(1, 28), (30, 16)])
def test_pools_past_two_to_the_31_elements(B, rows, n_q):
    """Weights and moves at element offsets that 32 bits do not hold."""
    rng = np.random.default_rng(22)
    n_kv, hd, page, tokens = 4, 128, 16, 4_300_000 // 16 * 16   # 2.2e9 elements a pool
    counts, ctx = np.array([rows, 2]), np.array([100, 33])
    start, n = np.concatenate([[0], np.cumsum(counts)]), ctx + counts
    cache, table = far_cache(B, rng, n_kv, hd, page, n, tokens)
    q = randn(rng, (int(start[-1]), n_q, hd), "bf16", 1.5)
    # the weights' heads far apart as well
    big = torch.empty(3 << 30, dtype=torch.float32, device="cuda")
    w = big.as_strided((2, n_kv, int(n.max())), (1 << 30, 1 << 28, 1))
    w.copy_(torch.rand(w.shape))
    before = host(w)
    most = int(counts.max())
    ws = B.alloc_workspace(B.kv_weigh_workspace_size(B.BF16, len(q), most, n_q, n_kv, hd, 2, w.shape[2]))
    B.specfold_kv_weigh(q, cache, ints(start), ints(ctx), most, w, ws, decay=0.5)
    # the oracle on the used pages alone
    used = table[table > 0]
    slots = torch.from_numpy((used[:, None].astype(np.int64) * page + np.arange(page)).reshape(-1)).cuda()
    small = np.zeros_like(table)
    small[table > 0] = np.arange(len(used))
    kp, vp = host(cache.k_pool[slots]), host(cache.v_pool[slots])
    ref, new, score = orc.weigh(host(q), kp, small, page, start, ctx, before, 0.5)
    d = 2 * hd * E * score + 2.0 ** -21
    assert (np.abs(host(w) - ref) <= (2 * d + (4160 + rows * n_q) * E) * new + 3 * E * np.abs(ref)).all()
    assert B.specfold_get_status(ws) == 0
    kept, new_len, status = torch.zeros(2, n_kv, 25, dtype=torch.int32, device="cuda"), ints([0, 0]), word()
    B.specfold_kv_select(w, ints(n), 25, kept, new_len, 1, 3, status)
    w1 = host(w)
    B.specfold_kv_compact(cache, kept, ints(n), new_len, weights=w, status=status)
    torch.cuda.synchronize()
    got = kept.cpu().numpy()
    for s, sets in enumerate(orc.select(w1, n, 25, 1, 3)):
        assert np.array_equal(got[s], np.stack(sets))
    k2, v2, w2 = orc.compact(kp, vp, small, page, got, n, [25, 25], w1)
    assert np.array_equal(host(cache.k_pool[slots]), k2) and np.array_equal(host(cache.v_pool[slots]), v2)
    assert np.array_equal(host(w), w2) and int(status) == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 40])
def test_two_streams_at_once(B, dt, rows):
    """Calls that overlap, each with a workspace of its own."""
    rng = np.random.default_rng(rows)
    b = [Weigh(B, rng, dt, 64, 8, 2, 16, "split", [rows, rows, 1], [2000 + 300 * i, 70, 900]) for i in range(2)]
    ref = []
    for x in b:
        w = x.w.clone()
        x.call(1.0, w=w)
        ref.append(w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    got = [[x.w.clone() for _ in range(8)] for x in b]
    torch.cuda.synchronize()
    for k in range(8):
        for i, x in enumerate(b):
            x.call(1.0, w=got[i][k], stream=streams[i])
    torch.cuda.synchronize()
    for i, x in enumerate(b):
        assert all(torch.equal(w, ref[i]) for w in got[i]) and B.specfold_get_status(x.ws) == 0


@pytest.mark.parametrize("rows", [1, 40])
def test_a_captured_call_follows_its_lengths(B, rows):
    """A graph replayed with other lengths, tables and rows than it was captured with."""
    rng = np.random.default_rng(rows)
    b = Weigh(B, rng, "bf16", 128, 8, 2, 16, "fused", [rows, rows], [600, 90], tail=rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.call(1.0, w=b.w.clone())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    w = b.w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call(0.5, w=w)
    for counts, ctx in (([rows, rows], [600, 90]), ([0, rows], [5, 33]), ([rows, 0], [0, 7]), ([0, 0], [9, 9]),
                        ([max(1, rows // 3), rows], [599, 0])):
        b.counts, b.ctx, b.start = np.array(counts), np.array(ctx), np.concatenate([[0], np.cumsum(counts)])
        b.at[0].copy_(ints(b.start))
        b.at[1].copy_(ints(b.ctx))
        w.copy_(b.w)
        graph.replay()
        torch.cuda.synchronize()
        b.check(host(b.w), host(w), 0.5)
    assert B.specfold_get_status(b.ws) == 0


def test_select_and_compact_captured(B):
    rng = np.random.default_rng(11)
    cache, table = make_cache(B, rng, "bf16", 64, 2, 16, [9000, 400], "split")
    w = torch.rand(2, 2, 9000, device="cuda")
    n, new = ints([9000, 400]), ints([0, 0])
    kept = torch.zeros(2, 2, 1000, dtype=torch.int32, device="cuda")

    def cut():
        B.specfold_kv_select(w, n, 1000, kept, new, 4, 100)
        B.specfold_kv_compact(cache, kept, n, new, weights=w)
    state = [t.clone() for t in (cache.k_pool, cache.v_pool, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cut()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cut()
    for lengths in ([9000, 400], [1001, 0], [700, 399], [8999, 400]):
        for t, old in zip((cache.k_pool, cache.v_pool, w), state):
            t.copy_(old)
        n.copy_(ints(lengths))
        w0, k0, v0 = w.cpu().numpy(), host(cache.k_pool), host(cache.v_pool)
        graph.replay()
        torch.cuda.synchronize()
        m = np.minimum(lengths, 1000)
        assert np.array_equal(new.cpu().numpy(), m)
        got = kept.cpu().numpy()
        for s, sets in enumerate(orc.select(w0, lengths, 1000, 4, 100)):
            for u in range(2):
                assert np.array_equal(got[s, u, :m[s]], sets[u])
        k2, v2, w2 = orc.compact(k0, v0, table, 16, got, lengths, m, w0)
        assert np.array_equal(host(cache.k_pool), k2) and np.array_equal(host(cache.v_pool), v2)
        assert np.array_equal(w.cpu().numpy(), w2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_guards_intact(B, dt):
    """Nothing outside of outputs and workspace is written."""
    rng = np.random.default_rng(12)
    for rows, hd in ((1, 128), (33, 64)):
        b = Weigh(B, rng, dt, hd, 8, 2, 16, "heads", [rows, 3], [300, 45])
        n = b.ws.numel()
        buf = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        buf[4096:4096 + n] = 0
        b.ws = buf[4096:4096 + n]
        wide = torch.full((4, b.n_kv + 2, b.tokens + 64), 3.0, device="cuda")
        w = wide[1:3, 1:-1, 32:-32]
        b.call(0.0, w=w)
        torch.cuda.synchronize()
        assert (buf[:4096] == 0xA5).all() and (buf[4096 + n:] == 0xA5).all()
        w.fill_(3.0)
        assert (wide == 3.0).all()


# ----------------------------------------------------- a run of them --

def test_calls_on_a_stream_of_their_own(B):
    rng = np.random.default_rng(5)
    b = Weigh(B, rng, "bf16", 128, 8, 2, 16, "split", [3, 1], [500, 40])
    plain = b.w.clone()
    b.call(1.0, w=plain)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mine = b.w.clone()
    kept = [torch.full((2, 2, 64), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    new, n = [ints([0, 0]) for _ in range(2)], ints([503, 41])
    torch.cuda.synchronize()
    b.call(1.0, w=mine, stream=st)
    B.specfold_kv_select(mine, n, 64, kept[0], new[0], 2, 8, stream=st)
    B.specfold_kv_select(plain, n, 64, kept[1], new[1], 2, 8)
    torch.cuda.synchronize()
    assert torch.equal(mine, plain) and torch.equal(kept[0], kept[1]) and torch.equal(new[0], new[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("captured", [False, True])
def test_a_cache_is_kept_to_its_budget(B, dt, captured):
    """Steps of a decoder whose tokens sit at three axes: rows normed, rotated and
    appended, their attention, their weights; then the cache is cut to its
    budget and the next step goes on behind what stays."""
    from oracle import cache_oracle
    rng = np.random.default_rng(6)
    S, n_q, n_kv, hd, page, budget, rows = 3, 8, 2, 64, 16, 96, 4
    pairs = [8, 12, 12]
    axes = B.RopeAxes(1e4, pairs, in_turn=True)
    ctx0 = np.array([96, 40, 95])
    cache, table = make_cache(B, rng, dt, hd, n_kv, page, [budget + rows] * S, "fused")
    T = S * rows
    start = ints(np.arange(S + 1) * rows)
    x = torch.empty(T, n_q + 2 * n_kv, hd, device="cuda", dtype=DT[dt])
    q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    qo, o, pos = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous()), torch.zeros(3, T, dtype=torch.int32, device="cuda")
    ctx, length = ints(ctx0), ints(ctx0)
    w = torch.rand(S, n_kv, budget + rows, device="cuda")
    kept, new_len = torch.zeros(S, n_kv, budget, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    dtc = B.dtype_code(DT[dt])
    ws = B.alloc_workspace(B.tree_attention_workspace_size(dtc, n_q, n_kv, hd, rows))
    ws2 = B.alloc_workspace(B.kv_weigh_workspace_size(dtc, T, rows, n_q, n_kv, hd, S, budget + rows))
    status = word()

    def step():
        B.specfold_qk_norm_rope_axes(q, None, qo, None, axes, pos)
        B.specfold_kv_append_axes(k, v, cache, start, ctx, axes, pos, status=status)
        B.specfold_tree_attention(qo, cache, None, start, ctx, rows, o, ws)
        B.specfold_kv_weigh(qo, cache, start, ctx, rows, w, ws2, decay=0.9)
        length.copy_(ctx + rows)
        B.specfold_kv_select(w, length, budget, kept, new_len, sinks=2, recent=8, status=status)
        B.specfold_kv_compact(cache, kept, length, new_len, weights=w, status=status)
        ctx.copy_(new_len)

    graph = None
    if captured:
        state = [t.clone() for t in (cache.k_pool, cache.v_pool, w, ctx)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        x.normal_()
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, old in zip((cache.k_pool, cache.v_pool, w, ctx), state):
            t.copy_(old)
    for it in range(4):
        x.copy_(randn(rng, tuple(x.shape), dt))
        pos.copy_(ints(rng.integers(0, 5000, (3, T))))
        c = ctx.cpu().numpy()
        kp, vp, w0 = host(cache.k_pool), host(cache.v_pool), host(w)
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        # the definition, from the state before the step; the rotated values as rounded
        ref, _ = orc.norm_rotate_axes(host(q), None, 0.0, host(pos), pairs, True, 1e4, False)
        assert (np.abs(host(qo) - ref) <= half_step(dt) * np.abs(ref) + 1e-5 * 8).all()
        n = c + rows
        order = [list(range(t)) for t in n]
        kk, vv = kp.copy(), vp.copy()
        rk, _ = orc.norm_rotate_axes(host(k), None, 0.0, host(pos), pairs, True, 1e4, False)
        rk = torch.from_numpy(rk).to(DT[dt]).double().numpy()
        for s in range(S):
            for i in range(rows):
                at = cache_oracle.slot_of(table, page, kp.shape[0] // page, s, c[s] + i)
                kk[at], vv[at] = rk[s * rows + i], host(v)[s * rows + i]
        want_o, spread, _ = cache_oracle.tree_attention(host(qo), kk, vv, table, page, None, np.arange(S + 1) * rows, c)
        assert (np.abs(host(o) - want_o) <= 4 * half_step(dt) * (np.abs(want_o) + spread) + 2e-5).all()
        want_w, _, _ = orc.weigh(host(qo), kk, table, page, np.arange(S + 1) * rows, c, w0, 0.9)
        got_n, got_kept, got_w = new_len.cpu().numpy(), kept.cpu().numpy(), host(w)
        assert np.array_equal(got_n, np.minimum(n, budget))
        for s in range(S):
            for u in range(n_kv):
                ids = got_kept[s, u, :got_n[s]]
                assert (np.diff(ids) > 0).all() and ids[-1] == n[s] - 1
                assert np.allclose(got_w[s, u, :got_n[s]], want_w[s, u, ids], rtol=2e-2, atol=1e-4)
                if n[s] > budget:   # no token that went weighs more than one that stayed, but for the roundings
                    gone = np.setdiff1d(np.arange(n[s]), ids)
                    assert want_w[s, u, gone].max() <= want_w[s, u, ids[2:-8]].min() * 1.02 + 1e-4
        end_k, end_v, _ = orc.compact(kk, vv, table, page, got_kept, n, got_n)
        assert np.array_equal(host(cache.v_pool), end_v)
        assert (np.abs(host(cache.k_pool) - end_k) <= 2 * half_step(dt) * np.abs(end_k) + 1e-5 * 8).all()
    assert int(status) == 0 and B.specfold_get_status(ws) == 0 and B.specfold_get_status(ws2) == 0
