"""Positions with several axes and the operators that thin out a paged cache, on
the host: closed forms that pin the oracle, and every refusal (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_oracle, evict_oracle as orc
from tests.test_cache_ops import A, _bad_caches, _cache, _hr


@pytest.fixture(scope="module")
def B():
    from diffusion_branch_speculative_gb300 import build, binding
    build.build()
    binding.lib()
    return binding


# ------------------------------------------------------------------ oracle --

def test_oracle_axes_in_blocks_and_in_turn():
    assert [a for a, _ in orc.axis_pairs([2, 1, 3], False)] == [0, 0, 1, 2, 2, 2]
    assert orc.axis_pairs([2, 1, 3], True) == [(0, 0), (1, 0), (2, 0), (0, 1), (2, 1), (2, 2)]
    assert orc.axis_pairs([0, 2], True) == [(1, 0), (1, 1)]
    f = orc.frequencies([2, 2], False, 16.0, False)
    assert np.allclose(np.float64(f), [1, 0.5, 0.25, 0.125])
    assert np.allclose(np.float64(orc.frequencies([2, 2], True, 16.0, True)), [1, 1, 0.25, 0.25])


def test_oracle_axes_alike_are_one_position():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 2, 64)), rng.integers(0, 1000, 5)
    one, _ = cache_oracle.norm_rotate(x, None, 0.0, pos, 1e4)
    for pairs, turn in (([32], False), ([8, 12, 12], False), ([8, 12, 12], True), ([30, 0, 2, 0], True)):
        y, _ = orc.norm_rotate_axes(x, None, 0.0, np.tile(pos, (len(pairs), 1)), pairs, turn, 1e4, False)
        assert np.allclose(y, one, atol=1e-12)


def test_oracle_weigh_against_dense():
    rng = np.random.default_rng(1)
    kp = rng.standard_normal((24, 2, 64))
    q, w = rng.standard_normal((6, 6, 64)), rng.random((1, 2, 20))
    table = np.array([[2, 0, 1]], np.int32)
    got, new, _ = orc.weigh(q, kp, table, 8, [0, 3], [10], w, 0.5, rows=[5, 0, 2])
    k = torch.from_numpy(kp[np.concatenate([np.arange(16, 24), np.arange(8)])][:13].repeat(3, 1)).transpose(0, 1)
    x = torch.from_numpy(q[[5, 0, 2]]).transpose(0, 1) @ k.transpose(1, 2) / 8
    x = x.masked_fill(torch.arange(13)[None] > torch.arange(3)[:, None] + 10, -float("inf"))
    p = torch.softmax(x, -1).reshape(2, 9, 13).sum(1).numpy()
    assert np.allclose(new[0, :, :13], p) and np.isclose(new.sum(), 18)
    assert np.allclose(got[0, :, :10], 0.5 * w[0, :, :10] + p[:, :10])
    assert np.allclose(got[0, :, 10:13], p[:, 10:]) and np.array_equal(got[0, :, 13:], w[0, :, 13:])


def test_oracle_select():
    nan = float("nan")
    w = np.array([[[0.1, 5, 0.2, 5, nan, -0.0, 0.0, 9]]])
    pick = lambda n, keep, sinks=0, recent=0: list(orc.select(w, [n], keep, sinks, recent)[0][0])
    assert pick(8, 3) == [1, 3, 7]
    assert pick(8, 2) == [1, 7]                # of equal weights the first
    assert pick(8, 6) == [0, 1, 2, 3, 5, 7]    # zeros are equal: the first of them
    assert pick(8, 7) == [0, 1, 2, 3, 5, 6, 7]  # the NaN goes first
    assert pick(8, 3, sinks=1, recent=1) == [0, 1, 7]
    assert pick(7, 3, sinks=1, recent=2) == [0, 5, 6]
    assert pick(4, 4) == [0, 1, 2, 3] and pick(0, 3) == []
    assert orc.select(w, [9, -1], 3, 0, 0) == [None, None]


def test_oracle_compact():
    kp = np.arange(32.0).reshape(16, 2, 1)
    table = np.array([[1, 0]], np.int32)
    k, v, w = orc.compact(kp, kp + 100, table, 8, [[[0, 2, 9], [1, 2, 3]]], [12], [3], np.arange(24.0).reshape(1, 2, 12))
    assert list(k[8:11, 0, 0]) == [kp[8, 0, 0], kp[10, 0, 0], kp[1, 0, 0]] and k[11, 0, 0] == kp[11, 0, 0]
    assert list(v[8:11, 1, 0]) == [kp[9, 1, 0] + 100, kp[10, 1, 0] + 100, kp[11, 1, 0] + 100]
    assert list(w[0, 0, :4]) == [0, 2, 9, 3] and list(w[0, 1, :4]) == [13, 14, 15, 15]
    one, _, _ = orc.compact(kp, kp, table, 8, [[[1]]], [12], [1])
    assert one[8, 0, 0] == kp[9, 0, 0] and one[8, 1, 0] == kp[9, 1, 0]


def test_oracle_compact_leaves_a_token_without_a_page():
    kp = np.arange(32.0).reshape(16, 2, 1)
    table = np.array([[1, 7]], np.int32)            # the second page lies outside the pool
    k, v, w = orc.compact(kp, kp, table, 8, [[[1, 9]]], [12], [2], np.arange(12.0).reshape(1, 1, 12))
    assert k[8, 0, 0] == kp[9, 0, 0] and k[9, 0, 0] == v[9, 0, 0] == kp[9, 0, 0]
    assert list(w[0, 0, :3]) == [1, 1, 2]


# ----------------------------------------------------------- C ABI refusals --
# Aligned fake addresses: every call below is refused before a launch.

FAR = A + (1 << 16)


def _axes(B, theta=1e4, n=3, pairs=(16, 24, 24, 0), order=0, own=0):
    return B.specfold_rope_axes(theta, n, (ctypes.c_int * 4)(*pairs), order, own)


def _bad_axes(B):
    yield _axes(B, theta=0.0), B.EINVAL
    yield _axes(B, theta=-1.0), B.EINVAL
    yield _axes(B, theta=float("nan")), B.EINVAL
    yield _axes(B, theta=float("inf")), B.EINVAL
    yield _axes(B, n=0), B.EINVAL
    yield _axes(B, n=5), B.EINVAL
    yield _axes(B, pairs=(16, 24, 23, 1)), B.EINVAL      # the fourth is not read
    yield _axes(B, pairs=(16, 24, 25, 0)), B.EINVAL
    yield _axes(B, pairs=(-8, 48, 24, 0)), B.EINVAL
    yield _axes(B, pairs=(2 ** 31 - 1, 24, 24, 0)), B.EINVAL
    yield _axes(B, order=2), B.EINVAL
    yield _axes(B, own=2), B.EINVAL


def _qk_axes(B, axes=None, pos=A, T=4, n_q=4, n_kv=2, hd=128, dtype=0, eps=1e-6, q=None, ko=None):
    x = _axes(B) if axes is None else axes
    r = lambda v: _hr(B) if v is None else v
    return B.lib().specfold_qk_norm_rope_axes(dtype, T, n_q, n_kv, hd, r(q), r(None), r(None), r(ko), A, A, eps,
                                              ctypes.byref(x), B.specfold_axis_positions(pos, 1, T), None)


def _append_axes(B, axes=None, pos=A, T=4, n_kv=2, hd=128, dtype=0, eps=1e-6, k=None, v=None, n_src=4, cache=None,
                 start=A, ctx=A, n_seqs=2):
    x = _axes(B) if axes is None else axes
    r = lambda y: _hr(B) if y is None else y
    c = _cache(B) if cache is None else cache
    return B.lib().specfold_kv_append_axes(dtype, T, n_kv, hd, r(k), r(v), n_src, None, None, eps, ctypes.byref(x),
                                           B.specfold_axis_positions(pos, 1, T), ctypes.byref(c), start, ctx, n_seqs,
                                           None, None)


def test_qk_norm_rope_axes_refusals(B):
    for axes, rc in _bad_axes(B):
        assert _qk_axes(B, axes=axes) == rc
    assert B.lib().specfold_qk_norm_rope_axes(0, 4, 4, 2, 128, _hr(B), _hr(B), _hr(B), _hr(B), A, A, 1e-6, None,
                                              B.specfold_axis_positions(A, 1, 4), None) == B.EINVAL
    assert _qk_axes(B, pos=None) == B.EINVAL
    assert _qk_axes(B, hd=96) == B.EUNSUPPORTED
    assert _qk_axes(B, hd=64) == B.EINVAL                # 64 pairs for 32
    assert _qk_axes(B, dtype=3) == B.EINVAL
    assert _qk_axes(B, T=-1) == B.EINVAL
    assert _qk_axes(B, eps=-1.0) == B.EINVAL
    assert _qk_axes(B, n_q=B.MAX_HEADS + 1) == B.ECAPACITY
    assert _qk_axes(B, q=_hr(B, ptr=A + 2)) == B.EALIGN
    assert _qk_axes(B, ko=_hr(B, ptr=None)) == B.EINVAL
    assert _qk_axes(B, T=0) == B.OK and _qk_axes(B, n_q=0, n_kv=0) == B.OK


def test_kv_append_axes_refusals(B):
    for axes, rc in _bad_axes(B):
        assert _append_axes(B, axes=axes) == rc
    for cache, rc in _bad_caches(B):
        assert _append_axes(B, cache=cache) == rc
    assert _append_axes(B, pos=None) == B.EINVAL
    assert _append_axes(B, n_src=3) == B.EINVAL
    assert _append_axes(B, n_kv=0) == B.EINVAL
    assert _append_axes(B, n_seqs=1025) == B.ECAPACITY
    assert _append_axes(B, start=None) == B.EINVAL
    assert _append_axes(B, eps=float("inf")) == B.EINVAL
    assert _append_axes(B, k=_hr(B, rs=4)) == B.EALIGN
    assert _append_axes(B, k=_hr(B, ptr=A)) == B.EINVAL   # a pool's rows
    assert _append_axes(B, T=0) == B.OK


def _tw(B, ptr=A, ss=4000, hs=1000, tokens=1000):
    return B.specfold_token_weights(ptr, ss, hs, tokens)


def _kt(B, ptr=A, ss=400, us=100, sets=2, cap=100):
    return B.specfold_kept_tokens(ptr, ss, us, sets, cap)


# strides under which written rows lie on one another: [2 sequences, 2 heads]
OVERLAP = [(4000, 999), (1999, 1000), (0, 1000), (4000, 0), (1000, 1000), (999, 4000), (1000, 1999)]


def _weigh(B, dtype=0, T=4, rows_=4, n_q=4, n_kv=2, hd=128, q=None, n_src=4, rows=None, cache=None, start=A, ctx=A,
           n_seqs=2, scale=0.0, decay=1.0, w=None, ws=A, nbytes=1 << 40):
    c = _cache(B) if cache is None else cache
    return B.lib().specfold_kv_weigh(dtype, T, rows_, n_q, n_kv, hd, _hr(B) if q is None else q, n_src, rows,
                                     ctypes.byref(c), start, ctx, n_seqs, scale, decay, _tw(B) if w is None else w, ws,
                                     nbytes, None)


def test_kv_weigh_refusals(B):
    for cache, rc in _bad_caches(B):
        assert _weigh(B, cache=cache) == rc
    assert _weigh(B, dtype=2) == B.EINVAL
    assert _weigh(B, T=-1) == B.EINVAL
    assert _weigh(B, rows_=0) == B.EINVAL
    assert _weigh(B, rows_=257) == B.ECAPACITY
    assert _weigh(B, n_q=3) == B.EUNSUPPORTED
    assert _weigh(B, n_q=258, n_kv=2) == B.EUNSUPPORTED
    assert _weigh(B, n_q=B.MAX_HEADS + 2, n_kv=B.MAX_HEADS + 2) == B.ECAPACITY
    assert _weigh(B, hd=32) == B.EUNSUPPORTED
    for bad in (-1.0, float("nan"), float("inf")):
        assert _weigh(B, scale=bad) == B.EINVAL
        assert _weigh(B, decay=bad) == B.EINVAL
    assert _weigh(B, start=None) == B.EINVAL
    assert _weigh(B, ctx=None) == B.EINVAL
    assert _weigh(B, n_seqs=0) == B.EINVAL
    assert _weigh(B, n_seqs=1025) == B.ECAPACITY
    assert _weigh(B, q=_hr(B, hs=4)) == B.EALIGN
    assert _weigh(B, q=_hr(B, ptr=None)) == B.EINVAL
    assert _weigh(B, n_src=3) == B.EINVAL
    assert _weigh(B, n_src=-1, rows=A) == B.EINVAL
    assert _weigh(B, n_src=0, rows=A) == B.EINVAL
    assert _weigh(B, ws=None) == B.EINVAL
    assert _weigh(B, ws=A + 8) == B.EALIGN
    assert _weigh(B, w=_tw(B, ptr=None)) == B.EINVAL
    assert _weigh(B, w=_tw(B, ptr=A + 2)) == B.EALIGN
    assert _weigh(B, w=_tw(B, tokens=0)) == B.EINVAL
    assert _weigh(B, w=_tw(B, ss=-4000)) == B.EINVAL
    assert _weigh(B, w=_tw(B, ss=1 << 40, hs=1 << 36, tokens=B.MAX_TOKENS + 1)) == B.ECAPACITY
    for ss, hs in OVERLAP:
        assert _weigh(B, w=_tw(B, ss=ss, hs=hs)) == B.EINVAL
    need = B.kv_weigh_workspace_size(B.BF16, 4, 4, 4, 2, 128, 2, 1000)
    assert _weigh(B, nbytes=need - 1) == B.ECAPACITY
    assert _weigh(B, T=0) == B.OK


def test_kv_weigh_workspace_size(B):
    size = B.kv_weigh_workspace_size
    assert size(B.BF16, 64, 1, 28, 4, 128, 64, 8192) > 0 and size(B.F32, 0, 1, 4, 2, 64, 1, 1) > 0
    for args in ((B.BF16, -1, 1, 28, 4, 128, 64, 8192), (B.BF16, 64, 0, 28, 4, 128, 64, 8192),
                 (B.BF16, 64, 257, 28, 4, 128, 64, 8192), (B.BF16, 64, 1, 28, 3, 128, 64, 8192),
                 (B.BF16, 64, 1, 28, 4, 96, 64, 8192), (B.BF16, 64, 1, 28, 4, 128, 0, 8192),
                 (B.BF16, 64, 1, 28, 4, 128, 1025, 8192), (B.BF16, 64, 1, 28, 4, 128, 64, 0),
                 (9, 64, 1, 28, 4, 128, 64, 8192), (B.BF16, 64, 1, 28, 4, 128, 64, B.MAX_TOKENS + 1)):
        assert size(*args) == 0
    # shapes that no memory holds ask for more than there is, not for what 64 bits leave of it
    assert size(B.F32, 64, 256, 65536, 512, 128, 1024, B.MAX_TOKENS) > 1 << 60
    assert size(B.F32, 64, 256, 128, 1, 128, 1024, B.MAX_TOKENS) > 1 << 50
    # few rows of bf16 and all of fp32 keep their scores: eight rows of a group, 16 bytes and more a token
    small, large = size(B.BF16, 64, 1, 28, 4, 128, 64, 40000), size(B.BF16, 64, 1, 28, 4, 128, 64, 65536)
    assert large - small == 64 * 4 * (65536 - 40000) * 8 * 4
    for tokens in (8192, 16384):
        assert size(B.BF16, 64, 1, 28, 4, 128, 64, tokens) == 256          # in registers
    assert size(B.BF16, 64, 1, 28, 4, 128, 64, 16385) > 1 << 27
    assert size(B.F32, 64, 1, 28, 4, 128, 64, 8192) > 64 * 4 * 8192 * 8 * 4
    assert size(B.BF16, 64, 1, 28, 4, 128, 1024, 1 << 20) < 1 << 28        # past 1 GB: computed twice


def _select(B, w=None, lengths=A, n_seqs=2, keep=50, sinks=4, recent=8, kept=None, new_len=FAR):
    return B.lib().specfold_kv_select(_tw(B) if w is None else w, lengths, n_seqs, keep, sinks, recent,
                                      _kt(B) if kept is None else kept, new_len, None, None)


def test_kv_select_refusals(B):
    assert _select(B, w=_tw(B, ptr=None)) == B.EINVAL
    assert _select(B, w=_tw(B, tokens=0)) == B.EINVAL
    assert _select(B, w=_tw(B, tokens=B.MAX_TOKENS + 1)) == B.ECAPACITY
    assert _select(B, kept=_kt(B, ss=1 << 40, us=1 << 36, cap=B.MAX_TOKENS + 1)) == B.ECAPACITY
    assert _select(B, w=_tw(B, ptr=A + 1)) == B.EALIGN
    assert _select(B, lengths=None) == B.EINVAL
    assert _select(B, new_len=None) == B.EINVAL
    assert _select(B, new_len=A) == B.EINVAL             # the lengths themselves
    assert _select(B, new_len=A + 4) == B.EINVAL
    assert _select(B, n_seqs=0) == B.EINVAL
    assert _select(B, n_seqs=1025) == B.ECAPACITY
    for kw in (dict(keep=0), dict(keep=-1), dict(sinks=-1), dict(recent=-1), dict(sinks=43), dict(recent=47),
               dict(keep=101), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert _select(B, **kw) == B.EINVAL, kw
    assert _select(B, kept=_kt(B, ptr=None)) == B.EINVAL
    assert _select(B, kept=_kt(B, ptr=A + 2)) == B.EALIGN
    assert _select(B, kept=_kt(B, sets=0)) == B.EINVAL
    assert _select(B, kept=_kt(B, sets=B.MAX_HEADS + 1, us=100, ss=1 << 40)) == B.ECAPACITY
    for ss, us in OVERLAP:
        assert _select(B, kept=_kt(B, ss=ss, us=us, cap=1000)) == B.EINVAL


def _compact(B, dtype=0, n_kv=2, hd=128, cache=None, kept=None, lengths=A, new_len=FAR, n_seqs=2, w=None):
    c = _cache(B) if cache is None else cache
    return B.lib().specfold_kv_compact(dtype, n_kv, hd, ctypes.byref(c), _kt(B) if kept is None else kept, lengths,
                                       new_len, n_seqs, None if w is None else ctypes.byref(w), None, None)


def test_kv_compact_refusals(B):
    for cache, rc in _bad_caches(B):
        assert _compact(B, cache=cache) == rc
    assert _compact(B, dtype=2) == B.EINVAL
    assert _compact(B, n_kv=0) == B.EINVAL
    assert _compact(B, n_kv=B.MAX_HEADS + 1) == B.ECAPACITY
    assert _compact(B, hd=256) == B.EUNSUPPORTED
    assert _compact(B, lengths=None) == B.EINVAL
    assert _compact(B, new_len=None) == B.EINVAL
    assert _compact(B, new_len=A) == B.EINVAL
    assert _compact(B, n_seqs=0) == B.EINVAL
    assert _compact(B, n_seqs=1025) == B.ECAPACITY
    assert _compact(B, kept=_kt(B, sets=3)) == B.EINVAL
    assert _compact(B, kept=_kt(B, cap=0)) == B.EINVAL
    assert _compact(B, kept=_kt(B, us=-1)) == B.EINVAL
    assert _compact(B, kept=_kt(B, cap=B.MAX_TOKENS + 1)) == B.ECAPACITY
    assert _compact(B, w=_tw(B, ss=1 << 40, hs=1 << 36, tokens=B.MAX_TOKENS + 1)) == B.ECAPACITY
    assert _compact(B, w=_tw(B, ptr=None)) == B.EINVAL
    assert _compact(B, w=_tw(B, hs=-1)) == B.EINVAL
    for ss, hs in OVERLAP:
        assert _compact(B, w=_tw(B, ss=ss, hs=hs)) == B.EINVAL


# --------------------------------------------------------- binding refusals --

def test_rope_axes_of_the_binding(B):
    x = B.RopeAxes(5e6, [16, 24, 24], in_turn=True, own_frequencies=True)
    assert (x.struct.n_axes, list(x.struct.pairs), x.struct.order, x.struct.own_frequencies) == (3, [16, 24, 24, 0], 1, 1)
    for pairs in ([], [1] * 5):
        with pytest.raises(ValueError, match="axes"):
            B.RopeAxes(1e4, pairs)


def test_binding_refuses_host_tensors_and_shapes(B):
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    x, pos = B.RopeAxes(1e4, [16, 16]), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.specfold_qk_norm_rope_axes(q, k, q, k, x, pos)
    with pytest.raises(ValueError, match="Q or K"):
        B.specfold_qk_norm_rope_axes(None, None, None, None, x, pos)
    with pytest.raises(ValueError, match="Q_out"):
        B.specfold_qk_norm_rope_axes(q, k, None, k, x, pos)
    w, n = torch.zeros(2, 2, 9), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.specfold_kv_select(w, n, 4, torch.zeros(2, 2, 4, dtype=torch.int32), n.clone())


def test_binding_refuses_positions(B):
    x, good = B.RopeAxes(1e4, [16, 16]), torch.zeros(2, 3, dtype=torch.int32)
    at = B._axis_positions(good.t().contiguous().t(), x, 3, -1)
    assert (at.row_stride, at.axis_stride) == (2, 1)
    for bad in (None, good[0], good.long(), good[:1], torch.zeros(3, 3, dtype=torch.int32), good[:, :2]):
        with pytest.raises(ValueError, match="positions"):
            B._axis_positions(bad, x, 3, -1)
    with pytest.raises(ValueError, match="device"):
        B._axis_positions(good, x, 3, 0)


def test_binding_refuses_per_token_tensors(B):
    w = torch.zeros(4, 2, 10)
    assert B._per_token(w[:, :, 2:7], 3, 2, torch.float32, -1, "weights")[1:] == (20, 10, 5)
    assert B._per_token(w[:, :, ::10], 4, 2, torch.float32, -1, "weights")[3] == 1
    for bad in (w[0], w[:2], w[:, :1], w[:, :, ::2], w.transpose(1, 2), w.double(), w.int()):
        with pytest.raises(ValueError, match="weights"):
            B._per_token(bad, 3, 2, torch.float32, -1, "weights")
    with pytest.raises(ValueError, match="device"):
        B._per_token(w, 3, 2, torch.float32, 0, "weights")
