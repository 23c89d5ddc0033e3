"""The operators of a decoder's paged cache on the host: closed forms that pin
the oracle, and every refusal of the C ABI and the binding (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc


@pytest.fixture(scope="module")
def B():
    from diffusion_branch_speculative_gb300 import build, binding
    build.build()
    binding.lib()
    return binding


# ------------------------------------------------------------------ oracle --

def test_oracle_rotation_closed_form():
    x = np.zeros((2, 1, 4))
    x[:, 0, 0] = 1.0          # pair (0, 2) at frequency 1
    x[:, 0, 1] = 2.0          # pair (1, 3) at frequency theta^(-1/2) = 0.1
    y, size = orc.norm_rotate(x, None, 0.0, [0, 3], 100.0)
    assert np.allclose(y[0, 0], [1, 2, 0, 0])
    assert np.allclose(y[1, 0], [np.cos(3), 2 * np.cos(0.3), np.sin(3), 2 * np.sin(0.3)])
    assert np.allclose(size[1, 0], [1, 2, 1, 2])


def test_oracle_norm_closed_form():
    y, _ = orc.norm_rotate(np.full((1, 1, 4), 3.0), np.array([1.0, 2.0, 3.0, 4.0]), 0.0, [0], 0.0)
    assert np.allclose(y[0, 0], [1, 2, 3, 4])
    z, _ = orc.norm_rotate(np.zeros((1, 1, 4)), np.ones(4), 1e-6, [0], 0.0)
    assert np.all(z == 0)


def test_oracle_scores_depend_on_distance_only():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 64))
    dots = []
    for base in (0, 12345):
        a, _ = orc.norm_rotate(q, None, 0.0, [base + 7], 1e4)
        b, _ = orc.norm_rotate(k, None, 0.0, [base], 1e4)
        dots.append((a * b).sum())
    assert np.isclose(dots[0], dots[1], atol=1e-10)


def test_oracle_ancestors():
    # 0 and 3 are roots; 1, 2 below 0; 4 below 2; 5 padding; 6 below the padding row
    sees = orc.ancestors([-1, 0, 0, -1, 2, -2, 5], 7)
    assert [list(np.nonzero(r)[0]) for r in sees] == [[0], [0, 1], [0, 2], [3], [0, 2, 4], [], [6]]
    assert np.array_equal(orc.ancestors(None, 5), np.tril(np.ones((5, 5), bool)))


def test_oracle_attention_against_dense():
    rng = np.random.default_rng(1)
    page, n_kv, g, hd = 8, 2, 3, 64
    kp, vp = rng.standard_normal((2, 5 * page, n_kv, hd))
    table = np.array([[3, 1, 4]], np.int32)
    q = rng.standard_normal((4, n_kv * g, hd))
    o, spread, _ = orc.tree_attention(q, kp, vp, table, page, None, [0, 4], [9])
    idx = np.concatenate([np.arange(8) + 24, np.arange(8) + 8])[:13]
    k = torch.from_numpy(np.repeat(kp[idx], g, 1)).transpose(0, 1)
    v = torch.from_numpy(np.repeat(vp[idx], g, 1)).transpose(0, 1)
    mask = torch.arange(13)[None] <= torch.arange(4)[:, None] + 9
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).transpose(0, 1), k, v, attn_mask=mask)
    assert np.allclose(o, ref.transpose(0, 1).numpy())
    assert (spread >= np.abs(o) - 1e-12).all()


def test_oracle_append_writes_its_slots_only():
    rng = np.random.default_rng(2)
    kp, vp = rng.standard_normal((2, 32, 1, 64))
    K, V = rng.standard_normal((2, 3, 1, 64))
    table = np.array([[2, 0], [1, 3]], np.int32)
    k2, v2, size = orc.append(kp, vp, table, 8, K, V, [0, 2, 3], [7, 0], None, 0.0, None, 0.0)
    assert sorted(size) == [0, 8, 23]        # tokens 7 and 8 of sequence 0, token 0 of sequence 1
    assert np.array_equal(k2[23], K[0]) and np.array_equal(v2[0], V[1]) and np.array_equal(k2[8], K[2])
    rest = np.setdiff1d(np.arange(32), list(size))
    assert np.array_equal(k2[rest], kp[rest]) and np.array_equal(v2[rest], vp[rest])


# ----------------------------------------------------------- C ABI refusals --
# Aligned fake addresses: every call below is refused before a launch.

A = 1 << 20


def _hr(B, ptr=A, rs=512, hs=128):
    return B.specfold_head_rows(ptr, rs, hs)


def _cache(B, **kw):
    base = dict(k=A, v=A, kt=512, kh=128, vt=512, vh=128, table=A, tstride=4, tpages=4, page=16, pages=8)
    base.update(kw)
    b = base
    return B.specfold_paged_cache(b["k"], b["v"], b["kt"], b["kh"], b["vt"], b["vh"], b["table"], b["tstride"],
                                  b["tpages"], b["page"], b["pages"])


def _qk(B, dtype=0, T=4, n_q=4, n_kv=2, hd=128, q=None, k=None, qo=None, ko=None, eps=1e-6, pos=A, theta=1e4):
    r = lambda v: _hr(B) if v is None else v
    return B.lib().specfold_qk_norm_rope(dtype, T, n_q, n_kv, hd, r(q), r(k), r(qo), r(ko), A, A, eps, pos, theta, None)


def _append(B, dtype=0, T=4, n_kv=2, hd=128, k=None, v=None, n_src=4, rows=None, eps=1e-6, theta=1e4, cache=None,
            start=A, ctx=A, n_seqs=2):
    r = lambda x: _hr(B) if x is None else x
    c = _cache(B) if cache is None else cache
    return B.lib().specfold_kv_append(dtype, T, n_kv, hd, r(k), r(v), n_src, rows, None, eps, None, theta,
                                      ctypes.byref(c), start, ctx, n_seqs, None, None)


def _tree(B, dtype=0, T=4, nodes=4, n_q=4, n_kv=2, hd=128, q=None, o=None, cache=None, start=A, ctx=A, n_seqs=2,
          scale=0.0, ws=A, nbytes=1 << 40):
    r = lambda x: _hr(B) if x is None else x
    c = _cache(B) if cache is None else cache
    return B.lib().specfold_tree_attention(dtype, T, nodes, n_q, n_kv, hd, r(q), ctypes.byref(c), None, start, ctx,
                                           n_seqs, scale, r(o), ws, nbytes, None)


def test_qk_norm_rope_refusals(B):
    assert _qk(B, dtype=7) == B.EINVAL
    assert _qk(B, T=-1) == B.EINVAL
    assert _qk(B, n_q=-1) == B.EINVAL
    assert _qk(B, hd=96) == B.EUNSUPPORTED
    for eps in (-1.0, float("nan"), float("inf")):
        assert _qk(B, eps=eps) == B.EINVAL
    for theta in (-1.0, float("nan"), float("inf")):
        assert _qk(B, theta=theta) == B.EINVAL
    assert _qk(B, pos=None) == B.EINVAL
    for which in ("q", "k", "qo", "ko"):
        assert _qk(B, **{which: _hr(B, ptr=None)}) == B.EINVAL
        assert _qk(B, **{which: _hr(B, rs=0)}) == B.EINVAL
        assert _qk(B, **{which: _hr(B, hs=-128)}) == B.EINVAL
        assert _qk(B, **{which: _hr(B, ptr=A + 8)}) == B.EALIGN
        assert _qk(B, **{which: _hr(B, rs=516)}) == B.EALIGN
    # nothing to do: no rows, or no heads
    assert _qk(B, T=0) == B.OK
    assert _qk(B, n_q=0, n_kv=0) == B.OK


def _bad_caches(B):
    yield _cache(B, k=None), B.EINVAL
    yield _cache(B, table=None), B.EINVAL
    yield _cache(B, tpages=0), B.EINVAL
    yield _cache(B, tstride=-1), B.EINVAL
    yield _cache(B, page=0), B.EINVAL
    yield _cache(B, page=12), B.EUNSUPPORTED
    yield _cache(B, pages=0), B.EINVAL
    yield _cache(B, vt=0), B.EINVAL
    yield _cache(B, kh=100), B.EALIGN
    yield _cache(B, v=A + 4), B.EALIGN
    yield _cache(B, page=1 << 16, pages=1 << 16), B.ECAPACITY


def test_kv_append_refusals(B):
    for cache, rc in _bad_caches(B):
        assert _append(B, cache=cache) == rc
    assert _append(B, dtype=2) == B.EINVAL
    assert _append(B, T=-1) == B.EINVAL
    assert _append(B, n_kv=0) == B.EINVAL
    assert _append(B, n_src=-1) == B.EINVAL
    assert _append(B, n_src=3) == B.EINVAL           # fewer rows than the batch, none picked
    assert _append(B, hd=32) == B.EUNSUPPORTED
    assert _append(B, start=None) == B.EINVAL
    assert _append(B, ctx=None) == B.EINVAL
    assert _append(B, n_seqs=0) == B.EINVAL
    assert _append(B, n_seqs=1025) == B.ECAPACITY
    assert _append(B, eps=float("nan")) == B.EINVAL
    assert _append(B, theta=-2.0) == B.EINVAL
    assert _append(B, k=_hr(B, ptr=None)) == B.EINVAL
    assert _append(B, v=_hr(B, rs=4)) == B.EALIGN
    assert _append(B, T=0) == B.OK


def test_tree_attention_refusals(B):
    for cache, rc in _bad_caches(B):
        assert _tree(B, cache=cache) == rc
    assert _tree(B, dtype=2) == B.EINVAL
    assert _tree(B, T=-1) == B.EINVAL
    assert _tree(B, nodes=0) == B.EINVAL
    assert _tree(B, nodes=257) == B.ECAPACITY
    assert _tree(B, n_q=3) == B.EUNSUPPORTED
    assert _tree(B, n_q=258, n_kv=2) == B.EUNSUPPORTED
    assert _tree(B, n_kv=0) == B.EINVAL
    assert _tree(B, hd=256) == B.EUNSUPPORTED
    for scale in (-1.0, float("nan"), float("inf")):
        assert _tree(B, scale=scale) == B.EINVAL
    assert _tree(B, start=None) == B.EINVAL
    assert _tree(B, n_seqs=4096) == B.ECAPACITY
    assert _tree(B, q=_hr(B, hs=4)) == B.EALIGN
    assert _tree(B, o=_hr(B, ptr=None)) == B.EINVAL
    assert _tree(B, ws=None) == B.EINVAL
    assert _tree(B, ws=A + 8) == B.EALIGN
    need = B.tree_attention_workspace_size(B.BF16, 4, 2, 128, 4)
    assert _tree(B, nbytes=need - 1) == B.ECAPACITY
    assert _tree(B, T=0) == B.OK


def test_tree_workspace_size(B):
    size = B.tree_attention_workspace_size
    assert size(B.BF16, 28, 4, 128, 64) > 0
    assert size(B.BF16, 28, 4, 96, 64) == 0
    assert size(B.BF16, 28, 4, 128, 0) == 0
    assert size(B.BF16, 28, 4, 128, 257) == 0
    assert size(B.BF16, 28, 3, 128, 64) == 0
    assert size(5, 28, 4, 128, 64) == 0


# --------------------------------------------------------- binding refusals --

def test_binding_refuses_host_tensors_and_shapes(B):
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.specfold_qk_norm_rope(q, k, q, k, positions=pos, rope_theta=1e4)
    with pytest.raises(ValueError, match="Q or K"):
        B.specfold_qk_norm_rope(None, None, None, None)
    with pytest.raises(ValueError, match="positions"):
        B.specfold_qk_norm_rope(q, k, q, k, rope_theta=1e4)
    with pytest.raises(ValueError, match="K_out"):
        B.specfold_qk_norm_rope(q, k, q, torch.zeros(3, 2, 128))
    with pytest.raises(ValueError, match="same rows"):
        B.specfold_qk_norm_rope(q, k[:2], q, k[:2])
    with pytest.raises(ValueError, match="dtype"):
        B.specfold_qk_norm_rope(q, k, q.bfloat16(), k)
    with pytest.raises(ValueError, match="unit last stride"):
        B.specfold_qk_norm_rope(q.transpose(1, 2), None, q, None)


def test_binding_refuses_bad_caches(B):
    pool, table = torch.zeros(32, 2, 64), torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.PagedCache(pool, pool, table, 16)
    with pytest.raises(ValueError, match="whole pages"):
        B.PagedCache(pool, pool, table, 24)
    with pytest.raises(ValueError, match="int32"):
        B.PagedCache(pool, pool, table.long(), 16)
    with pytest.raises(ValueError, match="one shape"):
        B.PagedCache(pool, pool[:, :1], table, 16)


def test_too_many_heads_are_refused(B):
    assert B.MAX_HEADS == 65536
    for n in (B.MAX_HEADS + 1, 2 ** 31 - 1):
        assert _qk(B, n_q=n) == B.ECAPACITY
        assert _qk(B, n_kv=n) == B.ECAPACITY
        assert _append(B, n_kv=n) == B.ECAPACITY
        assert _tree(B, n_q=n, n_kv=n) == B.ECAPACITY
        assert B.tree_attention_workspace_size(B.BF16, n, n, 128, 4) == 0


def test_binding_refuses_missing_outputs(B):
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    for args, what in (((q, k, None, k), "Q_out"), ((q, k, q, None), "K_out"), ((q, None, None, None), "Q_out"),
                       ((None, k, None, None), "K_out"), ((q, k[:, 0], q, k), "K must be"),
                       ((q, k[0, 0], q, k), "K must be")):
        with pytest.raises(ValueError, match=what):
            B.specfold_qk_norm_rope(*args)


def test_append_refuses_sources_in_the_pools(B):
    """Pools of 128 tokens of 1024 bytes, keys at A, values behind them; sources of four rows."""
    size = 128 * 1024
    v = A + size
    cache = _cache(B, v=v)
    far = _hr(B, ptr=A + 4 * size)
    for src in (_hr(B, ptr=A), _hr(B, ptr=v), _hr(B, ptr=A + 4 * 1024), _hr(B, ptr=v + size - 1024),
                _hr(B, ptr=A - 3 * 1024),                               # the last of them the pool's first
                _hr(B, ptr=A + 256), _hr(B, ptr=A + 1024 - 256),        # a head on; a head back, of the next token
                _hr(B, ptr=A + 4096, rs=256), _hr(B, ptr=A + 4096, hs=256)):    # other strides, in the range
        assert _append(B, k=src, v=far, cache=cache) == B.EINVAL
        assert _append(B, k=far, v=src, cache=cache) == B.EINVAL
