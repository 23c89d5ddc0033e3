"""Norm with rotation, append and tree attention at the calls that their
documentation allows beside the ordinary ones."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache_ops import B, DT, ints, make_cache

pytestmark = pytest.mark.gpu
BITS = {"bf16": torch.int16, "f32": torch.int32}


def patterns(rng, shape, dt):
    """Every kind of bit pattern: a fifth of the elements are NaN of either sign
    and any payload, infinities, subnormals or zeros of either sign."""
    info = np.iinfo(np.int16 if dt == "bf16" else np.int32)
    x = rng.integers(info.min, info.max, shape, endpoint=True)
    ones = {"bf16": 0x7F80, "f32": 0x7F800000}[dt]
    kind = rng.integers(0, 20, shape)
    x = np.where(kind < 2, x | ones, np.where(kind == 2, x & ~ones, np.where(kind == 3, x & info.min, x)))
    return torch.from_numpy(x.astype(info.dtype)).cuda().view(DT[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hd,n_kv", [(64, 3), (128, 2), (128, 9)])
@pytest.mark.parametrize("picked", [False, True])
def test_append_copies_bit_for_bit(B, dt, hd, n_kv, picked):
    """Values always, keys where they are neither normed nor rotated."""
    rng = np.random.default_rng(61)
    counts, ctx = [70, 0, 1, 300], [5, 0, 63, 17]
    start = np.concatenate([[0], np.cumsum(counts)])
    T = int(start[-1])
    x = patterns(rng, (2 * T, 2, n_kv, hd), dt)
    rows = rng.integers(0, 2 * T, T) if picked else np.arange(T)
    for theta in (0.0, 1e4):
        cache, table = make_cache(B, rng, dt, hd, n_kv, 16, np.array(ctx) + counts, "fused")
        B.specfold_kv_append(x[:, 0], x[:, 1], cache, ints(start), ints(ctx), rope_theta=theta,
                             rows=ints(rows) if picked else None)
        torch.cuda.synchronize()
        tok = np.concatenate([c + np.arange(n) for c, n in zip(ctx, counts)])
        seq = np.repeat(np.arange(4), counts)
        at = torch.from_numpy(table[seq, tok // 16].astype(np.int64) * 16 + tok % 16).cuda()
        src = torch.from_numpy(rows[:T]).cuda()
        assert torch.equal(cache.v_pool[at].view(BITS[dt]), x[src, 1].contiguous().view(BITS[dt]))
        if theta == 0.0:
            assert torch.equal(cache.k_pool[at].view(BITS[dt]), x[src, 0].contiguous().view(BITS[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9, 3000])
def test_heads_neither_normed_nor_rotated_are_copies(B, dt, T):
    rng = np.random.default_rng(62)
    x = patterns(rng, (T, 9, 128), dt)
    q, k = x[:, :7], x[:, 7:]
    qo, ko = torch.empty_like(q), torch.empty((2, T, 128), device="cuda", dtype=DT[dt]).transpose(0, 1)
    B.specfold_qk_norm_rope(q, k, qo, ko)
    torch.cuda.synchronize()
    assert torch.equal(qo.contiguous().view(BITS[dt]), q.contiguous().view(BITS[dt]))
    assert torch.equal(ko.contiguous().view(BITS[dt]), k.contiguous().view(BITS[dt]))
    # one side normed, the other still a copy
    B.specfold_qk_norm_rope(q, k, qo, ko, gk=torch.ones(128, device="cuda", dtype=DT[dt]))
    torch.cuda.synchronize()
    assert torch.equal(qo.contiguous().view(BITS[dt]), q.contiguous().view(BITS[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["beside", "between heads", "behind", "head-major"])
def test_append_from_the_pools_own_buffer(B, dt, layout):
    """Sources and pools are slices of one buffer that share no element."""
    rng = np.random.default_rng(63)
    tokens, n, n_kv, hd = 96, 40, 3, 64
    if layout == "beside":                              # a token: the pools' heads, then the sources'
        x = patterns(rng, (tokens, 4, n_kv, hd), dt)
        kp, vp, K, V = x[:, 0], x[:, 1], x[:n, 2], x[:n, 3]
    elif layout == "between heads":                     # a head of each in turn
        x = patterns(rng, (tokens, n_kv, 4, hd), dt)
        kp, vp, K, V = x[:, :, 0], x[:, :, 1], x[5:5 + n, :, 2], x[5:5 + n, :, 3]
    elif layout == "behind":
        x = patterns(rng, (2, tokens + n, n_kv, hd), dt)
        kp, vp, K, V = x[0, :tokens], x[1, :tokens], x[0, tokens:], x[1, tokens:]
    else:                                               # head by head, the sources behind each head's pool
        x = patterns(rng, (2, n_kv, tokens + n, hd), dt).transpose(1, 2)
        kp, vp, K, V = x[0, :tokens], x[1, :tokens], x[0, tokens:], x[1, tokens:]
    cache = B.PagedCache(kp, vp, ints(np.arange(12)[None]), 8)
    keep = K.clone(), V.clone()
    B.specfold_kv_append(K, V, cache, ints([0, n]), ints([30]))
    torch.cuda.synchronize()
    for pool, src in ((kp, keep[0]), (vp, keep[1])):
        assert torch.equal(pool[30:30 + n].contiguous().view(BITS[dt]), src.contiguous().view(BITS[dt]))
    with pytest.raises(B.SpecfoldError) as e:           # and from the pool itself
        B.specfold_kv_append(kp[:n], V, cache, ints([0, n]), ints([30]))
    assert e.value.code == B.EINVAL


@pytest.mark.parametrize("writer", ["append", "norm"])
@pytest.mark.parametrize("P", [500, 3000])
def test_prefix_read_right_behind_the_call_that_writes_it(B, writer, P):
    """A contiguous prefix (head-major, which the layer's attention may read before
    it waits), written by append or by norm with rotation, and directly behind it
    the attention alone or the whole layer: the same bits as with a wait between."""
    from diffusion_branch_speculative_gb300 import synth
    from tests.gpu_cases import DeviceInputs
    n_q, n_kv, hd, L = 8, 2, 128, 12
    inp = synth.make_layer_inputs(synth.small_workload(d=512, n_q=n_q, n_kv=n_kv, hd=hd, F=384, P=P, L=L,
                                                       levels=(1, 3, 4)), seed=8)
    dev = DeviceInputs(inp)
    nb = dev.B
    R = nb * L
    bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    page = -(-P // 8) * 8
    pk, pv = (torch.zeros(n_kv, page, hd, **bf).transpose(0, 1) for _ in range(2))
    cache = B.PagedCache(pk, pv, torch.zeros(1, 1, **i32), page)
    start, ctx = ints([0, P]), ints([0])
    ws, cw = B.alloc_workspace(B.workspace_size(dev.dims, nb, L)), B.make_weights(dev.W)
    Q = torch.randn(n_kv, R * (n_q // n_kv), hd, **bf)
    bK, bV = torch.randn(R, n_kv, hd, **bf), torch.randn(R, n_kv, hd, **bf)
    src, packed, n = torch.arange(R, **i32), torch.arange(R, **i32), torch.full((1,), R, **i32)
    gain = torch.ones(hd, **bf)

    def step(whole, wait):
        pk.zero_()
        if writer == "append":
            pv.zero_()
            B.specfold_kv_append(dev.pk, dev.pv, cache, start, ctx, gk=gain)
        else:
            pv[:P] = dev.pv
            torch.cuda.synchronize()
            B.specfold_qk_norm_rope(None, dev.pk, None, pk[:P], gk=gain)
        if wait:
            torch.cuda.synchronize()
        if whole:
            out = torch.empty_like(dev.H)
            B.specfold_layer_forward(dev.dims, cw, dev.H, dev.parent, pk[:P], pv[:P], P, 0.05, out, ws)
        else:
            out = torch.empty(R, n_q * hd, **bf)
            B.specfold_attention(dev.dims, Q, pk[:P], pv[:P], P, bK, bV, src, packed, n, nb, L, out, ws)
        return out

    for whole in (False, True):
        ref = step(whole, True)
        outs = [step(whole, False) for _ in range(20)]
        torch.cuda.synchronize()
        assert B.specfold_get_status(ws) == 0
        assert torch.isfinite(ref).all() and all(torch.equal(o, ref) for o in outs)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_that_name_one_token_leave_elements_of_theirs(B, dt):
    """Forty sequences whose tables share a page write the same eight tokens."""
    n_seqs, n_kv, hd = 40, 5, 128
    gen = torch.Generator(device="cuda").manual_seed(65)
    x = torch.randn(n_seqs * 8, 2, n_kv, hd, device="cuda", generator=gen).to(DT[dt])
    kp, vp = torch.zeros(2, 32, n_kv, hd, device="cuda", dtype=DT[dt])
    cache = B.PagedCache(kp, vp, torch.full((n_seqs, 1), 2, dtype=torch.int32, device="cuda"), 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.specfold_kv_append(x[:, 0], x[:, 1], cache, ints(np.arange(n_seqs + 1) * 8), ints(np.zeros(n_seqs)), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for pool, src in ((kp, x[:, 0]), (vp, x[:, 1])):
        assert (pool[16:24][None] == src.reshape(n_seqs, 8, n_kv, hd)).any(0).all()
        assert (pool[:16] == 0).all() and (pool[24:] == 0).all()
