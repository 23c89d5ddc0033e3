// Tree attention with many rows a head group on the 5th-generation tensor
// cores.  A unit's piece (tree_sched.cuh) is 128 query rows of one sequence's
// key/value head over a run of 128-key blocks of its cache.
//
// A block is worked in two halves of 64 keys, h = 0, 1, that run independently
// within a piece: S_h = Q K_h^T and O_h += P_h V_h are tcgen05.mma into TMEM
// (two S buffers per half, so the next S overlaps the softmax; one O per half),
// each half with its own running maximum and sum.  P_h (bf16, the tensor cores'
// operand: each weight off by half a step) goes over the half's own keys,
// which S_h has finished with.  The halves merge once at the end of a piece.
//
// Roles (384 threads): warps 0-1 load, warps 2 and 3 issue half 0's and half
// 1's products (warp 3 owns the TMEM allocation), warps 4-11 are two threads
// per query row, one per half.  Blocks of cached tokens alone come by TMA, one
// box per run of tokens inside a page (page_size's power of two, 8 to 64), the
// boxes issued by the loaders' lanes side by side; blocks that hold the tree's
// tokens, or end the sequence, are gathered row by row, zero-filled past the
// end.  Which of them a row sees is 64 bits a half, found by walking up its
// ancestors when such a block is met.
#include "tree_sched.cuh"

namespace sf {
namespace {

constexpr int kTcThreads = 384;
constexpr int kLoaders = 64;
constexpr int kAtom = 128 * 128;  // one 128-row x 128-byte swizzle block
constexpr int kOddBufs = 4;       // units whose odd-value notes may be alive at once

struct TcArgs {
  CUtensorMap mapK, mapV;  // {dim, heads, pool tokens}, box {64, 1, box}
  TreeArgs t;
  int box;  // tokens of a box
};

template <int HD>
struct Tc {
  static constexpr int NATOM = HD / 64;
  static constexpr int Q_BYTES = kAtom * NATOM;
  static constexpr int KV_BYTES = kAtom * NATOM;  // one K (or V) tile of 128 keys
  // K half by half: keys [64h, 64h + 64) at h * KH_BYTES in NATOM swizzle atoms
  // of 64 rows, so that P_h may go over them
  static constexpr int KH_BYTES = KV_BYTES / 2;
  static constexpr int KH_ATOM = 64 * 128;
  static constexpr int PH_BYTES = kAtom;  // P of one half: 128 rows x 64 keys
  static constexpr int STAGES = 3;
  static constexpr bool P_IN_K = PH_BYTES <= KH_BYTES;
  static constexpr int OFF_KV = Q_BYTES;  // stage s: K (then P) at +2s*KV, V at +(2s+1)*KV
  static constexpr int OFF_P = OFF_KV + 2 * STAGES * KV_BYTES;
  static constexpr int SMEM = OFF_P + (P_IN_K ? 0 : STAGES * 2 * PH_BYTES) + 1024;  // and the base's alignment
  static constexpr int p_off(int stage, int h) {
    return P_IN_K ? OFF_KV + 2 * stage * KV_BYTES + h * KH_BYTES : OFF_P + (2 * stage + h) * PH_BYTES;
  }
  // TMEM: S of half h, buffer b at columns (2h + b) * 64; O of half h at COL_O + h * HD
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_O = 256;
};

// The ancestors (and itself) of node i among nodes [e0, e0 + 64), as bits, for
// a node that is no padding row.  par: the sequence's parents, null: a chain.
SF_DEV uint64_t sees_window(const int32_t* par, int i, int e0, uint32_t* status) {
  if (!par) {
    const int hi = min(i - e0, 63);
    return hi < 0 ? 0ull : (~0ull >> (63 - hi)) & (e0 < 0 ? ~0ull << min(-e0, 63) : ~0ull);
  }
  uint64_t bits = 0ull;
  int a = i, up = par[i];
  while (a >= e0) {
    if (a < e0 + 64) bits |= 1ull << (a - e0);
    if (up == -1) break;
    int above = SPECFOLD_TREE_PAD;
    if (up >= 0 && up < a) above = par[up];
    if (above == SPECFOLD_TREE_PAD) {  // not a parent
      atomicOr(status, SPECFOLD_DEV_BAD_PARENT);
      break;
    }
    a = up;
    up = above;
  }
  return bits;
}

template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1) tree_attn_tc_kernel(const __grid_constant__ TcArgs ta) {
  using C = Tc<HD>;
  const TreeArgs& p = ta.t;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[25];
  __shared__ uint32_t tmem_slot_s;
  __shared__ volatile int abort_s;
  __shared__ volatile int okflag[C::STAGES];
  __shared__ volatile int okq;
  __shared__ float2 xch[128];
  __shared__ TreeLocate loc;
  // nodes whose values are not all finite, by unit (see the loaders)
  __shared__ uint32_t odd[kOddBufs][SPECFOLD_MAX_TREE / 32];
  uint64_t* q_full = bars + 0;
  uint64_t* kv_full = bars + 1;   // [STAGES]
  uint64_t* kv_empty = bars + 4;  // [STAGES]: both halves' P V of the block are done
  uint64_t* s_full = bars + 7;    // [half][2]
  uint64_t* s_free = bars + 11;   // [half][2]
  uint64_t* p_full = bars + 15;   // [half][2], alternating by block: never two phases ahead of its reader
  uint64_t* o_full = bars + 19;   // [half]: one completion per P V product of the half
  uint64_t* q_empty = bars + 21;  // both halves' S products of a unit are done: Q may be replaced
  uint64_t* o_empty = bars + 22;  // the softmax warps have read a unit's outputs
  uint64_t* drain = bars + 23;    // [half]
  volatile int* abort_flag = &abort_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  TreeWalk w;
  if (!tree_locate<kTcThreads>(p, loc, w)) {
    if (threadIdx.x == 0) tree_describe_none(p);
    return;
  }
  if (threadIdx.x == 0) {
    tree_describe(p, w, loc.per, loc.lo);
    mbar_init(smem_u32(q_full), 1);
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&kv_full[i]), 1);
      mbar_init(smem_u32(&kv_empty[i]), 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_free[i]), 128);
      mbar_init(smem_u32(&p_full[i]), 128);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_u32(&o_full[h]), 1);
      mbar_init(smem_u32(&drain[h]), 1);
    }
    mbar_init(smem_u32(q_empty), 2);
    mbar_init(smem_u32(o_empty), 256);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(&tmem_slot_s), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot_s;
  const int g = p.g;

  // Every role walks the same pieces in the same order; gt counts this CTA's
  // blocks so far (ring stage and phases), j its pieces.
  if (warp < 2) {
    // ------------------------------------------------------------ loaders --
    const int lt = threadIdx.x;
    int gt = 0, j = 0, issued = -1;
    bool ok = true;
    if (lt == 0) {
      prefetch_tmap(&ta.mapK);
      prefetch_tmap(&ta.mapV);
    }
    const int boxes = kTreeTcKeys / ta.box;
    const int pool = p.cache.num_pages * p.cache.page_size;
    for (; w.left > 0 && ok; w.next(p), ++j) {
      const int h = w.head(), m0 = tree_m0(p, w), rows = tree_tile_rows(p, w), ctx = w.q.ctx, len = ctx + w.q.n;
      const int nt = w.blocks();
      // pool token of this lane's box of block b (boxes by lane: warp 0's for
      // K, warp 1's for V); read one block ahead of its use
      auto box_token = [&](int b) {
        const int tok = b * kTreeTcKeys + lane * ta.box;
        if (lane >= boxes || b >= w.b0 + nt || (b + 1) * kTreeTcKeys > ctx) return 0;
        const int at = tree_pool_token(p, w.s, tok);
        return at < 0 ? pool : at;  // wholly past the pool: the box reads zeros
      };
      int z = box_token(w.b0);
      // the previous unit's S products must be done with the Q buffer
      if (lt == 0)
        okq = j == 0 || mbar_wait(smem_u32(q_empty), (j - 1) & 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnQEmpty);
      named_bar_sync(1, kLoaders);
      if (!okq) {
        ok = false;
        break;
      }
      if (lt < SPECFOLD_MAX_TREE / 32) odd[j % kOddBufs][lt] = 0u;
#pragma unroll
      for (int q = 0; q < 128 / kLoaders; ++q) {
        const int r = lt + q * kLoaders, m = m0 + r;
        const uint32_t n = r < rows ? 16u : 0u;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q);
        if (r < rows) src += (w.q.row0 + m / g) * p.q_rs + (h * g + m % g) * p.q_hs;
#pragma unroll
        for (int c = 0; c < HD / 8; ++c)
          cp_async16(smem_u32(smem + (c >> 3) * kAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4)), src + c * 8, n);
      }
      for (int t = 0; t < nt; ++t, ++gt) {
        const int b = w.b0 + t;
        const int st = gt % C::STAGES;
        const bool whole = (b + 1) * kTreeTcKeys <= ctx;  // cached tokens alone
        const uint32_t fb = smem_u32(&kv_full[st]);
        if (lt == 0) {
          const bool free = mbar_wait(smem_u32(&kv_empty[st]), ((gt / C::STAGES) & 1) ^ 1, abort_flag, p.status,
                                      kWaitLimitNs, kSiteAttnKvEmpty);
          if (free && whole) {
            mbar_arrive_expect_tx(fb, 2 * C::KV_BYTES);
            issued = gt;
          }
          okflag[st] = free;
        }
        named_bar_sync(1, kLoaders);
        if (!okflag[st]) {
          ok = false;
          break;
        }
        uint8_t* sK = smem + C::OFF_KV + (2 * st) * C::KV_BYTES;
        uint8_t* sV = sK + C::KV_BYTES;
        if (whole) {
          if (lane < boxes) {
            const int r = lane * ta.box;  // first row of the box in the block
            for (int a = 0; a < C::NATOM; ++a) {
              if (warp == 0)
                tma_load_3d(smem_u32(sK + (r >> 6) * C::KH_BYTES + a * C::KH_ATOM + (r & 63) * 128), &ta.mapK, fb,
                            a * 64, h, z);
              else
                tma_load_3d(smem_u32(sV + a * kAtom + r * 128), &ta.mapV, fb, a * 64, h, z);
            }
          }
          z = box_token(b + 1);
        } else {
          // gathered rows: every row's pool token first, then its 16-byte
          // pieces straight to their swizzled places, all in flight at once
          constexpr int RPT = 128 / kLoaders;
          int at[RPT];
#pragma unroll
          for (int q = 0; q < RPT; ++q) {
            const int tok = b * kTreeTcKeys + lt + q * kLoaders;
            at[q] = tok < len ? tree_pool_token(p, w.s, tok) : -1;
          }
#pragma unroll
          for (int q = 0; q < RPT; ++q) {
            const int kr = lt + q * kLoaders, kh = kr >> 6, kq = kr & 63;
            const uint32_t n = at[q] < 0 ? 0u : 16u;
            const long long tk = max(at[q], 0);  // any valid address when nothing is read
            const __nv_bfloat16* ks =
                static_cast<const __nv_bfloat16*>(p.cache.k) + tk * p.cache.k_token_stride + h * p.cache.k_head_stride;
            const __nv_bfloat16* vs =
                static_cast<const __nv_bfloat16*>(p.cache.v) + tk * p.cache.v_token_stride + h * p.cache.v_head_stride;
#pragma unroll
            for (int c = 0; c < HD / 8; ++c) {
              const int sw = ((c & 7) ^ (kr & 7)) << 4;
              cp_async16(smem_u32(sK + kh * C::KH_BYTES + (c >> 3) * C::KH_ATOM + kq * 128 + sw), ks + c * 8, n);
              cp_async16(smem_u32(sV + (c >> 3) * kAtom + kr * 128 + sw), vs + c * 8, n);
            }
          }
          cp_async_commit();
          cp_async_wait<0>();
          // A weight of zero does not silence an infinite value or a NaN in a
          // product: such values of the tree's tokens are taken out here, noted,
          // and added at the end to the rows that see them.
#pragma unroll
          for (int q = 0; q < RPT; ++q) {
            const int kr = lt + q * kLoaders, e = b * kTreeTcKeys + kr - ctx;
            if (e < 0 || at[q] < 0) continue;
            bool note = false;
#pragma unroll
            for (int c = 0; c < HD / 8; ++c) {
              uint4* v = reinterpret_cast<uint4*>(sV + (c >> 3) * kAtom + kr * 128 + (((c & 7) ^ (kr & 7)) << 4));
              uint4 u = *v;
              bool mine = false;
              uint32_t* x = &u.x;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((x[k] & 0x7f80u) == 0x7f80u) x[k] &= 0xffff0000u, mine = true;
                if ((x[k] & 0x7f800000u) == 0x7f800000u) x[k] &= 0xffffu, mine = true;
              }
              if (mine) *v = u;
              note = note || mine;
            }
            if (note) atomicOr(&odd[j % kOddBufs][e >> 5], 1u << (e & 31));
          }
          fence_proxy_async_smem();
          named_bar_sync(1, kLoaders);
          if (lt == 0) mbar_arrive(fb);
          z = box_token(b + 1);
        }
        if (t == 0) {  // the queries, behind the first block's loads
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async_smem();
          named_bar_sync(1, kLoaders);
          if (lt == 0) mbar_arrive(smem_u32(q_full));
        }
      }
    }
    if (lt == 0 && *abort_flag && issued >= 0) {
      // let the copies already issued land before the CTA exits
      int never = 0;
      mbar_wait(smem_u32(&kv_full[issued % C::STAGES]), (issued / C::STAGES) & 1, &never, nullptr, 10000000ull);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax --
    // Half hf of a row owns keys [64 hf, 64 hf + 64) of every block.  It raises
    // its reference maximum m, and rescales O_hf in place, only when the maximum
    // grows by more than 2^8, so its weights stay below 2^8.  At the end, with
    // M = max(m_0, m_1) and w_h = 2^(m_h - M), the row's output is (w_0 O_0 + w_1
    // O_1) / (w_0 l_0 + w_1 l_1), half hf writing columns [hf HD/2, (hf + 1) HD/2).
    const int qw = warp & 3;
    const int hf = (warp - 4) >> 2;
    const int row = qw * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(qw * 32) << 16;
    constexpr int OH = HD / 2;
    const uint32_t to_own = tmem + lane_off + C::COL_O + hf * HD;
    const int pair_bar = 2 + qw;  // named barrier of the two warps sharing these rows
    int gt = 0, j = 0;
    bool ok = true;
    for (bool first = true; w.left > 0 && ok; first = false, w.next(p)) {
      const int h = w.head(), m = tree_m0(p, w) + row, ctx = w.q.ctx, nt = w.blocks();
      const bool valid = row < tree_tile_rows(p, w);
      const int node = valid ? m / g : 0;
      const int32_t* par = p.parent ? p.parent + w.q.row0 : nullptr;
      const bool dead = !valid || (par && par[node] == SPECFOLD_TREE_PAD);  // sees nothing
      float m_ref = -INFINITY, l = 0.f;
      for (int t = 0; t < nt; ++t) {
        const int gi = gt + t;
        const int sb = gi & 1;
        const int key0 = (w.b0 + t) * kTreeTcKeys + hf * 64;  // first key of this half
        const bool allv = key0 + 64 <= ctx;
        // what the row sees of these 64 keys: cached tokens, its ancestors
        uint64_t km = ~0ull;
        if (!allv) {
          const int e0 = key0 - ctx;
          km = dead ? 0ull : sees_window(par, node, e0, p.status);
          if (e0 < 0 && !dead) km |= (1ull << -e0) - 1ull;  // -e0 < 64 here
        }
        // every wait's outcome is made warp-uniform: a lane whose wait ran out
        // takes its whole warp along
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s_full[2 * hf + sb]), (gi >> 1) & 1, abort_flag, p.status,
                                               kWaitLimitNs, kSiteAttnSFull))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ts = tmem + lane_off + (2 * hf + sb) * 64;
        uint32_t sv[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(ts + c * 32, sv[c]);
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld_wait(sv[c]);
        tc_fence_before();
        mbar_arrive(smem_u32(&s_free[2 * hf + sb]));  // the S buffer may be refilled now
        float mx8[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) mx8[q] = -INFINITY;
        if (allv) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) mx8[e & 7] = fmaxf(mx8[e & 7], __uint_as_float(sv[c][e]));
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              mx8[e & 7] = fmaxf(mx8[e & 7], ((km >> (32 * c + e)) & 1u) ? __uint_as_float(sv[c][e]) : -INFINITY);
        }
        const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                               fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        const float m_new = fmaxf(m_ref, mx * p.sl2);
        float alpha = 1.f;
        bool rescale = false;
        if (m_ref == -INFINITY) {
          m_ref = m_new;  // nothing accumulated yet (every earlier weight was 0)
        } else if (m_new > m_ref + 8.f) {
          alpha = ex2(m_ref - m_new);
          m_ref = m_new;
          rescale = true;
        }
        l *= alpha;
        // O_hf may only be rescaled once it holds the previous block's P V
        bool rescale_waited = false;
        if (t >= 1 && __any_sync(0xffffffffu, rescale)) {
          rescale_waited = true;
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&o_full[hf]), (gi - 1) & 1, abort_flag, p.status,
                                                 kWaitLimitNs, kSiteAttnRescale))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t r[32];
            tmem_ld32(to_own + c * 32, r);
            tmem_ld_wait(r);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st32(to_own + c * 32, r);
          }
          tmem_st_wait();
        }
        // weights -> bf16 P_hf (128 rows x 64 keys, K-major, 128-byte swizzle)
        uint8_t* sP = smem + C::p_off(gi % C::STAGES, hf);
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
          if (allv) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float x0 = ex2(fmaf(__uint_as_float(sv[c][e]), p.sl2, -m_ref));
              const float x1 = ex2(fmaf(__uint_as_float(sv[c][e + 1]), p.sl2, -m_ref));
              ls[(e >> 1) & 3] += x0 + x1;
              pk[e / 2] = pack_bf16x2(x0, x1);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float pv[2];
#pragma unroll
              for (int uu = 0; uu < 2; ++uu) {
                const float x = ex2(fmaf(__uint_as_float(sv[c][e + uu]), p.sl2, -m_ref));
                pv[uu] = ((km >> (32 * c + e + uu)) & 1u) ? x : 0.f;
              }
              ls[(e >> 1) & 3] += pv[0] + pv[1];
              pk[e / 2] = pack_bf16x2(pv[0], pv[1]);
            }
          }
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const int kc = c * 4 + q4;  // 8-key piece of the half
            const int off = row * 128 + ((kc ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(sP + off) = make_uint4(pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]);
          }
        }
        l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        // A parity wait is exact only while its barrier cannot run two phases
        // ahead: the piece's last block waits for the P V before it here, so
        // that afterwards only the last P V is out.
        if (t == nt - 1 && t >= 1 && !rescale_waited) {
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&o_full[hf]), (gi - 1) & 1, abort_flag, p.status,
                                                 kWaitLimitNs, kSiteAttnLastP))) {
            ok = false;
            break;
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&p_full[2 * hf + sb]));
      }
      const int glast = gt + nt - 1;
      const bool oku = ok && mbar_wait(smem_u32(&o_full[hf]), glast & 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnEnd);
      // the halves' meeting: both leave together or neither.  Half 1 hands its
      // (m, l) to half 0, which computes the merge's factors and hands half 1
      // its pair back; the first barrier also orders half 0's reads of the
      // previous unit's hand-back before this write.
      const bool whole = w.whole();
      if (hf == 1) xch[row] = make_float2(m_ref, l);
      tc_fence_before();
      __syncwarp();
      if (!named_bar_and(pair_bar, 64, oku)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float a0 = 0.f, a1 = 0.f, M = 0.f, lrow = 0.f;
      if (hf == 0) {
        const float2 o1 = xch[row];
        M = fmaxf(m_ref, o1.x);
        const float w0 = merge_weight(m_ref, M), w1 = merge_weight(o1.x, M);
        lrow = w0 * l + w1 * o1.y;
        const float sc = whole ? merge_scale(lrow) : 1.f;  // a partial stays unnormalised
        a0 = w0 * sc;
        a1 = w1 * sc;
        xch[row] = make_float2(a0, a1);
      }
      named_bar_sync(pair_bar, 64);
      if (hf == 1) {
        const float2 f = xch[row];
        a0 = f.x;
        a1 = f.y;
      }
      const uint32_t t0 = tmem + lane_off + C::COL_O + hf * OH;  // columns [hf OH, (hf + 1) OH) of O_0
      const uint32_t t1 = t0 + HD;                                // ... and of O_1
      uint32_t any_odd = 0u;
#pragma unroll
      for (int k = 0; k < SPECFOLD_MAX_TREE / 32; ++k) any_odd |= odd[j % kOddBufs][k];
      const size_t pr = static_cast<size_t>(tree_slot(first)) * p.tile_rows + row;
      float* po = p.part_o + pr * HD + hf * OH;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + (w.q.row0 + node) * p.o_rs +
                           (h * g + (valid ? m % g : 0)) * p.o_hs + hf * OH;
#pragma unroll
      for (int c = 0; c < OH / 32; ++c) {
        uint32_t r0[32], r1[32];
        tmem_ld32(t0 + c * 32, r0);
        tmem_ld32(t1 + c * 32, r1);
        tmem_ld_wait(r0);
        tmem_ld_wait(r1);
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = dead ? 0.f : a0 * __uint_as_float(r0[e]) + a1 * __uint_as_float(r1[e]);
        if (any_odd && !dead) {  // rare: infinities and NaN among the tree's values
          for (int i = 0; i <= node; ++i) {
            const int tok = ctx + i;
            if (!(odd[j % kOddBufs][i >> 5] >> (i & 31) & 1u)) continue;
            if (tok < w.b0 * kTreeTcKeys || tok >= (w.b0 + nt) * kTreeTcKeys) continue;
            if (!(sees_window(par, node, i, p.status) & 1ull)) continue;
            const int at = tree_pool_token(p, w.s, tok);
            if (at < 0) continue;
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.cache.v) +
                                     static_cast<long long>(at) * p.cache.v_token_stride + h * p.cache.v_head_stride +
                                     hf * OH + c * 32;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float x = __bfloat162float(v[e]);
              if (!isfinite(x)) o[e] += x;
            }
          }
        }
        if (valid && whole) {
#pragma unroll
          for (int q8 = 0; q8 < 4; ++q8)
            reinterpret_cast<uint4*>(dst)[c * 4 + q8] =
                make_uint4(pack_bf16x2(o[8 * q8], o[8 * q8 + 1]), pack_bf16x2(o[8 * q8 + 2], o[8 * q8 + 3]),
                           pack_bf16x2(o[8 * q8 + 4], o[8 * q8 + 5]), pack_bf16x2(o[8 * q8 + 6], o[8 * q8 + 7]));
        } else if (valid) {
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4)
            reinterpret_cast<float4*>(po + c * 32)[q4] =
                make_float4(o[4 * q4], o[4 * q4 + 1], o[4 * q4 + 2], o[4 * q4 + 3]);
        }
        __syncwarp();  // the next load of TMEM is the whole warp's
      }
      if (!whole && valid && hf == 0) {
        p.part_ml[pr * 2] = dead ? -INFINITY : M;
        p.part_ml[pr * 2 + 1] = dead ? 0.f : lrow;
      }
      // the accumulators are free for the next unit's first P V products
      tc_fence_before();
      mbar_arrive(smem_u32(o_empty));
      gt += nt;
      ++j;
    }
  } else {
    // ---------------------------------------------------------------- MMA --
    const int hm = warp - 2;
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16_f32(128, 64, false);
      constexpr uint32_t idPV = idesc_bf16_f32(128, HD, true);
      const uint32_t aQ = smem_u32(smem);
      const uint32_t tO = tmem + C::COL_O + hm * HD;
      int gt = 0, j = 0;
      bool ok = true;
      // P_h V_h of block gi (first: the unit's first block, which overwrites
      // O_h: the softmax warps have read the previous unit's by then)
      auto issue_pv = [&](int gi, bool first) -> bool {
        if (!mbar_wait(smem_u32(&p_full[2 * hm + (gi & 1)]), (gi >> 1) & 1, abort_flag, p.status, kWaitLimitNs,
                       kSiteAttnPFull))
          return false;
        tc_fence_after();
        const int kst = gi % C::STAGES;
        const uint32_t aP = smem_u32(smem + C::p_off(kst, hm));
        const uint32_t aV = smem_u32(smem + C::OFF_KV + (2 * kst + 1) * C::KV_BYTES);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          tc_mma_f16(tO, sdesc_sw128(aP + kk * 32, 16, 1024), sdesc_sw128(aV + (4 * hm + kk) * 2048, kAtom, 1024),
                     idPV, (!first || kk > 0) ? 1u : 0u);
        }
        tc_commit(smem_u32(&o_full[hm]));
        tc_commit(smem_u32(&kv_empty[kst]));
        return true;
      };
      for (; w.left > 0 && ok; w.next(p)) {
        const int nt = w.blocks();
        if (!mbar_wait(smem_u32(q_full), j & 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnQFull)) break;
        for (int t = 0; t < nt && ok; ++t) {
          const int gi = gt + t;
          const int sb = gi & 1;
          const int kst = gi % C::STAGES;
          if (!mbar_wait(smem_u32(&kv_full[kst]), (gi / C::STAGES) & 1, abort_flag, p.status, kWaitLimitNs,
                         kSiteAttnKvFull) ||
              !mbar_wait(smem_u32(&s_free[2 * hm + sb]), ((gi >> 1) & 1) ^ 1, abort_flag, p.status, kWaitLimitNs,
                         kSiteAttnSFree)) {
            ok = false;
            break;
          }
          // Before the unit's second S (or its only P V): both halves have
          // read the previous unit's outputs.  Waiting here, not just before
          // the first P V, keeps p_full exact: with S(1) not yet issued, the
          // softmax can hand over at most block 0's P before the wait for it.
          if (t == 1 && j >= 1 &&
              !mbar_wait(smem_u32(o_empty), (j - 1) & 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnOEmpty)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t aK = smem_u32(smem + C::OFF_KV + (2 * kst) * C::KV_BYTES + hm * C::KH_BYTES);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            tc_mma_f16(tmem + (2 * hm + sb) * 64, sdesc_sw128(aQ + (kk >> 2) * kAtom + (kk & 3) * 32, 16, 1024),
                       sdesc_sw128(aK + (kk >> 2) * C::KH_ATOM + (kk & 3) * 32, 16, 1024), idS, kk > 0 ? 1u : 0u);
          }
          tc_commit(smem_u32(&s_full[2 * hm + sb]));
          if (t == nt - 1) tc_commit(smem_u32(q_empty));  // Q is read by no later product of this unit
          if (t >= 1 && !issue_pv(gi - 1, t == 1)) ok = false;
        }
        if (!ok) break;
        if (nt == 1 && j >= 1 &&
            !mbar_wait(smem_u32(o_empty), (j - 1) & 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnOEmpty))
          break;
        if (!issue_pv(gt + nt - 1, nt == 1)) break;
        gt += nt;
        ++j;
      }
      tc_commit(smem_u32(&drain[hm]));
      int never = 0;
      mbar_wait(smem_u32(&drain[hm]), 0, &never, nullptr, 10000000ull);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int HD>
int tc_go(const TreeArgs& a, int grid, cudaStream_t st) {
  using C = Tc<HD>;
  TcArgs ta;
  ta.t = a;
  const specfold_paged_cache& c = a.cache;
  ta.box = c.page_size % 64 == 0 ? 64 : c.page_size % 32 == 0 ? 32 : c.page_size % 16 == 0 ? 16 : 8;
  const uint64_t tokens = static_cast<uint64_t>(c.num_pages) * c.page_size;
  if (const int rc = make_map_3d(&ta.mapK, c.k, HD, a.n_kv, tokens, c.k_head_stride, c.k_token_stride, ta.box)) return rc;
  if (const int rc = make_map_3d(&ta.mapV, c.v, HD, a.n_kv, tokens, c.v_head_stride, c.v_token_stride, ta.box)) return rc;
  if (const int rc = smem_limit_once(tree_attn_tc_kernel<HD>, C::SMEM)) return rc;
  launch_k(tree_attn_tc_kernel<HD>, dim3(grid), dim3(kTcThreads), C::SMEM, st, ta);
  count_launch();
  return check_launch();
}

}  // namespace

int launch_tree_tc(const TreeArgs& a, int hd, int grid, cudaStream_t st) {
  return hd == 128 ? tc_go<128>(a, grid, st) : tc_go<64>(a, grid, st);
}

}  // namespace sf
