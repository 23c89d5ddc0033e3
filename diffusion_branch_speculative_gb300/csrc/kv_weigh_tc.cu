// Attention weights of many rows a head group, bf16, on the 5th-generation tensor
// cores (specfold_kv_weigh; kv_weigh.cuh has the two launches' division).  The
// scores are too many to keep, so both launches compute them, each with the
// operand order that leaves its reduction inside a thread:
//   statistics  S = Q K^T, a thread a query row: its maximum and sum over the keys
//   weights     S = K Q^T, a thread a key: the sum of 2^(x - m) / l over the rows
// A row-major tile is either operand as it lies, so both read the same K and Q
// tiles.  Keys come by TMA through a ring, as in tree_attn_tc.cu, whose roles these
// are (384 threads): warp 0 loads keys, warps 1 and 3 gather queries, warp 2 issues
// the products, warps 4 to 11 reduce.  A score costs one product and one
// exponential a launch.
//
// Up to about 100 rows a group the memory bounds it, which has to deliver the keys
// twice: 32 rows of 24 / 8 heads over 4 x 32700 tokens, 2 x 217 MB, take 72 to 74 us, 5870 to
// 6030 GB/s or 0.87 to 0.89 of the copy rate (44 us a launch alone and cold, DRAM 63 % and
// tensor cores 26 and 18 % busy, 8 us of it the start; the two cannot share an SM).  Beyond,
// neither memory nor a unit does: 252 rows (36 of 28 / 4 heads) take 64 us
// for 2 x 107 MB, 896 rows 250 us, where a tile of 256 rows takes 0.95 us a block in the
// first launch and 1.7 in the second.  Of 896 rows the first launch has the exponentials' unit
// 48 % busy and the tensor cores 44 %; the second 25 % and 19 %, shared memory 17 %, DRAM 8 %, and
// its warps wait: a half has one buffer of 128 keys by 256 rows, whose next product starts
// when the reads of the one before are done.  Keeping a part of the keys in L2 from one launch to
// the next by hints saves 1 to 2 us; the scores of 96 rows would be 1.5 times the keys.
#include "kv_weigh.cuh"
#include "weigh_order.h"

namespace sf {
namespace {

constexpr int kTcThreads = 384;
constexpr int kAtom = 128 * 128;  // one 128-row x 128-byte swizzle block
constexpr int kBlock = kWeighTcKeys;

struct WTcArgs {
  CUtensorMap mapK;  // {dim, heads, pool tokens}, box {64, 1, box}
  WeighArgs a;
  int box;
};

template <int HD>
struct WTc {
  static constexpr int NATOM = HD / 64;
  static constexpr int Q_ATOM = 2 * kAtom;      // 64 dimensions of 256 query rows
  static constexpr int TILE = kAtom * NATOM;    // 128 keys
  static constexpr int RING = HD == 128 ? 4 : 8;
  static constexpr int OFF_RING = Q_ATOM * NATOM;
  static constexpr int SMEM = OFF_RING + RING * TILE + 1024;  // and the base's alignment
};

// Keys of a run's blocks, one TMA box per run of tokens inside a page: warp 0.
// Returns false if a wait ran out.  BACK: the last block first (see the weights'
// kernel).
template <int HD, bool BACK>
struct KeyLoader {
  using C = WTc<HD>;
  int it = 0;
  SF_DEV bool piece(const WTcArgs& ta, const TreeWalk& w, uint8_t* smem, uint64_t* full, uint64_t* empty,
                    volatile int* abort_flag) {
    const TreeArgs& p = ta.a.t;
    const int lane = threadIdx.x & 31;
    const int ps = p.cache.page_size, pool = p.cache.num_pages * ps, len = w.q.ctx + w.q.n;
    const int box = lane & 15, atom = lane >> 4;  // what this thread issues of a tile
    const bool issues = box < kBlock / ta.box && atom < C::NATOM;
    // the table's entry is read a tile ahead of its use and looked at only then
    const unsigned tok0 = static_cast<unsigned>(w.b0 + (BACK ? w.n - 1 : 0)) * kBlock + box * ta.box;
    int pg = tok0 / static_cast<unsigned>(ps), off = tok0 - pg * ps;
    const int dpg = kBlock / ps, doff = kBlock - dpg * ps;
    const int32_t* table = p.cache.block_table + w.s * p.cache.table_stride;
    long long left = static_cast<long long>(len) - tok0;
    auto entry = [&](int t) { return issues && t < w.n && left > 0 && pg < p.cache.table_pages ? table[pg] : -1; };
    int page = entry(0);
    const uint64_t once = policy_evict_first();
    for (int t = 0; t < w.n; ++t, ++it) {
      const int st = it % C::RING;
      const uint32_t fb = smem_u32(&full[st]);
      bool ok = true;
      if (lane == 0) {
        ok = mbar_wait(smem_u32(&empty[st]), ((it / C::RING) & 1) ^ 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnKvEmpty);
        if (ok) mbar_arrive_expect_tx(fb, C::TILE);
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
      if (issues) {
        const bool there = page >= 0 && page < p.cache.num_pages;
        if (!there && left > 0) atomicOr(p.status, SPECFOLD_DEV_BAD_PAGE);
        // a box without a page lies wholly past the pool: it reads zeros
        tma_load_3d_hint(smem_u32(smem + C::OFF_RING + st * C::TILE + atom * kAtom + box * ta.box * 128), &ta.mapK, fb,
                         atom * 64, w.head, there && left > 0 ? page * ps + off : pool, once);
      }
      if constexpr (BACK) {
        left += kBlock;
        pg -= dpg;
        off -= doff;
        if (off < 0) {
          off += ps;
          --pg;
        }
      } else {
        left -= kBlock;
        pg += dpg;
        off += doff;
        if (off >= ps) {
          off -= ps;
          ++pg;
        }
      }
      page = entry(t + 1);
    }
    return true;
  }
  // let the copies already issued land before the CTA exits
  SF_DEV void drain(uint64_t* full, volatile int* abort_flag) {
    if ((threadIdx.x & 31) == 0 && *abort_flag) ring_land(full, C::RING, it - 1);
    __syncwarp();
  }
};

// A tile's queries by THREADS threads (tid 0 ..): `most` rows from m0 on, those past
// the last the copies of it (zeros times an infinite key would be NaN).  Returns with
// this thread's part visible to the tensor cores.
template <int HD, int THREADS>
SF_DEV void gather_rows(const WeighArgs& a, const TreeWalk& w, int m0, int rows, int most, uint8_t* smem, int tid) {
  constexpr int CPR = HD / 8, RSTEP = THREADS / CPR;  // rows of one step; a row's node and head follow by steps
  const TreeArgs& p = a.t;
  const int c = tid % CPR, g = p.g, dn = RSTEP / g, dj = RSTEP % g;
  const uint32_t at = smem_u32(smem) + (c >> 3) * WTc<HD>::Q_ATOM;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + w.head * g * p.q_hs + c * 8;
  auto from = [&](int node, int j) {
    const int t = w.q.row0 + node;
    return q + (a.rows ? max(weigh_src(a, t), 0) : t) * p.q_rs + j * p.q_hs;
  };
  const __nv_bfloat16* last = from((m0 + rows - 1) / g, (m0 + rows - 1) % g);
  int node = (m0 + tid / CPR) / g, j = (m0 + tid / CPR) - node * g;
#pragma unroll 4
  for (int r = tid / CPR; r < most; r += RSTEP) {
    cp_async16(at + r * 128 + (((c & 7) ^ (r & 7)) << 4), r < rows ? from(node, j) : last, 16u);
    node += dn;
    j += dj;
    if (j >= g) {
      j -= g;
      ++node;
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  fence_proxy_async_smem();
}

// D[128 x n] = A B^T over the HD dimensions of two tiles in shared memory.
template <int HD>
SF_DEV void tile_product(bool me, uint32_t d, uint32_t at_a, uint32_t a_atom, uint32_t at_b, uint32_t b_atom, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    warp_mma(me, d, sdesc_sw128(at_a + (kk >> 2) * a_atom + (kk & 3) * 32, 16, 1024),
             sdesc_sw128(at_b + (kk >> 2) * b_atom + (kk & 3) * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
}

// ------------------------------------------------------------- statistics --
// Two lanes of 128 rows as in tree_attn_tc.cu: their own rows and every block, or,
// of a tile of at most 128 rows, the same rows and alternate blocks.  A lane has
// two score buffers, so the products run ahead.
template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1) weigh_stats_tc_kernel(const __grid_constant__ WTcArgs ta) {
  using C = WTc<HD>;
  const WeighArgs& a = ta.a;
  const TreeArgs& p = a.t;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[2 * C::RING + 11];
  __shared__ uint32_t tmem_slot_s;
  __shared__ volatile int abort_s;
  __shared__ float2 xch[2][128];
  uint64_t* full = bars;
  uint64_t* empty = bars + C::RING;    // the lanes' two arrivals
  uint64_t* q_full = bars + 2 * C::RING;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;       // [lane * 2 + buffer]
  uint64_t* s_free = q_full + 6;       // [lane * 2 + buffer], a warp an arrival
  uint64_t* drain = q_full + 10;
  volatile int* abort_flag = &abort_s;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 2);
    }
    mbar_init(smem_u32(q_full), 2);   // the gathering warps, or the lanes
    mbar_init(smem_u32(q_empty), 2);  // the lanes
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_free[i]), 4);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&ta.mapK);
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(&tmem_slot_s), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  TreeWalk w;
  unsigned per;
  const bool work = tree_locate(p, w, per);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot_s;
  if (!work) {
    if (warp == 3) tmem_dealloc(tmem, 512);
    return;
  }
  if (warp == 0) {
    KeyLoader<HD, false> keys;
    for (; w.n > 0 && keys.piece(ta, w, smem, full, empty, abort_flag); w.next(p)) {
    }
    keys.drain(full, abort_flag);
  } else if (warp == 1 || warp == 3) {
    w.next(p);  // the first unit's come from the reducing warps, idle then
    for (int j = 1; w.n > 0; w.next(p), ++j) {
      bool ok = true;
      if (lane == 0)
        ok = mbar_wait(smem_u32(q_empty), (j - 1) & 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnQEmpty);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const int rows = tree_tile_rows(p, w);
      gather_rows<HD, 64>(a, w, tree_m0(p, w), rows, rows > 128 ? 256 : 128, smem, (warp >> 1) * 32 + lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(q_full));
    }
  } else if (warp == 2) {
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, false);
    const bool me = lane == 0;
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity, int site) {
      ok = __all_sync(0xffffffffu,
                      ok && mbar_wait(smem_u32(bar), parity & 1, abort_flag, p.status, kWaitLimitNs, site));
      return ok;
    };
    const uint32_t base = uniform(smem_u32(smem)), tm = uniform(tmem);
    int it = 0, cnt0 = 0, cnt1 = 0;
    for (int j = 0; uniform(w.n > 0) && ok; w.next(p), ++j) {
      const int nt = uniform(w.n);
      const bool pair = uniform(tree_tile_rows(p, w) > 128);
      if (!wait(q_full, j, kSiteAttnQFull)) break;
      for (int t = 0; t < nt && ok; ++t, ++it) {
        if (!wait(&full[it % C::RING], it / C::RING, kSiteAttnKvFull)) break;
        for (int x = pair ? 0 : t & 1; x < (pair ? 2 : (t & 1) + 1); ++x) {
          int& cnt = x ? cnt1 : cnt0;
          const int buf = x * 2 + (cnt & 1);
          if (cnt >= 2 && !wait(&s_free[buf], (cnt >> 1) - 1, kSiteAttnSFree)) break;
          tc_fence_after();
          tile_product<HD>(me, tm + buf * 128, base + (pair && x ? kAtom : 0), C::Q_ATOM,
                           base + C::OFF_RING + (it % C::RING) * C::TILE, kAtom, idS);
          warp_commit(me, smem_u32(&s_full[buf]));
          ++cnt;
        }
      }
    }
    warp_commit(me, smem_u32(drain));
    int never = 0;
    mbar_wait(smem_u32(drain), 0, &never, nullptr, 10000000ull);
    __syncwarp();
  } else {
    const int x = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int pair_bar = 2 + (warp & 3);
    const bool leader = (warp & 3) == 0 && lane == 0;
    int cnt = 0, it = 0, j = 0;
    gather_rows<HD, 256>(a, w, tree_m0(p, w), tree_tile_rows(p, w), tree_tile_rows(p, w) > 128 ? 256 : 128, smem,
                         threadIdx.x - 128);
    named_bar_sync(1, 256);
    if (leader) mbar_arrive(smem_u32(q_full));
    bool ok = true;
    for (bool first = true; w.n > 0 && ok; first = false, w.next(p), ++j) {
      if (warp == 4 && lane == 0 && w.b0 == 0) weigh_note_span(a, w, first, per);
      const int nt = w.n, rows = tree_tile_rows(p, w), ctx = w.q.ctx;
      const bool pair = rows > 128;
      const int r = pair ? x * 128 + row : row, m = tree_m0(p, w) + min(r, rows - 1);
      const int seen = ctx + m / p.g;  // the last token that the row sees
      const int t_step = pair ? 1 : 2;
      float top = -INFINITY, l = 0.f;
      if (leader && !pair && x >= nt) mbar_arrive(smem_u32(q_empty));  // no block of this unit
      for (int t = pair ? 0 : x; t < nt; t += t_step, ++cnt) {
        const int buf = x * 2 + (cnt & 1);
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s_full[buf]), (cnt >> 1) & 1, abort_flag, p.status, kWaitLimitNs,
                                               kSiteAttnSFull))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader) {  // the products are done: with the keys, and after the last one the queries
          const uint32_t eb = smem_u32(&empty[(it + t) % C::RING]);
          mbar_arrive(eb);
          if (!pair) mbar_arrive(eb);
          if (t + t_step >= nt) mbar_arrive(smem_u32(q_empty));
        }
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tmem + lane_off + buf * 128 + c * 32, s[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(s[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_free[buf]));
        const long long key0 = static_cast<long long>(w.b0 + t) * kBlock;
        if (key0 + kBlock > ctx + 1) {
          const int lim = static_cast<int>(seen - key0);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e > lim) s[c][e] = 0xff800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
        const float now = fmaxf(top, fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * p.sl2);
        const float b = now == -INFINITY ? 0.f : now;
        l *= top == now ? 1.f : ex2(top - b);
        top = now;
        const float2 scale2 = make_float2(p.sl2, p.sl2), b2 = make_float2(-b, -b);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), scale2, b2);
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], make_float2(ex2(y.x), ex2(y.y)));
          }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      it += nt;
      // where the lanes share rows, lane 1 hands its own to lane 0
      if (x == 1) xch[j & 1][row] = make_float2(top, l);
      if (!named_bar_and(pair_bar, 64, ok)) {
        ok = false;
        break;
      }
      float2 v = make_float2(top, l);
      if (!pair && x == 0) v = weigh_merge(v, xch[j & 1][row]);
      if (pair || x == 0) weigh_leave(a, w, first, r, v);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- weights --
// A unit is a (sequence, head); its rows are tiles of 256.  One tile stays in
// place while the blocks stream by; with more, a group of RING blocks stays and the
// tiles pass, back and forth, so that a tile is gathered once for a group.  A
// product's 128 keys are TMEM's lanes, its rows the columns of one of two buffers;
// the two halves of the reducing warps take alternate blocks, a buffer each, so that
// none waits for the other.  A row's weight is 2^(x - (m + log2 l)): the one number a
// row that the sum needs is rounded once more than m alone, by 2^-24 of itself, which
// is no more than the products' own rounding of the scores, and halves what a score
// reads of shared memory.  Blocks go from a run's last to its first: what the
// statistics read last is still in L2.  Tiles of 128 rows, two buffers a half and the
// next tile gathered ahead were slower (36 rows of 28 / 4 heads 73.8 us where this takes
// 63.7, 128 rows 256 where this takes 249): products half as wide read more of shared
// memory for each score.
template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1) weigh_tokens_tc_kernel(const __grid_constant__ WTcArgs ta) {
  using C = WTc<HD>;
  const WeighArgs& a = ta.a;
  const TreeArgs& p = a.t;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[2 * C::RING + 7];
  __shared__ uint32_t tmem_slot_s;
  __shared__ volatile int abort_s;
  __shared__ __align__(16) float s_off[2][kWeighTcRows];  // -(m + log2 l) of a tile's rows, by turns
  __shared__ __align__(16) int s_blind[2][8];  // whether a warp's of these rows are without a source
  __shared__ float s_sum[C::RING][kBlock];  // of a group's blocks over the tiles so far
  uint64_t* full = bars;
  uint64_t* empty = bars + C::RING;
  uint64_t* q_full = bars + 2 * C::RING;
  uint64_t* q_empty = q_full + 1;
  uint64_t* d_full = q_full + 2;  // [buffer]
  uint64_t* d_free = q_full + 4;  // [buffer], a warp an arrival
  uint64_t* drain = q_full + 6;
  volatile int* abort_flag = &abort_s;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    mbar_init(smem_u32(q_full), 2);
    mbar_init(smem_u32(q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&d_full[i]), 1);
      mbar_init(smem_u32(&d_free[i]), 4);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&ta.mapK);
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(&tmem_slot_s), 512);
    tmem_relinquish();
  }
  TreeWalk w;
  unsigned per;
  // Of what this kernel reads the first launch, which has waited for all before it, writes the
  // statistics alone: only the warps that read them wait for it.
  const bool work = tree_locate(p, w, per);
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot_s;
  if (!work) {
    pdl_wait();
    if (warp == 3) tmem_dealloc(tmem, 512);
    return;
  }
  auto all_rows = [&]() { return w.q.n * p.g; };
  auto tiles_of = [&]() { return (all_rows() + kWeighTcRows - 1) / kWeighTcRows; };
  auto rows_of = [&](int tile) { return min(kWeighTcRows, all_rows() - tile * kWeighTcRows); };

  if (warp == 0) {
    KeyLoader<HD, true> keys;
    for (; w.n > 0 && keys.piece(ta, w, smem, full, empty, abort_flag); w.next(p)) {
    }
    keys.drain(full, abort_flag);
  } else if (warp == 1 || warp == 3) {
    bool ok = true;
    int ql = 0;  // tiles gathered so far; the first by the reducing warps
    for (; w.n > 0 && ok; w.next(p)) {
      WItems q(w.n, tiles_of(), C::RING);
      bool fresh = true;
      while (q.g0 < q.n) {
        if (fresh && ql > 0) {
          if (lane == 0)
            ok = mbar_wait(smem_u32(q_empty), (ql - 1) & 1, abort_flag, p.status, kWaitLimitNs, kSiteAttnQEmpty);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          const int rows = rows_of(q.tile_at);
          gather_rows<HD, 64>(a, w, q.tile_at * kWeighTcRows, rows, (rows + 31) & ~31, smem, (warp >> 1) * 32 + lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(q_full));
        }
        if (fresh) ++ql;
        fresh = q.next();
      }
    }
  } else if (warp == 2) {
    const bool me = lane == 0;
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity, int site) {
      ok = __all_sync(0xffffffffu,
                      ok && mbar_wait(smem_u32(bar), parity & 1, abort_flag, p.status, kWaitLimitNs, site));
      return ok;
    };
    const uint32_t base = uniform(smem_u32(smem)), tm = uniform(tmem);
    int it = 0, cnt0 = 0, cnt1 = 0, ql = 0;
    for (; uniform(w.n > 0) && ok; w.next(p)) {
      WItems q(uniform(w.n), uniform(tiles_of()), C::RING);
      bool fresh = true;
      while (q.g0 < q.n && ok) {
        if (fresh) {
          if (!wait(q_full, ql, kSiteAttnQFull)) break;
          ++ql;
        }
        const int cols = uniform((rows_of(q.tile_at) + 31) & ~31);
        const uint32_t id = idesc_bf16_f32(128, cols, false);
        const int nb = q.blocks();
        for (int b = 0; b < nb; ++b) {
          const int i = it + q.g0 + b, buf = i & 1;
          int& cnt = buf ? cnt1 : cnt0;
          if (q.done == 0 && !wait(&full[i % C::RING], i / C::RING, kSiteAttnKvFull)) break;
          if (cnt > 0 && !wait(&d_free[buf], cnt - 1, kSiteAttnSFree)) break;
          tc_fence_after();
          tile_product<HD>(me, tm + buf * 256, base + C::OFF_RING + (i % C::RING) * C::TILE, kAtom, base, C::Q_ATOM, id);
          warp_commit(me, smem_u32(&d_full[buf]));
          ++cnt;
        }
        fresh = q.next();
        // another tile follows, or another unit's: the queries are done with once these products are
        if (ok && (fresh || q.g0 >= q.n)) warp_commit(me, smem_u32(q_empty));
      }
      it += q.n;
    }
    warp_commit(me, smem_u32(drain));
    int never = 0;
    mbar_wait(smem_u32(drain), 0, &never, nullptr, 10000000ull);
    __syncwarp();
  } else {
    const int x = (warp - 4) >> 2, key = (warp & 3) * 32 + lane, tid = threadIdx.x - 128;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const bool leader = (warp & 3) == 0 && lane == 0;
    const float2 scale2 = make_float2(p.sl2, p.sl2);
    int it = 0, cnt = 0, ql = 0;
    gather_rows<HD, 256>(a, w, 0, rows_of(0), (rows_of(0) + 31) & ~31, smem, tid);
    named_bar_sync(1, 256);
    if (leader) mbar_arrive(smem_u32(q_full));
    pdl_wait();
    bool ok = true;
    for (; w.n > 0; w.next(p)) {
      const int ctx = w.q.ctx, len = ctx + w.q.n;
      float* wt = a.w.ptr + w.s * a.w.seq_stride + w.head * a.w.head_stride;
      bool blind = false;
      auto tile = [&](const WItems& q, bool mine) {  // its statistics, a thread a row
        float off = -INFINITY;  // no such row, or one that weighs nothing
        const bool there = tid < rows_of(q.tile_at);
        if (there) {
          const float2 v = weigh_gather(a, weigh_unit(a, w, q.tile_at), weigh_row_ml(a, w.q.row0, w.head, q.tile_at * kWeighTcRows + tid), tid, 0, 1);
          if (v.x != INFINITY || v.y != 0.f) off = -(v.x + log2f(v.y));
        }
        s_off[ql & 1][tid] = off;
        if (a.rows) {
          const bool none = __any_sync(0xffffffffu, there && off == -INFINITY);
          if (lane == 0) s_blind[ql & 1][warp - 4] = none;
        }
        if (!named_bar_and(1, 256, mine)) return false;
        if (a.rows) {
          const int4 u = reinterpret_cast<const int4*>(s_blind[ql & 1])[0], v = reinterpret_cast<const int4*>(s_blind[ql & 1])[1];
          blind = u.x | u.y | u.z | u.w | v.x | v.y | v.z | v.w;
        }
        ++ql;
        return true;
      };
      auto block = [&](const WItems& q, int b) {
        const float* so = s_off[(ql - 1) & 1];
        const int cols = (rows_of(q.tile_at) + 31) & ~31, m0 = q.tile_at * kWeighTcRows;
        const bool last = q.last();
        const long long t0 = static_cast<long long>(w.b0 + q.n - 1 - (q.g0 + b)) * kBlock;
        const bool tail = t0 + kBlock > ctx;
        const bool mine = last && t0 + key < len;  // this thread writes a weight
        const float old = mine && t0 + key < ctx && a.decay != 0.f ? wt[t0 + key] : 0.f;
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&d_full[x]), cnt & 1, abort_flag, p.status, kWaitLimitNs,
                                               kSiteAttnSFull)))
          return false;
        ++cnt;
        tc_fence_after();
        if (leader && last) mbar_arrive(smem_u32(&empty[(it + q.g0 + b) % C::RING]));
        // the first row that sees this key; rows without a source see none
        const int from = tail ? static_cast<int>(min(max(t0 + key - ctx, 0ll) * p.g - m0, 1ll << 20)) : 0;
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto add = [&](const uint32_t(&s)[32], int c0, auto hides) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 o4 = *reinterpret_cast<const float4*>(so + c0 + e);
            float2 y = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), scale2, make_float2(o4.x, o4.y));
            float2 z = fma2(make_float2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), scale2, make_float2(o4.z, o4.w));
            constexpr int kHides = decltype(hides)::value;  // nothing, tokens behind a row's own, rows without a source too
            auto hidden = [&](int i, float off) { return c0 + e + i < from || (kHides == 2 && off == -INFINITY); };
            if constexpr (kHides > 0) {
              if (hidden(0, o4.x)) y.x = -INFINITY;
              if (hidden(1, o4.y)) y.y = -INFINITY;
              if (hidden(2, o4.z)) z.x = -INFINITY;
              if (hidden(3, o4.w)) z.y = -INFINITY;
            }
            acc[0] = add2(acc[0], make_float2(ex2(y.x), ex2(y.y)));
            acc[1] = add2(acc[1], make_float2(ex2(z.x), ex2(z.y)));
          }
        };
        // 32 columns at a time, the next ones on their way
        const uint32_t at = tmem + lane_off + x * 256;
        uint32_t s0[32], s1[32];
        auto loaded = [&](uint32_t(&s)[32], uint32_t(&then)[32], int c) {
          tmem_ld_wait(s);
          if (c + 32 < cols) {
            tmem_ld32(at + c + 32, then);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&d_free[x]));
          }
        };
        auto columns = [&](auto hides) {
          tmem_ld32(at, s0);
#pragma unroll 1
          for (int c = 0; c < cols; c += 64) {
            loaded(s0, s1, c);
            add(s0, c, hides);
            if (c + 32 < cols) {
              loaded(s1, s0, c + 32);
              add(s1, c + 32, hides);
            }
          }
        };
        if (blind)
          columns(std::integral_constant<int, 2>{});
        else if (tail)
          columns(std::integral_constant<int, 1>{});
        else
          columns(std::integral_constant<int, 0>{});
        float sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
        if (q.tiles > 1) {
          if (q.done > 0) sum += s_sum[b][key];
          s_sum[b][key] = sum;
        }
        if (mine) wt[t0 + key] = fmaf(a.decay, old, sum);
        return true;
      };
      if (!half_pass(WItems(w.n, tiles_of(), C::RING), it, x, ok, tile, block)) break;
      it += w.n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD>
int tc_go(WeighArgs& a, int grid, cudaStream_t st) {
  using C = WTc<HD>;
  WTcArgs ta;
  const specfold_paged_cache& c = a.t.cache;
  ta.box = c.page_size % 64 == 0 ? 64 : c.page_size % 32 == 0 ? 32 : c.page_size % 16 == 0 ? 16 : 8;
  const uint64_t tokens = static_cast<uint64_t>(c.num_pages) * c.page_size;
  if (const int rc = make_map_3d(&ta.mapK, c.k, HD, a.t.n_kv, tokens, c.k_head_stride, c.k_token_stride, ta.box, HD * 2))
    return rc;
  a.t.kb = kBlock;
  a.t.tile_rows = kWeighTcRows;
  a.t.unit_cost = 5;
  a.t.w_full = 5;
  a.t.w_half = 3;
  ta.a = a;
  if (const int rc = smem_limit_once(weigh_stats_tc_kernel<HD>, C::SMEM)) return rc;
  launch_k(weigh_stats_tc_kernel<HD>, dim3(grid), dim3(kTcThreads), C::SMEM, st, ta);
  count_launch();
  if (const int rc = check_launch()) return rc;
  ta.a.t.tile_rows = SPECFOLD_MAX_TREE * 128;  // all of a head group's rows
  ta.a.t.w_full = ta.a.t.w_half = 1;
  if (const int rc = smem_limit_once(weigh_tokens_tc_kernel<HD>, C::SMEM)) return rc;
  launch_k(weigh_tokens_tc_kernel<HD>, dim3(grid), dim3(kTcThreads), C::SMEM, st, ta);
  count_launch();
  return check_launch();
}

}  // namespace

int launch_weigh_tc(WeighArgs& a, int hd, int grid, cudaStream_t st) {
  return hd == 128 ? tc_go<128>(a, grid, st) : tc_go<64>(a, grid, st);
}

}  // namespace sf
