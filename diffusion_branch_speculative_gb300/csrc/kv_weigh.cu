// The attention weight that cached tokens get from a batch of rows, added up per
// key/value head (specfold_kv_weigh): what an eviction goes by.  Keys alone are
// read.  kv_weigh.cuh has the two launches' division of work; here are the forms
// that keep the scores: few rows a head group, and fp32.  kv_weigh_tc.cu has many
// rows in bf16.
#include "kv_weigh.cuh"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace sf {
namespace {

constexpr int kThreads = 128;  // 4 warps, each with its own chunks of keys
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 64;        // keys of a block of the line
constexpr int kSmBudget = 160;   // SMs the workspace is sized for (>= one GB300)

// The warps' (m, l) of R rows, warp k's at s_ml[k * R], to their place.
template <int R>
SF_DEV void weigh_write_part(const WeighArgs& p, const TreeWalk& w, bool first, const float2* s_ml) {
  const int r = threadIdx.x;
  if (r >= R) return;
  float2 a = s_ml[r];
#pragma unroll
  for (int k = 1; k < kWarps; ++k) a = weigh_merge(a, s_ml[k * R + r]);
  weigh_leave(p, w, first, r, a);
}

// ------------------------------------------------------ few rows, bf16 --
// Up to 8 NT rows of a head group, so at most 8 NT operations a byte of the
// keys: the memory bounds it.  Each warp streams its own 4 KB chunks of keys
// through a private ring of asynchronous copies.  Keys are the 16 rows of the
// warps' matrix instructions and the queries their 8 columns, so that one token
// with a group of seven heads wastes one column in eight.  In two launches the
// scores go to the workspace, 32 bytes a token and eight rows, where the second
// finds them in L2 rather than the keys in DRAM: 8 sequences of 20000 tokens (28 / 4
// heads of 128, 122 MB of keys) take 33 us, 26 of them the first launch, DRAM 59 %
// busy, its start and uneven shares of the SMs the rest; one of 40000, 17.6.
template <int HD, int NT, int WARPS_ = kWarps>
struct WFew {
  static constexpr int WARPS = WARPS_;
  static constexpr int R = 8 * NT;
  static constexpr int CH = 2048 / HD;  // keys of a warp's step: 4 KB
  static constexpr int STAGES = 3;
  static constexpr int ROW = HD * 2;
  static constexpr int CPR = ROW / 16;
  static constexpr int STAGE = CH * ROW;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int OFF_Q = WARPS * RING;
  static constexpr int SMEM = OFF_Q + R * ROW;
};
constexpr int kFewCtas = 4;  // per SM, of two launches

// A block's keys key_lo .. key_hi - 1 of sequence s, head h: the warps' statistics to s_ml
// [WARPS][R], the scores to keep(i, kh, x): this warp's step i, 16 of its keys, x[nt][2 e + f]
// the score of the key lane / 4 + 8 e and the row 8 nt + 2 (lane % 4) + f.  STEPS: a warp's at
// most, all of them unrolled; 0: any number.
template <int HD, int NT, int WARPS, int STEPS, typename Keep>
SF_DEV void few_stream(const WeighArgs& a, int s, int h, const TreeSeq& q, int key_lo, int key_hi, uint8_t* smem, float2* s_ml,
                       Keep keep) {
  using C = WFew<HD, NT, WARPS>;
  using T = __nv_bfloat16;
  constexpr int R = C::R, KS = HD / 16, CH = C::CH, KH = CH / 16;
  const TreeArgs& p = a.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t once = policy_evict_first();  // the keys: L2 is for the scores
  uint8_t* ring = smem + warp * C::RING;
  uint8_t* s_q = smem + C::OFF_Q;
  const int rows = q.n * p.g;
  // this warp's chunks: key_lo + CH * (warp + 4 i)
  const int chunks = (key_hi - key_lo + CH - 1) / CH;
  const int mine = chunks > warp ? (chunks - warp + WARPS - 1) / WARPS : 0;
  auto key_of = [&](int i) { return key_lo + CH * (warp + WARPS * i); };
  // lanes 0..CH-1 have a chunk's keys; a chunk's pages are read two chunks ahead of its
  // loads, and followed by steps (no division a chunk)
  const int32_t* table = p.cache.block_table + s * p.cache.table_stride;
  const int ps = p.cache.page_size, dpg = CH * WARPS / ps, doff = CH * WARPS - dpg * ps;
  struct Page {
    int id, off;  // in the table; a key's place in it, -1: no key
  };
  const unsigned tok0 = static_cast<unsigned>(key_lo) + CH * warp + (lane & (CH - 1));
  int pg = tok0 / static_cast<unsigned>(ps), off = tok0 - pg * ps;
  int left = key_hi > static_cast<int>(tok0) ? (key_hi - static_cast<int>(tok0) + CH * WARPS - 1) / (CH * WARPS) : 0;  // this lane's keys
  auto page_next = [&]() {
    Page x = {-1, left > 0 ? off : -1};
    if (left > 0 && pg < p.cache.table_pages) x.id = table[pg];
    --left;
    pg += dpg;
    off += doff;
    if (off >= ps) {
      off -= ps;
      ++pg;
    }
    return x;
  };
  auto slot_of = [&](Page x) {
    if (x.id >= 0 && x.id < p.cache.num_pages) return x.id * ps + x.off;
    if (x.off >= 0) atomicOr(p.status, SPECFOLD_DEV_BAD_PAGE);
    return -1;
  };
  const T* kbase = static_cast<const T*>(p.cache.k) + h * p.cache.k_head_stride;
  auto load = [&](int i, int slot) {
    if (i < mine) {
      const uint32_t st = smem_u32(ring + (i % C::STAGES) * C::STAGE);
      constexpr int KEYS = 32 / C::CPR;  // keys of one step of the warp's lanes
      const int c = lane % C::CPR;
#pragma unroll
      for (int it = 0; it < CH / KEYS; ++it) {
        const int key = it * KEYS + lane / C::CPR;
        const int tk = __shfl_sync(0xffffffffu, slot, key);
        const long long tz = tk < 0 ? 0 : tk;  // any valid address when nothing is read
        cp_async16_hint(st + key * C::ROW + ((c ^ (key & 7)) << 4), kbase + tz * p.cache.k_token_stride + c * 8,
                        tk < 0 ? 0u : 16u, once);
      }
    }
    cp_async_commit();
  };
  Page page = page_next(), next = page_next();
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) {
    load(i, slot_of(page));
    page = next;
    next = page_next();
  }
  // queries: row m = row m / g of the sequence, head m % g of the group; the rows
  // past the last are its copies (zeros times an infinite key would be NaN)
  for (int i = threadIdx.x; i < R * C::CPR; i += 32 * WARPS) {
    const int r = i / C::CPR, c = i % C::CPR, m = min(r, rows - 1);
    const int src = max(weigh_src(a, q.row0 + m / p.g), 0);
    *reinterpret_cast<uint4*>(s_q + r * C::ROW + ((c ^ (r & 7)) << 4)) =
        *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + src * p.q_rs + (h * p.g + m % p.g) * p.q_hs + c * 8);
  }
  __syncthreads();
  // two of their fragments, dimensions 16 ks .. 16 ks + 31
  auto queries = [&](int nt, int ks, uint32_t (&b)[4]) {
    const int r = nt * 8 + (lane & 7);
    ldsm4(smem_u32(s_q + r * C::ROW + (((ks * 2 + (lane >> 3)) ^ (r & 7)) << 4)), b);
  };
  constexpr bool HELD = STEPS == 0 || NT == 1;  // beside the scores there is no room for two tiles'
  uint32_t qf[HELD ? NT : 1][KS / 2][4];
  if constexpr (HELD)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) queries(nt, ks, qf[nt][ks / 2]);
  // this thread's rows: 8 nt + 2 (lane % 4) and the next one; the last token each sees (-1: none)
  int seen[NT][2];
  float m[NT][2], l[NT][2];
  bool blind = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      seen[nt][e] = q.ctx + min(nt * 8 + (lane & 3) * 2 + e, rows - 1) / p.g;
      m[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
    }
  if (a.rows) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (!weigh_has_src(a, q.row0 + seen[nt][e] - q.ctx)) {
          seen[nt][e] = -1;
          blind = true;
        }
    blind = __any_sync(0xffffffffu, blind);
  }
  const int all_see = blind ? 0 : q.ctx;  // tokens before this one
  auto step = [&](int i) {
    load(i + C::STAGES - 1, slot_of(page));
    page = next;
    next = page_next();
    cp_async_wait<C::STAGES - 1>();
    __syncwarp();
    const uint8_t* stg = ring + (i % C::STAGES) * C::STAGE;
    const bool tail = key_of(i) + CH > all_see;  // holds tokens that not every row sees
#pragma unroll
    for (int kh = 0; kh < KH; ++kh) {
      float sc[NT][4] = {};
      const int key = kh * 16 + (lane & 15);
      const uint32_t base = smem_u32(stg + key * C::ROW);
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) {
        uint32_t k[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) ldsm4(base + ((((ks + x) * 2 + (lane >> 4)) ^ (key & 7)) << 4), k[x]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t b[4];
          if constexpr (!HELD) queries(nt, ks, b);
          const uint32_t(&f)[4] = HELD ? qf[HELD ? nt : 0][ks / 2] : b;
          mma16816(sc[nt], k[0], f[0], f[1]);
          mma16816(sc[nt], k[1], f[2], f[3]);
        }
      }
      const int t0 = key_of(i) + kh * 16 + (lane >> 2);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          sc[nt][x] *= p.sl2;
          if (tail && t0 + (x >> 1) * 8 > seen[nt][x & 1]) sc[nt][x] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float top = fmaxf(m[nt][e], fmaxf(sc[nt][e], sc[nt][2 + e]));
          const float b = top == -INFINITY ? 0.f : top;
          l[nt][e] = fmaf(l[nt][e], m[nt][e] == top ? 1.f : ex2(m[nt][e] - b), ex2(sc[nt][e] - b) + ex2(sc[nt][2 + e] - b));
          m[nt][e] = top;
        }
      }
      keep(i, kh, sc);
    }
    __syncwarp();  // the stage may be overwritten
  };
  if constexpr (STEPS > 0) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if (i >= mine) break;
      step(i);
    }
  } else {
    for (int i = 0; i < mine; ++i) step(i);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 v = make_float2(m[nt][e], l[nt][e]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        v = weigh_merge(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
      if (lane < 4) s_ml[warp * R + nt * 8 + lane * 2 + e] = v;
    }
}

template <int HD, int NT>
__global__ void __launch_bounds__(kThreads, kFewCtas) weigh_few_kernel(const __grid_constant__ WeighArgs a) {
  using C = WFew<HD, NT>;
  constexpr int R = C::R;
  const TreeArgs& p = a.t;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[kWarps * R];
  pdl_wait();
  pdl_trigger();
  TreeWalk w;
  unsigned per;
  if (!tree_locate(p, w, per)) return;
  for (bool first = true; w.n > 0; first = false, w.next(p)) {
    const int key_lo = w.b0 * p.kb;
    const int key_hi = min(static_cast<long long>(w.q.ctx + w.q.n), static_cast<long long>(w.b0 + w.n) * p.kb);
    if (threadIdx.x == 0 && w.b0 == 0) weigh_note_span(a, w, first, per);
    __syncthreads();  // the previous piece's shared memory is free
    float* out = a.scores + (static_cast<size_t>(w.s) * p.n_kv + w.head) * a.w.tokens * R;
    const int at = key_lo + C::CH * static_cast<int>(threadIdx.x >> 5) + ((threadIdx.x & 31) >> 2), len = w.q.ctx + w.q.n;
    few_stream<HD, NT, kWarps, 0>(a, w.s, w.head, w.q, key_lo, key_hi, smem, s_ml, [&](int i, int kh, const float(&x)[NT][4]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = at + C::CH * kWarps * i + 16 * kh + 8 * e;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (t < len)
            *reinterpret_cast<float2*>(out + static_cast<size_t>(t) * R + nt * 8 + (threadIdx.x & 3) * 2) = make_float2(x[nt][2 * e], x[nt][2 * e + 1]);
      }
    });
    __syncthreads();
    weigh_write_part<R>(a, w, first, s_ml);
  }
}

// The same in one launch where a unit's scores fit the registers of a cluster: its
// blocks have a slice of the tokens each and keep its scores, 64 a thread, tell each
// other their rows' statistics, and add up their tokens' weights.  No scores pass
// through memory, and one launch less is waited for and paid for on the host.  128
// registers a thread and 12 KB of keys on the way a warp let an SM have 16 warps; the
// unrolled steps are what lets registers hold the scores (in shared memory, beside
// two stages and three blocks an SM, 80 us where this takes 70; of the eight instances
// three, with two tiles of rows, spill 4 to 12 bytes).  64 sequences of up
// to 8000 tokens, one row of 28 / 4 heads of 128: 384 MB in 70 us, 5480 GB/s, 0.81 of
// the copy rate; 32 of 8 heads and eight rows 0.89; head size 64 0.67.  What is left is
// the blocks' own starts and exchanges.
constexpr int kUnitCluster = 8;        // blocks at most
constexpr int kUnitStep = 256;         // tokens that are worth a block more where SMs are idle,
constexpr int kUnitLeast = 2;          // and where they are not: the share of what its warps can hold
constexpr int kUnitScores = 2 * 1024;  // of a warp, at most: 64 a thread

// What a cluster's blocks share of a unit: every block's statistics of its rows.
template <int R>
struct UnitShared {
  float2 all[kUnitCluster][R];
  float m[R], rl[R];
  int spoilt;  // the last token that a row whose weights are no numbers sees
};
// This block's slice of the unit's tokens.
struct Slice {
  int lo, hi;
  SF_DEV Slice(int len, int blocks, int rank) {
    const int n = ((len - 1) / blocks / kKeys + 1) * kKeys;
    lo = min(static_cast<long long>(len), static_cast<long long>(rank) * n);
    hi = lo + min(len - lo, n);
  }
};

template <int HD, int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) weigh_unit_kernel(const __grid_constant__ WeighArgs a) {
  using C = WFew<HD, NT, WARPS>;
  constexpr int R = C::R, KH = C::CH / 16, STEPS = kUnitScores / R / C::CH;
  const TreeArgs& p = a.t;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[WARPS * R];
  __shared__ UnitShared<R> u;
  pdl_wait();
  pdl_trigger();
  const int rank = static_cast<int>(cluster_ctarank()), unit = static_cast<int>(blockIdx.x) / a.blocks;
  const int s = unit / p.n_kv, h = unit - s * p.n_kv, lane = threadIdx.x & 31;
  const TreeSeq q = tree_seq(p, s);
  if (q.bad && h == 0 && rank == 0 && threadIdx.x == 0) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
  if (q.n == 0) return;  // the same in all of the cluster
  // no more blocks than this unit's length is worth
  const int len = q.ctx + q.n, spread = min(a.spread, (len - 1) / kUnitStep + 1);
  const int blocks = min(a.blocks, max((len - 1) / (kUnitScores / R * WARPS / kUnitLeast) + 1, spread));
  if (rank >= blocks) return;  // (a cluster's barriers do not count those that have left)
  cluster_arrive();
  const Slice t(len, blocks, rank);
  float x[STEPS][KH][NT][4];
  few_stream<HD, NT, WARPS, STEPS>(a, s, h, q, t.lo, t.hi, smem, s_ml, [&](int i, int kh, const float(&sc)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][kh][nt][e] = sc[nt][e];
  });
  // Lane 4 k of four has the token k of 16, lane 4 k + 1 the token k + 8.
  const int first = t.lo + C::CH * static_cast<int>(threadIdx.x >> 5) + (lane >> 2) + 8 * (lane & 1);
  auto token = [&](int i, int kh) { return first + C::CH * WARPS * i + 16 * kh; };
  float* wt = a.w.ptr + s * a.w.seq_stride + h * a.w.head_stride;
  const bool writes = (lane & 3) < 2;
  const int olds = writes && a.decay != 0.f ? min(t.hi, q.ctx) : 0;
  float old[STEPS][KH];
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
#pragma unroll
    for (int kh = 0; kh < KH; ++kh) old[i][kh] = token(i, kh) < olds ? wt[token(i, kh)] : 0.f;
  if (threadIdx.x == 0) u.spoilt = -1;
  __syncthreads();
  cluster_wait();  // all of them have begun
  if (threadIdx.x < R) {
    const int r = threadIdx.x;
    float2 v = s_ml[r];
#pragma unroll
    for (int k = 1; k < WARPS; ++k) v = weigh_merge(v, s_ml[k * R + r]);
    if (r >= q.n * p.g || weigh_src(a, q.row0 + r / p.g) < 0) v = make_float2(INFINITY, 0.f);  // weighs nothing
    for (int k = 0; k < blocks; ++k) {
      const uint32_t at = dsmem_addr(smem_u32(&u.all[rank][r]), k);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
    }
  }
  cluster_sync_all();  // the only exchange: a block may end from here on
  if (threadIdx.x < R) {
    const int r = threadIdx.x;
    float2 v = u.all[0][r];
    for (int k = 1; k < blocks; ++k) v = weigh_merge(v, u.all[k][r]);
    // Such a row adds NaN to the tokens that it sees, and to no other (2^-inf times its NaN would be
    // one): its sum stays out, and the tokens up to its last one are written so.
    if (weigh_no_number(v)) {
      atomicMax(&u.spoilt, q.ctx + r / p.g);
      v = make_float2(INFINITY, 0.f);
    }
    u.m[r] = v.x;
    u.rl[r] = merge_scale(v.y);
  }
  __syncthreads();
  const int spoilt = u.spoilt;
  float m[NT][2], rl[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      m[nt][f] = u.m[nt * 8 + (lane & 3) * 2 + f];
      rl[nt][f] = u.rl[nt * 8 + (lane & 3) * 2 + f];
    }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    if (t.lo + C::CH * (static_cast<int>(threadIdx.x >> 5) + WARPS * i) >= t.hi) break;
#pragma unroll
    for (int kh = 0; kh < KH; ++kh) {
      float sum[2] = {};  // of the tokens lane / 4 and 8 behind it
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e >> 1] = fmaf(ex2(x[i][kh][nt][e] - m[nt][e & 1]), rl[nt][e & 1], sum[e >> 1]);
      // lanes with an even place end with the first token's, the others with the second's
      const bool odd = lane & 1;
      float mine = (odd ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, odd ? sum[0] : sum[1], 1);
      mine += __shfl_xor_sync(0xffffffffu, mine, 2);
      if (token(i, kh) <= spoilt) mine = NAN;
      if (writes && token(i, kh) < t.hi) wt[token(i, kh)] = fmaf(a.decay, old[i][kh], mine);
    }
  }
}

// ------------------------------------------------------------ fp32: few --
// The same for fp32 by multiply-adds, a tile of eight rows at a time (a piece of at
// most four does no other rows' arithmetic): a warp's step is 4 KB of keys, a lane
// (key, 32 of the dimensions), the queries broadcast from shared memory; a key's lanes
// add up by halves, so that each ends with some rows' scores.  Two steps at a time, whose
// keys share a query's read (alone, 16 sequences of 12239 tokens and twelve rows of 2 heads
// took 57.3 us where this takes 51.3, 8 of 4000 and 48 rows of 8 heads 120 and 105; short
// pieces wait 0.7 us longer for their first).  8 sequences of 8000 tokens, one row of 24 / 8
// heads of 128, 190 MB, take 48 us in all, 0.59 of the copy rate: 39 the first launch (cold;
// DRAM 66 % busy, shared memory's pipe 31 %, multiply-adds 19 %: warps wait for their
// keys, 12 of them an SM), then the second with the 12 MB of scores that eight rows' room
// for three comes to, 14 cold.  48 rows go over the keys six times, from L2: 105 us, where
// their bytes need 14.  7 of 1111 tokens and five rows of 4 / 2 heads of 64 take
// 12.2 us, 9.3 and 9.9 the two launches alone and cold: latency.  One launch by clusters,
// scores in shared memory, was slower (70.6 us where two took 47.4, and 15.6 where they
// took 13.8).
template <int HD>
struct WSimt {
  static constexpr int R = 8;
  static constexpr int CH = 1024 / HD;
  static constexpr int STAGES = 4;
  static constexpr int ROW = HD * 4;
  static constexpr int CPR = ROW / 16;
  static constexpr int STAGE = CH * ROW;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int OFF_Q = kWarps * RING;
  static constexpr int SMEM = OFF_Q + R * ROW;
  static constexpr int CTAS = 3;
};

// Rows m0 .. m0 + rows - 1 (at most R) of a block's keys key_lo .. key_hi - 1 of sequence s,
// head h: the scores to row_of(token) + m0, the warps' statistics to s_ml [kWarps][R].
template <typename C, int HD, typename RowOf>
SF_DEV void simt_stream(const WeighArgs& a, int s, int h, const TreeSeq& q, int m0, int rows, int key_lo, int key_hi,
                        uint8_t* smem, float2* s_ml, RowOf row_of) {
  constexpr int R = C::R, CH = C::CH, PARTS = HD / 32;
  const TreeArgs& p = a.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, len = q.ctx + q.n;
  uint8_t* ring = smem + warp * C::RING;
  float* s_q = reinterpret_cast<float*>(smem + C::OFF_Q);
  const int chunks = (key_hi - key_lo + CH - 1) / CH;
  const int mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
  auto key_of = [&](int i) { return key_lo + CH * (warp + kWarps * i); };
  auto slot_of = [&](int i) {
    const int tok = key_of(i) + (lane & (CH - 1));
    return i < mine && tok < key_hi ? tree_pool_token(p, s, tok) : -1;
  };
  const float* kbase = static_cast<const float*>(p.cache.k) + h * p.cache.k_head_stride;
  auto load = [&](int i, int slot) {
    if (i < mine) {
      uint8_t* st = ring + (i % C::STAGES) * C::STAGE;
#pragma unroll
      for (int it = 0; it < CH * C::CPR / 32; ++it) {
        const int idx = it * 32 + lane, c = idx % C::CPR, key = idx / C::CPR;
        const int tk = __shfl_sync(0xffffffffu, slot, key);
        const long long tz = tk < 0 ? 0 : tk;
        cp_async16(smem_u32(st + key * C::ROW + ((c ^ (key & 7)) << 4)), kbase + tz * p.cache.k_token_stride + c * 4,
                   tk < 0 ? 0u : 16u);
      }
    }
    cp_async_commit();
  };
  int slot[2] = {slot_of(0), slot_of(1)};  // of the next two steps to load
  auto load_two = [&](int i) {
    load(i, slot[0]);
    load(i + 1, slot[1]);
    slot[0] = slot_of(i + 2);
    slot[1] = slot_of(i + 3);
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 2; i += 2) load_two(i);
  for (int i = threadIdx.x; i < R * (HD / 4); i += kThreads) {
    const int r = i / (HD / 4), d = (i % (HD / 4)) * 4, m = m0 + min(r, rows - 1);
    const int src = max(weigh_src(a, q.row0 + m / p.g), 0);
    *reinterpret_cast<float4*>(s_q + r * HD + d) = *reinterpret_cast<const float4*>(
        static_cast<const float*>(p.q) + src * p.q_rs + (h * p.g + m % p.g) * p.q_hs + d);
  }
  __syncthreads();
  const int key = lane & (CH - 1), part = lane / CH;
  auto stream = [&](auto nr) {
    constexpr int NR = decltype(nr)::value;  // rows worked on
    constexpr int RP = NR / PARTS;           // of which a lane has RP's sums, from row part * RP on
    int seen[RP];
    float m[RP], l[RP];
    bool blind = false;
#pragma unroll
    for (int r = 0; r < RP; ++r) {
      seen[r] = q.ctx + (m0 + min(part * RP + r, rows - 1)) / p.g;
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
    if (a.rows) {
#pragma unroll
      for (int r = 0; r < RP; ++r)
        if (!weigh_has_src(a, q.row0 + seen[r] - q.ctx)) {
          seen[r] = -1;
          blind = true;
        }
      blind = __any_sync(0xffffffffu, blind);
    }
    const int all_see = blind ? 0 : q.ctx;  // tokens before this one
    for (int i = 0; i < mine; i += 2) {
      load_two(i + C::STAGES - 2);
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();
      const uint8_t* sk[2];
      float x[2][NR] = {};
#pragma unroll
      for (int u = 0; u < 2; ++u) sk[u] = ring + ((i + u) % C::STAGES) * C::STAGE + key * C::ROW;
#pragma unroll
      for (int d0 = 0; d0 < 32; d0 += 4) {
        // the parts start apart, so that their reads of a query share no bank
        const int d = part * 32 + ((d0 + part * CH) & 31);
        float4 k4[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) k4[u] = *reinterpret_cast<const float4*>(sk[u] + (((d >> 2) ^ (key & 7)) << 4));
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float4 q4 = *reinterpret_cast<const float4*>(s_q + r * HD + d);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            x[u][r] = fmaf(q4.x, k4[u].x, fmaf(q4.y, k4[u].y, fmaf(q4.z, k4[u].z, fmaf(q4.w, k4[u].w, x[u][r]))));
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (i + u >= mine) break;  // (an odd number of steps: nothing was loaded)
        // the parts' sums: each step halves the rows that a lane keeps
#pragma unroll
        for (int n = NR / 2, o = 16; o >= CH; n /= 2, o /= 2) {
          const bool upper = lane & o;
#pragma unroll
          for (int r = 0; r < n; ++r) {
            const float keep = upper ? x[u][n + r] : x[u][r], give = upper ? x[u][r] : x[u][n + r];
            x[u][r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        const int tok = key_of(i + u) + key;
        const bool tail = key_of(i + u) + CH > all_see;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          x[u][r] = tail && tok > seen[r] ? -INFINITY : x[u][r] * p.sl2;
          const float top = fmaxf(m[r], x[u][r]);
          const float b = top == -INFINITY ? 0.f : top;
          l[r] = fmaf(l[r], m[r] == top ? 1.f : ex2(m[r] - b), ex2(x[u][r] - b));
          m[r] = top;
        }
        if (!tail || tok < len) {
          float* to = row_of(tok) + m0 + part * RP;
          if constexpr (RP == 4)
            *reinterpret_cast<float4*>(to) = make_float4(x[u][0], x[u][1], x[u][2], x[u][3]);
          else if constexpr (RP == 2)
            *reinterpret_cast<float2*>(to) = make_float2(x[u][0], x[u][1]);
          else
            *to = x[u][0];
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int r = 0; r < RP; ++r) {
      float2 v = make_float2(m[r], l[r]);
#pragma unroll
      for (int o = 1; o < CH; o <<= 1)
        v = weigh_merge(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
      if (key == 0) s_ml[warp * R + part * RP + r] = v;
    }
  };
  if (rows <= R / 2)
    stream(std::integral_constant<int, R / 2>{});
  else
    stream(std::integral_constant<int, R>{});
}

template <int HD>
__global__ void __launch_bounds__(kThreads, WSimt<HD>::CTAS) weigh_simt_kernel(const __grid_constant__ WeighArgs a) {
  using C = WSimt<HD>;
  constexpr int R = C::R;
  const TreeArgs& p = a.t;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[kWarps * R];
  pdl_wait();
  pdl_trigger();
  TreeWalk w;
  unsigned per;
  if (!tree_locate(p, w, per)) return;
  for (bool first = true; w.n > 0; first = false, w.next(p)) {
    const int key_lo = w.b0 * p.kb;
    const int key_hi = min(static_cast<long long>(w.q.ctx + w.q.n), static_cast<long long>(w.b0 + w.n) * p.kb);
    if (threadIdx.x == 0 && w.b0 == 0) weigh_note_span(a, w, first, per);
    __syncthreads();  // the previous piece's shared memory is free
    float* out = a.scores + (static_cast<size_t>(w.s) * p.n_kv + w.head) * a.w.tokens * a.score_rows;
    simt_stream<C, HD>(a, w.s, w.head, w.q, tree_m0(p, w), tree_tile_rows(p, w), key_lo, key_hi, smem, s_ml,
                       [&](int t) { return out + static_cast<size_t>(t) * a.score_rows; });
    __syncthreads();
    weigh_write_part<R>(a, w, first, s_ml);
  }
}

// ------------------------------------------------- weights from the scores --
// Two threads a token, kSumTokens of them at once: the scores' 2^(x - m) / l, eight rows
// at a time, four a thread: a warp's read is 32 bytes a token.  The run is found
// before the wait for the first launch: that one waited for all before it, and reads
// the same lengths.  A piece's first scores are on their way while its rows' statistics
// are merged.  More rows than kSumRows come in groups, which add to the weights in turn.
// The scores of 8 sequences of 20000 tokens, 17 MB, take it 14.7 us alone and cold, 8 behind
// the first launch; four blocks an SM have too few registers (99.9 us where three, 80
// registers without a spill, took 87).
constexpr int kSumThreads = 256, kSumTokens = 8;
constexpr int kSumCtas = 3;    // per SM
constexpr int kSumRows = 512;  // of a group

__global__ void __launch_bounds__(kSumThreads, kSumCtas) weigh_sum_kernel(const __grid_constant__ WeighArgs a) {
  const TreeArgs& p = a.t;
  __shared__ float2 s_part[kSumThreads];
  __shared__ __align__(16) float s_m[kSumRows], s_rl[kSumRows];
  TreeWalk w;
  unsigned per;
  const bool work = tree_locate(p, w, per);
  pdl_wait();
  pdl_trigger();
  if (!work) return;
  const int SR = a.stat_rows, R = a.score_rows, half = threadIdx.x & 1;
  for (; w.n > 0; w.next(p)) {
    const int rows = w.q.n * p.g, len = w.q.ctx + w.q.n, key_lo = w.b0 * p.kb;
    const int key_hi = min(static_cast<long long>(len), static_cast<long long>(w.b0 + w.n) * p.kb);
    const size_t unit = static_cast<size_t>(w.s) * p.n_kv + w.head;
    const float* x = a.scores + unit * a.w.tokens * R + 4 * half;
    float* wt = a.w.ptr + w.s * a.w.seq_stride + w.head * a.w.head_stride;
    auto token = [&](int t0, int k) { return t0 + static_cast<int>(threadIdx.x >> 1) + k * (kSumThreads / 2); };
    auto load = [&](int t0, int r, float4 (&u)[kSumTokens]) {  // (a tile of at most four rows has four scores: the others are leftovers)
#pragma unroll
      for (int k = 0; k < kSumTokens; ++k)
        u[k] = token(t0, k) < key_hi && r + 4 * half < rows
                   ? *reinterpret_cast<const float4*>(x + static_cast<size_t>(token(t0, k)) * R + r)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    for (int lo = 0; lo < rows; lo += kSumRows) {  // rows lo .. hi - 1
      const int hi = min(lo + kSumRows, rows), r8 = (hi - lo + 7) & ~7;
      float4 u[kSumTokens];
      load(key_lo, lo, u);
      // their m and 1 / l: thread (lane of partials, row)
      const int zs = max(kSumThreads / r8, 1);
      __syncthreads();  // the group before has read them
      for (int r0 = 0; r0 < r8; r0 += kSumThreads) {
        const int i = r0 + (zs > 1 ? threadIdx.x % r8 : threadIdx.x), z0 = zs > 1 ? threadIdx.x / r8 : 0, r = lo + i;
        float2 ml = make_float2(INFINITY, 0.f);  // a row past the last weighs nothing
        if (r < hi && z0 < zs)
          ml = weigh_gather(a, unit * a.stat_tiles + r / SR, weigh_row_ml(a, w.q.row0, w.head, r), r % SR, z0, zs);
        if (zs > 1) {
          s_part[threadIdx.x] = ml;
          __syncthreads();
          if (z0 == 0 && r < hi)
            for (int z = 1; z < zs; ++z) ml = weigh_merge(ml, s_part[z * r8 + i]);
        }
        if (i < r8 && z0 == 0) {
          s_m[i] = ml.x;
          s_rl[i] = merge_scale(ml.y);
        }
      }
      __syncthreads();
      // old weights count times decay, those of the groups before once, the batch's own tokens' not at all
      const int olds = lo > 0 ? key_hi : a.decay != 0.f ? min(key_hi, w.q.ctx) : 0;
      const float factor = lo > 0 ? 1.f : a.decay;
      for (int t0 = key_lo; t0 < key_hi; t0 += kSumThreads / 2 * kSumTokens) {
        float sum[kSumTokens] = {}, old[kSumTokens];
        if (t0 > key_lo) load(t0, lo, u);
#pragma unroll
        for (int k = 0; k < kSumTokens; ++k)  // every second token's weight is this thread's
          old[k] = (k & 1) == half && token(t0, k) < olds ? wt[token(t0, k)] : 0.f;
        for (int i = 0;; load(t0, lo + i, u)) {
          const float4 m = *reinterpret_cast<const float4*>(s_m + i + 4 * half);
          const float4 rl = *reinterpret_cast<const float4*>(s_rl + i + 4 * half);
#pragma unroll
          for (int k = 0; k < kSumTokens; ++k) {
            sum[k] = fmaf(ex2(u[k].x - m.x), rl.x, sum[k]);
            sum[k] = fmaf(ex2(u[k].y - m.y), rl.y, sum[k]);
            sum[k] = fmaf(ex2(u[k].z - m.z), rl.z, sum[k]);
            sum[k] = fmaf(ex2(u[k].w - m.w), rl.w, sum[k]);
          }
          if ((i += 8) >= hi - lo) break;
        }
#pragma unroll
        for (int k = 0; k < kSumTokens; ++k) {
          float both = sum[k] + __shfl_xor_sync(0xffffffffu, sum[k], 1);
          if ((k & 1) == half && token(t0, k) < key_hi) {
            // a row whose weights are no numbers adds none to the tokens that it does not see, where the
            // sum has 2^-inf times its NaN: the rows that see one of the batch's own
            if (both != both && token(t0, k) > w.q.ctx) {
              both = 0.f;
#pragma unroll 1
              for (int i = max(lo, (token(t0, k) - w.q.ctx) * p.g); i < hi; ++i)
                both = fmaf(ex2(x[static_cast<size_t>(token(t0, k)) * R - 4 * half + i] - s_m[i - lo]), s_rl[i - lo], both);
            }
            wt[token(t0, k)] = fmaf(factor, old[k], both);
          }
        }
      }
    }
  }
}

// --------------------------------------------------------------- launches --
enum WeighForm { kUnit, kFew, kSimt, kTc };
struct WeighPlan {
  WeighForm form;
  int stat_rows, stat_tiles;  // of the first launch
  int ctas_per_sm;
  int blocks, warps;          // of a cluster, of a block (kUnit)
  int score_rows;
  size_t row_ml, part, span, scores;  // bytes
};
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Up to 16 rows of a head group keep their scores in bf16: in the registers of one launch
// where they fit, else, as long as they take a workspace of at most 1 GB, in memory.  More
// rows, and what does not fit, have them computed twice on the tensor cores.  The three (us;
// 8 key/value heads, groups of 4, sequences x tokens):
//                           32 x 8000             1 x 40000       8 x 500
//   head size 128,  8 rows   63.8   86.9  117     -  26.2  35.3    9.4  12.4  14.8
//                  16 rows   82.4  104.7  118     -  30.4  35.2    9.5  12.2  14.8
//                  24 rows      -  133.5  120                        -     -  14.6
//                  32 rows      -  167.8  120     -  50.2  35.4      -  14.8  14.6
//   head size 64,   8 rows   42.6   57.5   78.5
//                  16 rows   65.3   74.7   78.2
//                  32 rows      -  131.7   77.9
// fp32 keeps them in memory always: it would be bound by computing them twice.
WeighPlan plan_of(int dtype, int T, int max_rows, int n_q, int n_kv, int hd, int n_seqs, int tokens) {
  const int rows = max_rows * (n_q / n_kv), r8 = (rows + 7) / 8 * 8;
  WeighPlan pl{};
  pl.score_rows = r8;
  // (what passes 64 bits, which only shapes that no memory holds do, stays the most there is)
  const size_t rows_all = static_cast<size_t>(n_kv) * r8 * sizeof(float), most = ~size_t{0} / 4 / n_seqs / tokens;
  const size_t scores = std::min(rows_all, most) * n_seqs * tokens;
  const bool keeps = scores <= (size_t{1} << 30);
  if (dtype == SPECFOLD_BF16) {
    // A cluster for a unit wherever 4 or 8 warps a block hold its scores.  Both sides (one launch,
    // two; us; sequences x tokens, head size 128), one row of 28 / 4 heads: 64 x 8000 69.3 and
    // 88, 64 x 16000 127 and 165, 8 x 8000 14.9 and 20.2, 1 x 16000 13.9 and 12.8, 1 x 2047 9.2
    // and 12; four of 32 / 8: 32 x 8000 82.4 and 105, 1 x 8000 10.6 and 14.4.  The rule knows the
    // room of the weights, not the lengths; where there is room for more tokens: 64 x 8000 of
    // 16384 85.3 and 87, of 32768 and more only the two launches, 87; 64 x 2000 of 16384 29.5 and 30.3;
    // four rows of 32 x 4000 of 8192 63 and 57.  With 16 warps a block full lengths gained
    // (32 x 30000 135 and 157), shorter ones lost (64 x 4000 of 32768 57 and 50).
    const long long units = static_cast<long long>(n_seqs) * n_kv;
    auto slice = [&](int blocks) { return ((tokens - 1) / blocks / kKeys + 1) * kKeys; };
    int blocks = 1;
    while (blocks < kUnitCluster && slice(blocks) > 256 &&
           (static_cast<long long>(slice(blocks)) * r8 > 4 * kUnitScores || units * blocks < 2LL * kSmBudget))
      blocks *= 2;
    const long long w = (static_cast<long long>(slice(blocks)) * r8 + kUnitScores - 1) / kUnitScores;
    const int warps = w <= 4 ? 4 : 8;
    if (rows <= 16 && w <= warps) {
      pl.form = kUnit;
      pl.blocks = blocks;
      pl.warps = warps;
      return pl;
    }
    if (keeps && rows <= 16) {
      pl.form = kFew;
      pl.stat_rows = r8;
      pl.ctas_per_sm = kFewCtas;
    } else {
      pl.form = kTc;
      pl.stat_rows = kWeighTcRows;
      pl.ctas_per_sm = 1;
    }
  } else {
    pl.form = kSimt;
    pl.stat_rows = 8;
    pl.ctas_per_sm = WSimt<128>::CTAS;
  }
  pl.row_ml = up256(static_cast<size_t>(T) * n_q * sizeof(float2));
  pl.stat_tiles = (rows + pl.stat_rows - 1) / pl.stat_rows;
  pl.part = up256(2 * static_cast<size_t>(kSmBudget) * pl.ctas_per_sm * pl.stat_rows * sizeof(float2));
  pl.span = up256(static_cast<size_t>(n_seqs) * n_kv * pl.stat_tiles * sizeof(int4));
  pl.scores = pl.form == kTc ? 0 : up256(scores);
  return pl;
}

int start(void (*kernel)(WeighArgs), const WeighArgs& a, int grid, int threads, int smem, cudaStream_t st) {
  if (smem > 0)
    if (const int rc = smem_limit_once(kernel, smem)) return rc;
  launch_k(kernel, dim3(grid), dim3(threads), smem, st, a);
  count_launch();
  return check_launch();
}

template <int HD, int NT, int WARPS>
int unit_start(const WeighPlan& pl, WeighArgs& a, cudaStream_t st) {
  auto kernel = weigh_unit_kernel<HD, NT, WARPS>;
  constexpr int smem = WFew<HD, NT, WARPS>::SMEM;
  if (const int rc = smem_limit_once(kernel, smem)) return rc;
  a.blocks = pl.blocks;
  a.spread = num_sms() * (16 / WARPS) / (a.t.batch.n_seqs * a.t.n_kv) + 1;
  launch_kc(kernel, dim3(a.t.batch.n_seqs * a.t.n_kv * pl.blocks), dim3(32 * WARPS), smem, st, pl.blocks, a);
  count_launch();
  return check_launch();
}

template <int HD>
int weigh_go(const KvWeighCall& c, cudaStream_t st) {
  const WeighPlan pl = plan_of(c.dtype, c.batch.T, c.max_rows, c.n_q, c.n_kv, HD, c.batch.n_seqs, c.w.tokens);
  WeighArgs a{};
  TreeArgs& t = a.t;
  t.q = c.q.ptr;
  t.q_rs = c.q.row_stride;
  t.q_hs = c.q.head_stride;
  t.cache = c.cache;
  t.batch = c.batch;
  t.max_nodes = c.max_rows;
  t.n_kv = c.n_kv;
  t.g = c.n_q / c.n_kv;
  t.most_tokens = c.w.tokens;
  t.sl2 = static_cast<float>(1.4426950408889634 * (c.scale > 0.f ? c.scale : 1.0 / std::sqrt(static_cast<double>(HD))));
  t.status = static_cast<uint32_t*>(c.ws);
  a.rows = c.rows;
  a.n_src = c.n_src;
  a.decay = c.decay;
  a.w = c.w;
  a.stat_rows = pl.stat_rows;
  a.stat_tiles = pl.stat_tiles;
  uint8_t* ws = static_cast<uint8_t*>(c.ws) + 256;
  a.row_ml = reinterpret_cast<float2*>(ws);
  a.part = reinterpret_cast<float2*>(ws + pl.row_ml);
  a.span = reinterpret_cast<int4*>(ws + pl.row_ml + pl.part);
  a.scores = reinterpret_cast<float*>(ws + pl.row_ml + pl.part + pl.span);
  a.score_rows = pl.score_rows;
  const int grid = std::min(num_sms(), kSmBudget) * pl.ctas_per_sm;
  t.w_full = t.w_half = 1;
  if (pl.form == kTc) return launch_weigh_tc(a, HD, grid, st);
  t.tile_rows = SPECFOLD_MAX_TREE * 128;
  t.kb = kKeys;
  if (pl.form == kUnit) {
    if (pl.score_rows == 8)
      return pl.warps == 4 ? unit_start<HD, 1, 4>(pl, a, st) : unit_start<HD, 1, 8>(pl, a, st);
    return pl.warps == 4 ? unit_start<HD, 2, 4>(pl, a, st) : unit_start<HD, 2, 8>(pl, a, st);
  }
  t.tile_rows = pl.stat_rows;
  t.kb = kKeys;
  t.unit_cost = 4;
  const int rc = pl.form == kSimt       ? start(weigh_simt_kernel<HD>, a, grid, kThreads, WSimt<HD>::SMEM, st)
                 : pl.stat_rows == 8 ? start(weigh_few_kernel<HD, 1>, a, grid, kThreads, WFew<HD, 1>::SMEM, st)
                                     : start(weigh_few_kernel<HD, 2>, a, grid, kThreads, WFew<HD, 2>::SMEM, st);
  if (rc) return rc;
  t.tile_rows = SPECFOLD_MAX_TREE * 128;  // all of a head group's rows
  return start(weigh_sum_kernel, a, num_sms() * kSumCtas, kSumThreads, 0, st);
}

}  // namespace

size_t kv_weigh_ws_bytes(int dtype, int T, int max_rows, int n_q, int n_kv, int hd, int n_seqs, int tokens) {
  const WeighPlan pl = plan_of(dtype, T, max_rows, n_q, n_kv, hd, n_seqs, tokens);
  return 256 + pl.row_ml + pl.part + pl.span + pl.scores;
}

int launch_kv_weigh(const KvWeighCall& c, cudaStream_t st) { return c.hd == 128 ? weigh_go<128>(c, st) : weigh_go<64>(c, st); }

}  // namespace sf
