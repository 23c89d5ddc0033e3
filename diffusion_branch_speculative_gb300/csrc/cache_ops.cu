// The row-wise operators of a decoder's paged cache: norm and rotation of
// the query and key heads, and the append of keys and values to the page
// pools.  Both are bound by the bytes of their rows, each read once and
// written once.
//
// Lanes: a head's row of hd elements is held by hd/16 lanes, lane c with the
// elements [8c, 8c + 8) and [hd/2 + 8c, hd/2 + 8c + 8): the two halves of its
// eight rotation pairs, so a rotation needs no exchange, a norm log2(hd/16)
// shuffles, and every access is 16 bytes (bf16) of a run of hd/16 lanes.  A
// warp holds 512/hd heads at once.
//
// Angles: the turn count of position p at frequency j is p * f_j with
// f_j = theta^(-2j/hd) / (2 pi).  f_j mod 1 is held as a 64-bit fraction F_j, so
// that the wrapping 64-bit product p * F_j is the angle reduced to one turn, for
// every 32-bit position: no large floating product and no 64-bit floating
// arithmetic on the device.  f_j itself is computed on the host in 64 bits, which
// leaves the angle off by at most p * 2^-49 turns (a base below one, whose
// frequencies rise: p * 2^-49 / theta).
//
// Both may release their dependents early, although what they write may be the prefix of
// the layer's attention, which reads it before its wait: no call of this library starts
// with that kernel in that form.  It comes behind one of the same call that has waited
// for its predecessor, by when these are complete.  Norm with rotation does (a captured
// step of norm, append and attention takes 12.0 us, 12.5 without).
#include "sf_device.cuh"
#include "sf_internal.h"

#include <algorithm>
#include <cmath>

namespace sf {
namespace {

constexpr int kThreads = 256;
// Resident blocks an SM, which cap the registers.  Measured (16381 rows of 24 + 8
// heads; 12233 rows of 8 heads appended): 2, 3, 4, 5 blocks 56.5, 48.3, 46.3,
// 68.5 us and 24.0, 21.0, 23.8, 27.5 us (one group in flight): fewer hold too few
// bytes in flight, more spill (four spill a little of the norm: 32 or 36 bytes a
// thread, fp32 104).  That is 5820 GB/s of the rows' 268 MB (copy peak 6690); the same
// rows of head size 64 4850 (134 MB), fp32 5430 (half the rows) and 5570.  The append
// moves its 100 MB at 5030 GB/s, 50 MB of head size 64 at 4050, fp32 at 5710 (201 MB)
// and 5160: the grid is one round of chunks of seven rows, DRAM is busy 36 % of it, and
// the warps that have values only are done early.  Positions with several axes cost the
// reads of a lane's eight of them, whose places lie in shared memory: the same rows take
// 47.1 and 20.2 us, by one position 46.9 and 19.9.
constexpr int kQkBlocks = 4, kAppendBlocks = 3;

// A lane's two runs of eight elements as they lie in memory: what a warp has in
// flight while it works on the group of heads before.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u[2];
  SF_DEV void read(const __nv_bfloat16* p, int half) {
    u[0] = *reinterpret_cast<const uint4*>(p);
    u[1] = *reinterpret_cast<const uint4*>(p + half);
  }
  SF_DEV void unpack(int i, float2 (&x)[4]) const {
    const uint32_t v[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = make_float2(bf16lo(v[e]), bf16hi(v[e]));
  }
};
template <>
struct Raw<float> {
  float4 u[4];
  SF_DEV void read(const float* p, int half) {
    u[0] = reinterpret_cast<const float4*>(p)[0];
    u[1] = reinterpret_cast<const float4*>(p)[1];
    u[2] = reinterpret_cast<const float4*>(p + half)[0];
    u[3] = reinterpret_cast<const float4*>(p + half)[1];
  }
  SF_DEV void unpack(int i, float2 (&x)[4]) const {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[2 * e] = make_float2(u[2 * i + e].x, u[2 * i + e].y);
      x[2 * e + 1] = make_float2(u[2 * i + e].z, u[2 * i + e].w);
    }
  }
};
// copied: neither normed nor rotated, so the upper halves are the bits that were read
// (a rounding would lose a NaN's sign and payload).  Writing the raw vectors instead
// costs registers: 55.2 us, not 46.6, for 16381 rows of 24 + 8 heads.
SF_DEV void store8(__nv_bfloat16* p, const float2 (&y)[4], bool copied) {
  uint32_t v[4];
  if (copied) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __byte_perm(__float_as_uint(y[e].x), __float_as_uint(y[e].y), 0x7632);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pack_bf16x2(y[e].x, y[e].y);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}
SF_DEV void store8(float* p, const float2 (&y)[4], bool) {
  reinterpret_cast<float4*>(p)[0] = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
}

// Turn fractions F_j of the rotation frequencies (see the file comment).
struct Turns {
  uint64_t f[64];
};
void rope_turns(float theta, int hd, Turns* t) {
  const double r = std::pow(static_cast<double>(theta), -2.0 / hd);
  double f = 0.15915494309189535;  // 1 / (2 pi)
  for (int j = 0; j < hd / 2; ++j, f *= r)
    t->f[j] = static_cast<uint64_t>((f - std::floor(f)) * 18446744073709551616.0);
}

// The same for several axes, whose pairs come in blocks or in turn, by the pair's
// place among all or among its axis's own; and the axis of every pair.
void rope_turns(const specfold_rope_axes& x, int hd, Turns* t, uint8_t* axis) {
  int done[SPECFOLD_MAX_AXES] = {};
  int a = 0;
  for (int j = 0; j < hd / 2; ++j) {
    while (done[a] == x.pairs[a]) a = (a + 1) % x.n_axes;  // the pairs add up to hd / 2
    const double at = x.own_frequencies ? static_cast<double>(done[a]) / x.pairs[a] : 2.0 * j / hd;
    const double f = 0.15915494309189535 * std::pow(static_cast<double>(x.theta), -at);  // 1 / (2 pi)
    t->f[j] = static_cast<uint64_t>((f - std::floor(f)) * 18446744073709551616.0);
    axis[j] = static_cast<uint8_t>(a);
    ++done[a];
    if (x.order == SPECFOLD_AXES_IN_TURN) a = (a + 1) % x.n_axes;
  }
}

// cos and sin of this lane's eight pairs (j = 8c .. 8c + 7), pair j at position
// pos[j % PER] of the lane that computes it.  Lane l computes the pairs HD/64*l ..
// of the warp's HD/2 frequencies and the eight come by shuffles: every angle once per
// warp.  For bf16 results the special function unit's sine and cosine do (off by at
// most 2^-20 on one turn, against a rounding of 2^-8).
template <typename T, int HD>
SF_DEV void lane_angles(const uint64_t* s_f, const long long (&pos)[HD / 64], int lane, int c, float2 (&cs)[4],
                        float2 (&sn)[4]) {
  constexpr int PER = HD / 64;  // angles a lane computes: 2 or 1
  float myc[PER], mys[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const uint64_t turn = static_cast<uint64_t>(pos[e]) * s_f[lane * PER + e];
    // the fraction's upper 32 bits as a signed number: half turns in [-1, 1)
    const float half = static_cast<float>(static_cast<int32_t>(turn >> 32));
    if constexpr (sizeof(T) == 2)
      __sincosf(half * (3.14159265358979f / 2147483648.f), &mys[e], &myc[e]);
    else
      sincospif(half * (1.f / 2147483648.f), &mys[e], &myc[e]);
  }
  auto from = [&](const float (&mine)[PER], int e) {
    return __shfl_sync(0xffffffffu, mine[e % PER], (8 * c + e) / PER);
  };
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    cs[e] = make_float2(from(myc, 2 * e), from(myc, 2 * e + 1));
    sn[e] = make_float2(from(mys, 2 * e), from(mys, 2 * e + 1));
  }
}

// The rows' positions: one a row, or one a row and axis (AXES), of which a lane
// reads those of its own pairs.
struct Places {
  const int32_t* p;  // null, for one a row: the token's own index
  long long rs, as;  // from row to row, from axis to axis (AXES)
  uint8_t axis[64];  // of every pair (AXES)
};
// Row t's for this lane's pairs; s_off (AXES): where a pair's axis begins; own: the token's index.
template <int HD, bool AXES>
SF_DEV void read_places(const Places& at, const long long* s_off, int lane, long long t, long long own,
                        long long (&pos)[HD / 64]) {
  if constexpr (AXES) {
    const int32_t* row = at.p + t * at.rs;
#pragma unroll
    for (int e = 0; e < HD / 64; ++e) pos[e] = row[s_off[lane * (HD / 64) + e]];
  } else {
    const long long x = at.p ? at.p[t] : own;
#pragma unroll
    for (int e = 0; e < HD / 64; ++e) pos[e] = x;
  }
}

// One head's row in registers (two runs of eight, from 8c and HD/2 + 8c on): the
// norm with the gain g (null: none), then the rotation.  The whole warp takes
// part; g is at the lane's first element.
template <int HD>
SF_DEV void norm_rotate(float2 (&a)[4], float2 (&b)[4], const float* g, float eps, bool rope, const float2 (&cs)[4],
                        const float2 (&sn)[4]) {
  if (g) {
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fma2(a[e], a[e], fma2(b[e], b[e], ss));
    float sum = ss.x + ss.y;
#pragma unroll
    for (int o = HD / 32; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = rsqrtf(sum * (1.f / HD) + eps);  // off by at most 2^-22
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = mul2(mul2(a[e], inv2), reinterpret_cast<const float2*>(g)[e]);
      b[e] = mul2(mul2(b[e], inv2), reinterpret_cast<const float2*>(g + HD / 2)[e]);
    }
  }
  if (rope) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = a[e], y = b[e], minus = make_float2(-sn[e].x, -sn[e].y);
      a[e] = fma2(x, cs[e], mul2(y, minus));
      b[e] = fma2(y, cs[e], mul2(x, sn[e]));
    }
  }
}

template <typename T>
struct Rows {
  T* p;
  long long rs, hs;
};
template <typename T>
Rows<T> rows_of(const specfold_head_rows& v) {
  return {static_cast<T*>(v.ptr), v.row_stride, v.head_stride};
}

// ------------------------------------------------------ norm and rotation --
template <typename T>
struct QkArgs {
  Rows<T> q_in, k_in, q_out, k_out;
  const T* gq;
  const T* gk;
  int T_rows, n_q, n_kv, parts, rope;
  float eps;
  Turns turns;
  Places places;
};

// Work item: row t, one of `parts` shares of its heads (a few rows alone
// would leave most SMs idle), one warp each.
template <typename T, int HD, bool AXES>
__global__ void __launch_bounds__(kThreads, kQkBlocks) qk_norm_rope_kernel(const __grid_constant__ QkArgs<T> p) {
  constexpr int LPR = HD / 16, RPW = 32 / LPR;
  __shared__ uint64_t s_f[HD / 2];
  __shared__ __align__(16) float s_g[2][HD];
  __shared__ long long s_off[AXES ? HD / 2 : 1];
  if (p.rope && threadIdx.x < HD / 2) s_f[threadIdx.x] = p.turns.f[threadIdx.x];
  if (AXES && threadIdx.x < HD / 2) s_off[threadIdx.x] = p.places.axis[threadIdx.x] * p.places.as;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < HD; i += kThreads) {
    if (p.gq) s_g[0][i] = static_cast<float>(p.gq[i]);
    if (p.gk) s_g[1][i] = static_cast<float>(p.gk[i]);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  // a unit is a group of heads that a warp holds at once, queries' before keys'
  const int units_q = (p.n_q + RPW - 1) / RPW, units = units_q + (p.n_kv + RPW - 1) / RPW;
  const long long items = static_cast<long long>(p.T_rows) * p.parts;
  const long long step = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const int t = static_cast<int>(it / p.parts);
    const int first = static_cast<int>(it - static_cast<long long>(t) * p.parts);
    auto read = [&](int u, Raw<T>& x) {
      const bool is_q = u < units_q;
      const int h = (is_q ? u : u - units_q) * RPW + sub;
      const Rows<T>& in = is_q ? p.q_in : p.k_in;
      if (u < units && h < (is_q ? p.n_q : p.n_kv)) x.read(in.p + t * in.rs + h * in.hs + 8 * c, HD / 2);
    };
    Raw<T> next = {};
    read(first, next);
    float2 cs[4], sn[4];
    if (p.rope) {
      long long pos[HD / 64];
      read_places<HD, AXES>(p.places, s_off, lane, t, 0, pos);
      lane_angles<T, HD>(s_f, pos, lane, c, cs, sn);
    }
    for (int u = first; u < units; u += p.parts) {
      float2 a[4], b[4];
      next.unpack(0, a);
      next.unpack(1, b);
      read(u + p.parts, next);
      const bool is_q = u < units_q;
      const int h = (is_q ? u : u - units_q) * RPW + sub;
      const float* g = is_q ? (p.gq ? &s_g[0][8 * c] : nullptr) : (p.gk ? &s_g[1][8 * c] : nullptr);
      norm_rotate<HD>(a, b, g, p.eps, p.rope != 0, cs, sn);
      const Rows<T>& out = is_q ? p.q_out : p.k_out;
      if (h < (is_q ? p.n_q : p.n_kv)) {  // lanes behind the last head hold leftovers
        T* y = out.p + t * out.rs + h * out.hs + 8 * c;
        const bool copied = !g && !p.rope;
        store8(y, a, copied);
        store8(y + HD / 2, b, copied);
      }
    }
  }
}

// Frequencies and positions of a call; false: it does not rotate.
bool rotation(const RopePlan& r, int hd, Turns* turns, Places* at) {
  at->p = r.positions;
  at->rs = r.row_stride;
  at->as = r.axis_stride;
  if (!r.axes) {
    if (r.theta > 0.f) rope_turns(r.theta, hd, turns);
    return r.theta > 0.f;
  }
  rope_turns(*r.axes, hd, turns, at->axis);
  return true;
}

template <typename T, int HD, bool AXES>
int qk_go(const QkNormRopeCall& c, cudaStream_t st) {
  QkArgs<T> a;
  a.q_in = rows_of<T>(c.q_in);
  a.k_in = rows_of<T>(c.k_in);
  a.q_out = rows_of<T>(c.q_out);
  a.k_out = rows_of<T>(c.k_out);
  a.gq = static_cast<const T*>(c.gq);
  a.gk = static_cast<const T*>(c.gk);
  a.T_rows = c.T;
  a.n_q = c.n_q;
  a.n_kv = c.n_kv;
  a.eps = c.eps;
  a.rope = rotation(c.rope, HD, &a.turns, &a.places);
  const int units = (c.n_q + 512 / HD - 1) / (512 / HD) + (c.n_kv + 512 / HD - 1) / (512 / HD);
  // shares of a row's heads: enough that the last round of the grid's warps weighs little
  const long long want = 6LL * kQkBlocks * num_sms() * (kThreads / 32);
  a.parts = static_cast<int>(std::min<long long>(units, std::max<long long>(1, (want + c.T - 1) / c.T)));
  const long long blocks = (static_cast<long long>(c.T) * a.parts + kThreads / 32 - 1) / (kThreads / 32);
  launch_k(qk_norm_rope_kernel<T, HD, AXES>, dim3(static_cast<unsigned>(std::min<long long>(blocks, static_cast<long long>(kQkBlocks) * num_sms()))),
           dim3(kThreads), 0, st, a);
  count_launch();
  return check_launch();
}

// ---------------------------------------------------------------- append --
template <typename T>
struct AppendArgs {
  Rows<T> k, v;
  const int32_t* rows;
  const T* gk;
  specfold_paged_cache cache;
  SeqBatch batch;
  uint32_t* status;
  int n_kv, n_src, rope, chunk;
  float eps;
  Turns turns;
  Places places;
};

// Work item: the keys, or the values, of a chunk of consecutive rows, one warp.
// A row's place takes a search for its sequence (over the batch's entries in
// shared memory) and its table's entry: lane r has row r's, so a chunk waits
// for them once.  The rows' groups of heads then stream through with the next
// one in flight.
template <typename T, int HD, bool AXES>
__global__ void __launch_bounds__(kThreads, kAppendBlocks) kv_append_kernel(const __grid_constant__ AppendArgs<T> p) {
  constexpr int LPR = HD / 16, RPW = 32 / LPR;
  __shared__ uint64_t s_f[HD / 2];
  __shared__ __align__(16) float s_g[HD];
  __shared__ int s_start[SPECFOLD_MAX_SEQS + 1], s_ctx[SPECFOLD_MAX_SEQS];
  __shared__ long long s_off[AXES ? HD / 2 : 1];
  if (p.rope && threadIdx.x < HD / 2) s_f[threadIdx.x] = p.turns.f[threadIdx.x];
  if (AXES && threadIdx.x < HD / 2) s_off[threadIdx.x] = p.places.axis[threadIdx.x] * p.places.as;
  // Dependents are not released early: it would be sound (see above), but takes appended
  // prompts 20.3 us, not 19.9, and a captured step of norm, append and attention gains nothing.
  pdl_wait();
  if (p.gk)
    for (int i = threadIdx.x; i < HD; i += kThreads) s_g[i] = static_cast<float>(p.gk[i]);
  const SeqBatch& bt = p.batch;
  for (int s = threadIdx.x; s <= bt.n_seqs; s += kThreads) {
    s_start[s] = bt.row_start[s];
    if (s < bt.n_seqs) s_ctx[s] = bt.ctx_len[s];
  }
  __syncthreads();
  auto bad_seq = [&](int s) {
    return s_start[s] < 0 || s_start[s + 1] < s_start[s] || s_start[s + 1] > bt.T || s_ctx[s] < 0;
  };
  if (p.status && blockIdx.x == 0) {  // the batch's own validity, whether or not it has rows
    bool bad = false;
    for (int s = threadIdx.x; s < bt.n_seqs; s += kThreads) bad = bad || bad_seq(s);
    if (bad) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
  }
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  const specfold_paged_cache& ch = p.cache;
  const int units = (p.n_kv + RPW - 1) / RPW;
  const int chunks = (bt.T - 1) / p.chunk + 1;
  const long long items = 2LL * chunks, step = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const bool is_v = it & 1;
    const int t0 = static_cast<int>(it >> 1) * p.chunk, n = min(p.chunk, bt.T - t0);
    int src = -1, slot = -1;
    unsigned tok = 0;
    if (lane < n) {
      const int t = t0 + lane;
      src = p.rows ? p.rows[t] : t;
      int lo = -1, hi = bt.n_seqs;  // the last sequence that starts at t or before it
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= t)
          lo = mid;
        else
          hi = mid;
      }
      if (lo >= 0 && t < s_start[lo + 1] && !bad_seq(lo)) {
        uint32_t wrong = 0u;
        tok = static_cast<unsigned>(s_ctx[lo]) + static_cast<unsigned>(t - s_start[lo]);  // < 2^32
        const unsigned pg = tok / static_cast<unsigned>(ch.page_size);
        int page = -1;
        if (pg < static_cast<unsigned>(ch.table_pages)) page = ch.block_table[lo * ch.table_stride + pg];
        if (src < 0 || src >= p.n_src)
          wrong = SPECFOLD_DEV_BAD_SEQ;
        else if (page < 0 || page >= ch.num_pages)
          wrong = SPECFOLD_DEV_BAD_PAGE;
        else
          slot = page * ch.page_size + static_cast<int>(tok - pg * ch.page_size);
        if (wrong && p.status) atomicOr(p.status, wrong);
      }
    }
    const Rows<T>& in = is_v ? p.v : p.k;
    T* pool = static_cast<T*>(is_v ? ch.v : ch.k) + 8 * c;
    const long long ts = is_v ? ch.v_token_stride : ch.k_token_stride, hs = is_v ? ch.v_head_stride : ch.k_head_stride;
    const bool rope = p.rope && !is_v, norm = p.gk && !is_v;
    auto read = [&](int r, int u, Raw<T>& x) {  // the whole warp: row r's group u
      const int from = __shfl_sync(0xffffffffu, src, r), to = __shfl_sync(0xffffffffu, slot, r), h = u * RPW + sub;
      if (to >= 0 && h < p.n_kv) x.read(in.p + from * in.rs + h * in.hs + 8 * c, HD / 2);
    };
    // the chunk's groups in one sequence, kDepth of them in flight
    struct At {
      int r, u;
      SF_DEV void next(int units) {
        if (++u == units) {
          u = 0;
          ++r;
        }
      }
    };
    // (12233 rows of 8 heads: 21.0 us with one, 19.9 with two, 21.3 with three; fp32
    // has as many bytes in one)
    constexpr int kDepth = sizeof(T) == 2 ? 2 : 1;
    Raw<T> flight[kDepth] = {};
    At ahead = {0, 0}, now = {0, 0};
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (ahead.r < n) read(ahead.r, ahead.u, flight[d]);
      ahead.next(units);
    }
    float2 cs[4], sn[4];
    int to = -1;
    while (now.r < n) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (now.r >= n) break;
        if (now.u == 0) {
          to = __shfl_sync(0xffffffffu, slot, now.r);
          const long long at = __shfl_sync(0xffffffffu, tok, now.r);
          if (rope) {
            long long pos[HD / 64];
            read_places<HD, AXES>(p.places, s_off, lane, t0 + now.r, at, pos);
            lane_angles<T, HD>(s_f, pos, lane, c, cs, sn);
          }
        }
        const int h = now.u * RPW + sub;
        float2 a[4], b[4];
        flight[d].unpack(0, a);
        flight[d].unpack(1, b);
        if (ahead.r < n) read(ahead.r, ahead.u, flight[d]);
        ahead.next(units);
        norm_rotate<HD>(a, b, norm ? s_g + 8 * c : nullptr, p.eps, rope, cs, sn);
        if (to >= 0 && h < p.n_kv) {
          T* y = pool + to * ts + h * hs;
          const bool copied = !norm && !rope;
          store8(y, a, copied);
          store8(y + HD / 2, b, copied);
        }
        now.next(units);
      }
    }
  }
}

template <typename T, int HD, bool AXES>
int append_go(const KvAppendCall& c, cudaStream_t st) {
  AppendArgs<T> a;
  a.k = rows_of<T>(c.k);
  a.v = rows_of<T>(c.v);
  a.rows = c.rows;
  a.gk = static_cast<const T*>(c.gk);
  a.cache = c.cache;
  a.batch = c.batch;
  a.status = c.status;
  a.n_kv = c.n_kv;
  a.n_src = c.n_src;
  a.eps = c.eps;
  a.rope = rotation(c.rope, HD, &a.turns, &a.places);
  // chunks of rows such that the grid's warps take one each, and no more than a warp's lanes
  const long long warps = static_cast<long long>(kAppendBlocks) * num_sms() * (kThreads / 32);
  a.chunk = static_cast<int>(std::min<long long>(32, (2LL * c.batch.T + warps - 1) / warps));
  const long long blocks = (2LL * ((c.batch.T - 1) / a.chunk + 1) + kThreads / 32 - 1) / (kThreads / 32);
  launch_k(kv_append_kernel<T, HD, AXES>, dim3(static_cast<unsigned>(std::min<long long>(blocks, static_cast<long long>(kAppendBlocks) * num_sms()))),
           dim3(kThreads), 0, st, a);
  count_launch();
  return check_launch();
}

}  // namespace

// Element type, head size and kind of positions of a call to its instance.
#define SF_ROPE_DISPATCH(go)                                                                        \
  const bool axes = c.rope.axes != nullptr;                                                         \
  if (c.dtype == SPECFOLD_BF16) {                                                                   \
    if (c.hd == 128) return axes ? go<__nv_bfloat16, 128, true>(c, st) : go<__nv_bfloat16, 128, false>(c, st); \
    return axes ? go<__nv_bfloat16, 64, true>(c, st) : go<__nv_bfloat16, 64, false>(c, st);         \
  }                                                                                                 \
  if (c.hd == 128) return axes ? go<float, 128, true>(c, st) : go<float, 128, false>(c, st);        \
  return axes ? go<float, 64, true>(c, st) : go<float, 64, false>(c, st)

int launch_qk_norm_rope(const QkNormRopeCall& c, cudaStream_t st) { SF_ROPE_DISPATCH(qk_go); }
int launch_kv_append(const KvAppendCall& c, cudaStream_t st) { SF_ROPE_DISPATCH(append_go); }

}  // namespace sf
