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
// leaves the angle off by at most p * 2^-49 turns.
#include "sf_device.cuh"
#include "sf_internal.h"

#include <algorithm>
#include <cmath>

namespace sf {
namespace {

constexpr int kThreads = 256;

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
  SF_DEV void unpack(int i, float (&x)[8]) const {
    x[0] = bf16lo(u[i].x); x[1] = bf16hi(u[i].x); x[2] = bf16lo(u[i].y); x[3] = bf16hi(u[i].y);
    x[4] = bf16lo(u[i].z); x[5] = bf16hi(u[i].z); x[6] = bf16lo(u[i].w); x[7] = bf16hi(u[i].w);
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
  SF_DEV void unpack(int i, float (&x)[8]) const {
    const float4 a = u[2 * i], b = u[2 * i + 1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
SF_DEV void store8(__nv_bfloat16* p, const float (&y)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                            pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}
SF_DEV void store8(float* p, const float (&y)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
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

// cos and sin of this lane's eight pairs (j = 8c .. 8c + 7) at position pos.
// Lane l computes the pairs HD/64*l .. of the warp's HD/2 frequencies and the
// eight come by shuffles: every angle once per warp.
template <int HD>
SF_DEV void lane_angles(const uint64_t* s_f, long long pos, int lane, int c, float (&cs)[8], float (&sn)[8]) {
  constexpr int PER = HD / 64;  // angles a lane computes: 2 or 1
  float myc[PER], mys[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const uint64_t turn = static_cast<uint64_t>(pos) * s_f[lane * PER + e];
    // the fraction's upper 32 bits as a signed number: half turns in [-1, 1)
    const float half = static_cast<float>(static_cast<int32_t>(turn >> 32)) * (1.f / 2147483648.f);
    sincospif(half, &mys[e], &myc[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int from = (8 * c + e) / PER;
    cs[e] = __shfl_sync(0xffffffffu, myc[e % PER], from);
    sn[e] = __shfl_sync(0xffffffffu, mys[e % PER], from);
  }
}

// One head's row in registers (two runs of eight, from 8c and HD/2 + 8c on): the
// norm with the gain g where `normed`, then the rotation.  Every lane of the
// warp takes part in the sum.
template <int HD>
SF_DEV void norm_rotate(float (&a)[8], float (&b)[8], bool any_norm, bool normed, const float* g, float eps, bool rope,
                        const float (&cs)[8], const float (&sn)[8]) {
  if (any_norm) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
    for (int o = HD / 32; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (normed) {
      // a square root and a division, as the formula has them: one per row and lane
      const float inv = 1.f / sqrtf(ss * (1.f / HD) + eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = a[e] * inv * g[e];
        b[e] = b[e] * inv * g[HD / 2 + e];
      }
    }
  }
  if (rope) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = a[e], y = b[e];
      a[e] = x * cs[e] - y * sn[e];
      b[e] = y * cs[e] + x * sn[e];
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
  const int32_t* positions;
  int T_rows, n_q, n_kv, parts, rope;
  float eps;
  Turns turns;
};

// Work item: row t, one of `parts` shares of its heads (a few rows alone
// would leave most SMs idle), one warp each.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_kernel(const __grid_constant__ QkArgs<T> p) {
  constexpr int LPR = HD / 16, RPW = 32 / LPR;
  __shared__ uint64_t s_f[HD / 2];
  __shared__ float s_g[2][HD];
  if (p.rope && threadIdx.x < HD / 2) s_f[threadIdx.x] = p.turns.f[threadIdx.x];
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < HD; i += kThreads) {
    if (p.gq) s_g[0][i] = static_cast<float>(p.gq[i]);
    if (p.gk) s_g[1][i] = static_cast<float>(p.gk[i]);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  const int heads = p.n_q + p.n_kv, units = (heads + RPW - 1) / RPW;
  const long long items = static_cast<long long>(p.T_rows) * p.parts;
  const long long step = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const int t = static_cast<int>(it / p.parts);
    const int first = static_cast<int>(it - static_cast<long long>(t) * p.parts);
    auto read = [&](int u, Raw<T>& x) {
      const int hh = u * RPW + sub;
      if (u < units && hh < heads) {
        const Rows<T>& in = hh < p.n_q ? p.q_in : p.k_in;
        x.read(in.p + t * in.rs + (hh < p.n_q ? hh : hh - p.n_q) * in.hs + 8 * c, HD / 2);
      }
    };
    Raw<T> next = {};
    read(first, next);
    float cs[8], sn[8];
    if (p.rope) lane_angles<HD>(s_f, p.positions[t], lane, c, cs, sn);
    for (int u = first; u < units; u += p.parts) {
      const int hh = u * RPW + sub;
      const bool is_q = hh < p.n_q;
      float a[8], b[8];
      next.unpack(0, a);
      next.unpack(1, b);
      read(u + p.parts, next);
      // a warp may hold query and key heads at once, of which one side alone is
      // normed (and, behind the last head, lanes with leftovers, not stored)
      norm_rotate<HD>(a, b, p.gq || p.gk, is_q ? p.gq != nullptr : p.gk != nullptr, &s_g[is_q ? 0 : 1][8 * c], p.eps,
                      p.rope != 0, cs, sn);
      if (hh < heads) {
        const Rows<T>& out = is_q ? p.q_out : p.k_out;
        T* y = out.p + t * out.rs + (is_q ? hh : hh - p.n_q) * out.hs + 8 * c;
        store8(y, a);
        store8(y + HD / 2, b);
      }
    }
  }
}

template <typename T, int HD>
int qk_go(const QkNormRopeCall& c, cudaStream_t st) {
  QkArgs<T> a;
  a.q_in = rows_of<T>(c.q_in);
  a.k_in = rows_of<T>(c.k_in);
  a.q_out = rows_of<T>(c.q_out);
  a.k_out = rows_of<T>(c.k_out);
  a.gq = static_cast<const T*>(c.gq);
  a.gk = static_cast<const T*>(c.gk);
  a.positions = c.positions;
  a.T_rows = c.T;
  a.n_q = c.n_q;
  a.n_kv = c.n_kv;
  a.eps = c.eps;
  a.rope = c.theta > 0.f;
  if (a.rope) rope_turns(c.theta, HD, &a.turns);
  const int units = (c.n_q + c.n_kv + 512 / HD - 1) / (512 / HD);
  // shares of a row's heads: as many as give every SM two blocks
  const long long want = 2LL * num_sms() * (kThreads / 32);
  a.parts = static_cast<int>(std::min<long long>(units, std::max<long long>(1, want / c.T)));
  const long long blocks = (static_cast<long long>(c.T) * a.parts + kThreads / 32 - 1) / (kThreads / 32);
  launch_k(qk_norm_rope_kernel<T, HD>, dim3(static_cast<unsigned>(std::min<long long>(blocks, 4LL * num_sms()))),
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
  const int32_t* positions;
  specfold_paged_cache cache;
  SeqBatch batch;
  uint32_t* status;
  int n_kv, n_src, rope, chunk;
  float eps;
  Turns turns;
};

// Work item: the keys, or the values, of a chunk of consecutive rows, one warp.
// A row's place takes a search for its sequence (over the batch's entries in
// shared memory) and its table's entry: lane r has row r's, so a chunk waits
// for them once.  The rows' groups of heads then stream through with the next
// one in flight.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 4) kv_append_kernel(const __grid_constant__ AppendArgs<T> p) {
  constexpr int LPR = HD / 16, RPW = 32 / LPR;
  __shared__ uint64_t s_f[HD / 2];
  __shared__ float s_g[HD];
  __shared__ int s_start[SPECFOLD_MAX_SEQS + 1], s_ctx[SPECFOLD_MAX_SEQS];
  if (p.rope && threadIdx.x < HD / 2) s_f[threadIdx.x] = p.turns.f[threadIdx.x];
  // No early release of dependents: a dependent may read the cache (a prefix
  // view) before its own wait.
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
  const int chunks = (bt.T + p.chunk - 1) / p.chunk;
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
    Raw<T> next = {};
    read(0, 0, next);
    float cs[8], sn[8];
    for (int r = 0; r < n; ++r) {
      const int to = __shfl_sync(0xffffffffu, slot, r);
      if (rope) {
        const long long at = __shfl_sync(0xffffffffu, tok, r);
        lane_angles<HD>(s_f, p.positions ? p.positions[t0 + r] : at, lane, c, cs, sn);
      }
      for (int u = 0; u < units; ++u) {
        const int h = u * RPW + sub;
        float a[8], b[8];
        next.unpack(0, a);
        next.unpack(1, b);
        const bool last = u == units - 1;
        if (!last || r + 1 < n) read(last ? r + 1 : r, last ? 0 : u + 1, next);
        norm_rotate<HD>(a, b, norm, norm, s_g + 8 * c, p.eps, rope, cs, sn);
        if (to >= 0 && h < p.n_kv) {
          T* y = pool + to * ts + h * hs;
          store8(y, a);
          store8(y + HD / 2, b);
        }
      }
    }
  }
}

template <typename T, int HD>
int append_go(const KvAppendCall& c, cudaStream_t st) {
  AppendArgs<T> a;
  a.k = rows_of<T>(c.k);
  a.v = rows_of<T>(c.v);
  a.rows = c.rows;
  a.gk = static_cast<const T*>(c.gk);
  a.positions = c.positions;
  a.cache = c.cache;
  a.batch = c.batch;
  a.status = c.status;
  a.n_kv = c.n_kv;
  a.n_src = c.n_src;
  a.eps = c.eps;
  a.rope = c.theta > 0.f;
  if (a.rope) rope_turns(c.theta, HD, &a.turns);
  // chunks that give every SM the 32 warps it holds, and no more than a warp's rows
  a.chunk = std::min(32, std::max(1, static_cast<int>(2LL * c.batch.T / (32LL * num_sms()))));
  const long long blocks = (2LL * ((c.batch.T + a.chunk - 1) / a.chunk) + kThreads / 32 - 1) / (kThreads / 32);
  launch_k(kv_append_kernel<T, HD>, dim3(static_cast<unsigned>(std::min<long long>(blocks, 4LL * num_sms()))),
           dim3(kThreads), 0, st, a);
  count_launch();
  return check_launch();
}

}  // namespace

int launch_qk_norm_rope(const QkNormRopeCall& c, cudaStream_t st) {
  if (c.dtype == SPECFOLD_BF16) return c.hd == 128 ? qk_go<__nv_bfloat16, 128>(c, st) : qk_go<__nv_bfloat16, 64>(c, st);
  return c.hd == 128 ? qk_go<float, 128>(c, st) : qk_go<float, 64>(c, st);
}

int launch_kv_append(const KvAppendCall& c, cudaStream_t st) {
  if (c.dtype == SPECFOLD_BF16)
    return c.hd == 128 ? append_go<__nv_bfloat16, 128>(c, st) : append_go<__nv_bfloat16, 64>(c, st);
  return c.hd == 128 ? append_go<float, 128>(c, st) : append_go<float, 64>(c, st);
}

}  // namespace sf
