// The attention weight that cached tokens get from a batch of rows, added up per
// key/value head (specfold_kv_weigh): what an eviction goes by.  Keys alone are
// read.  Two passes over the scores: every row's maximum and sum, then each
// token's weights over the rows.
#include "sf_device.cuh"
#include "sf_internal.h"

#include <algorithm>
#include <cmath>

namespace sf {
namespace {

struct WeighArgs {
  const void* q;
  long long q_rs, q_hs;
  const int32_t* rows;
  int n_src;
  specfold_paged_cache cache;
  SeqBatch batch;
  int max_rows, n_kv, g;
  float sl2, decay;  // scale * log2(e)
  specfold_token_weights w;
  uint32_t* status;
  float2* stats;  // [T][n_kv * g]: a row's maximum in log2 units, and one over its sum
};

// One sequence of the batch: n rows behind ctx tokens; n 0 where it is invalid.
struct WeighSeq {
  int row0, n, ctx;
};
SF_DEV WeighSeq weigh_seq(const WeighArgs& p, int s, bool report) {
  WeighSeq q;
  q.row0 = p.batch.row_start[s];
  const int end = p.batch.row_start[s + 1];
  q.ctx = p.batch.ctx_len[s];
  const bool bad = q.row0 < 0 || end < q.row0 || end > p.batch.T || end - q.row0 > p.max_rows || q.ctx < 0 ||
                   static_cast<long long>(q.ctx) + (end - q.row0) > p.w.tokens;
  if (bad && report) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
  q.n = bad ? 0 : end - q.row0;
  return q;
}
SF_DEV int weigh_slot(const WeighArgs& p, int s, int tok) {
  const specfold_paged_cache& c = p.cache;
  const unsigned pg = static_cast<unsigned>(tok) / static_cast<unsigned>(c.page_size);
  if (pg < static_cast<unsigned>(c.table_pages)) {
    const int page = c.block_table[s * c.table_stride + pg];
    if (page >= 0 && page < c.num_pages) return page * c.page_size + (tok - static_cast<int>(pg) * c.page_size);
  }
  atomicOr(p.status, SPECFOLD_DEV_BAD_PAGE);
  return -1;
}
// The row of q that row t of the batch takes, or -1 (reported).
SF_DEV int weigh_row(const WeighArgs& p, int t) {
  const int r = p.rows ? p.rows[t] : t;
  if (r >= 0 && r < p.n_src) return r;
  atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
  return -1;
}

constexpr int kThreads = 128;

template <typename T, int HD>
SF_DEV float dot_row(const T* k, const float* q) {
  float a = 0.f;
#pragma unroll 8
  for (int d = 0; d < HD; ++d) a = fmaf(static_cast<float>(k[d]), q[d], a);
  return a;
}

// One block a row and query head.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) weigh_stats_kernel(const __grid_constant__ WeighArgs p) {
  __shared__ float s_q[HD], s_m[kThreads], s_l[kThreads];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / p.g;
  int s = 0;
  while (s < p.batch.n_seqs && !(p.batch.row_start[s] <= t && t < p.batch.row_start[s + 1])) ++s;
  if (s == p.batch.n_seqs) return;
  const WeighSeq q = weigh_seq(p, s, false);
  if (q.n == 0) return;
  float2* out = p.stats + static_cast<size_t>(t) * p.n_kv * p.g + hq;
  const int src = weigh_row(p, t);
  if (src < 0) {  // weighs nothing
    if (threadIdx.x == 0) *out = make_float2(INFINITY, 0.f);
    return;
  }
  for (int d = threadIdx.x; d < HD; d += kThreads)
    s_q[d] = static_cast<float>(static_cast<const T*>(p.q)[src * p.q_rs + hq * p.q_hs + d]);
  __syncthreads();
  const int len = q.ctx + (t - q.row0) + 1;
  float m = -INFINITY, l = 0.f;
  for (int k = threadIdx.x; k < len; k += kThreads) {
    const int slot = weigh_slot(p, s, k);
    float x = 0.f;
    if (slot >= 0)
      x = dot_row<T, HD>(static_cast<const T*>(p.cache.k) + slot * p.cache.k_token_stride + h * p.cache.k_head_stride, s_q) *
          p.sl2;
    const float top = fmaxf(m, x);
    const float base = top == -INFINITY ? 0.f : top;
    l = l * (m == top ? 1.f : ex2(m - base)) + ex2(x - base);
    m = top;
  }
  s_m[threadIdx.x] = m;
  s_l[threadIdx.x] = l;
  __syncthreads();
  if (threadIdx.x == 0) {
    float M = -INFINITY, L = 0.f;
    for (int i = 0; i < kThreads; ++i) M = fmaxf(M, s_m[i]);
    for (int i = 0; i < kThreads; ++i) L += s_m[i] == M ? s_l[i] : ex2(s_m[i] - M) * s_l[i];
    *out = make_float2(M, 1.f / L);
  }
}

// One thread a token and key/value head.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) weigh_tokens_kernel(const __grid_constant__ WeighArgs p) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.y, h = blockIdx.z;
  const WeighSeq q = weigh_seq(p, s, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  const int len = q.n > 0 ? q.ctx + q.n : 0;
  for (int k = blockIdx.x * kThreads + threadIdx.x; k < len; k += gridDim.x * kThreads) {
    const int slot = weigh_slot(p, s, k);
    const T* kp = static_cast<const T*>(p.cache.k) + max(slot, 0) * p.cache.k_token_stride + h * p.cache.k_head_stride;
    float kv[HD], sum = 0.f;
    for (int d = 0; d < HD; ++d) kv[d] = slot < 0 ? 0.f : static_cast<float>(kp[d]);
    for (int i = max(0, k - q.ctx); i < q.n; ++i) {
      const int src = weigh_row(p, q.row0 + i);
      if (src < 0) continue;
      for (int j = 0; j < p.g; ++j) {
        const int hq = h * p.g + j;
        const T* qp = static_cast<const T*>(p.q) + src * p.q_rs + hq * p.q_hs;
        const float2 ml = p.stats[static_cast<size_t>(q.row0 + i) * p.n_kv * p.g + hq];
        const float x = dot_row<T, HD>(qp, kv) * p.sl2;
        sum += (x == ml.x ? 1.f : ex2(x - ml.x)) * ml.y;
      }
    }
    float* w = p.w.ptr + s * p.w.seq_stride + h * p.w.head_stride + k;
    *w = k < q.ctx && p.decay != 0.f ? fmaf(p.decay, *w, sum) : sum;
  }
}

template <typename T, int HD>
int weigh_go(const KvWeighCall& c, cudaStream_t st) {
  WeighArgs a{};
  a.q = c.q.ptr;
  a.q_rs = c.q.row_stride;
  a.q_hs = c.q.head_stride;
  a.rows = c.rows;
  a.n_src = c.n_src;
  a.cache = c.cache;
  a.batch = c.batch;
  a.max_rows = c.max_rows;
  a.n_kv = c.n_kv;
  a.g = c.n_q / c.n_kv;
  a.sl2 = static_cast<float>(1.4426950408889634 * (c.scale > 0.f ? c.scale : 1.0 / std::sqrt(static_cast<double>(HD))));
  a.decay = c.decay;
  a.w = c.w;
  a.status = static_cast<uint32_t*>(c.ws);
  a.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(c.ws) + 256);
  launch_k(weigh_stats_kernel<T, HD>, dim3(c.batch.T, c.n_q), dim3(kThreads), 0, st, a);
  count_launch();
  if (const int rc = check_launch()) return rc;
  launch_k(weigh_tokens_kernel<T, HD>, dim3(std::min((c.w.tokens - 1) / kThreads + 1, 64), c.batch.n_seqs, c.n_kv), dim3(kThreads), 0,
           st, a);
  count_launch();
  return check_launch();
}

}  // namespace

size_t kv_weigh_ws_bytes(int, int T, int, int n_q, int, int, int, int) {
  return 256 + static_cast<size_t>(T) * n_q * sizeof(float2);
}

int launch_kv_weigh(const KvWeighCall& c, cudaStream_t st) {
  if (c.dtype == SPECFOLD_BF16) return c.hd == 128 ? weigh_go<__nv_bfloat16, 128>(c, st) : weigh_go<__nv_bfloat16, 64>(c, st);
  return c.hd == 128 ? weigh_go<float, 128>(c, st) : weigh_go<float, 64>(c, st);
}

}  // namespace sf
