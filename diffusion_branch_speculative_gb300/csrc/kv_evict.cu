// What stays in a paged cache, and closing its gaps: the choice of a sequence's
// tokens by their weights (specfold_kv_select) and the move of the kept ones to the
// front of its pages, in place (specfold_kv_compact).
#include "sf_device.cuh"
#include "sf_internal.h"

#include <algorithm>
#include <climits>

namespace sf {
namespace {

// ---------------------------------------------------------------- select --
struct SelectArgs {
  specfold_token_weights w;
  specfold_kept_tokens kept;
  const int32_t* lengths;
  int32_t* new_len;
  uint32_t* status;
  int keep, sinks, recent;
};

// Weights in their order as unsigned numbers: NaN below all, the zeros alike.
SF_DEV uint32_t weight_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (u << 1 > 0xff000000u) return 0u;
  if (u << 1 == 0u) u = 0u;
  return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kSelBits = 8, kSelBins = 1 << kSelBits;

// One block a (sequence, set).
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const __grid_constant__ SelectArgs p) {
  __shared__ int s_hist[kSelBins];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_warp[2][kSelWarps];
  pdl_wait();
  pdl_trigger();
  const int set = blockIdx.x % p.kept.n_sets, s = blockIdx.x / p.kept.n_sets;
  const int len = p.lengths[s];
  int32_t* out = p.kept.ptr + s * p.kept.seq_stride + set * p.kept.set_stride;
  if (len < 0 || len > p.w.tokens) {
    if (threadIdx.x == 0 && set == 0) {
      p.new_len[s] = -1;
      if (p.status) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
    }
    return;
  }
  if (threadIdx.x == 0 && set == 0) p.new_len[s] = min(len, p.keep);
  if (len <= p.keep) {
    for (int i = threadIdx.x; i < len; i += kSelThreads) out[i] = i;
    return;
  }
  const float* w = p.w.ptr + s * p.w.seq_stride + set * p.w.head_stride;
  // of the tokens [lo, hi) the `need` largest; there are more
  const int lo = p.sinks, hi = len - p.recent, need = p.keep - p.sinks - p.recent;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < lo; i += kSelThreads) out[i] = i;
  for (int i = threadIdx.x; i < p.recent; i += kSelThreads) out[lo + need + i] = hi + i;
  if (need == 0) return;
  // the need-th largest key, from its upper bits down
  uint32_t prefix = 0u;
  int rest = need;
  for (int shift = 32 - kSelBits; shift >= 0; shift -= kSelBits) {
    for (int i = threadIdx.x; i < kSelBins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = lo + threadIdx.x; i < hi; i += kSelThreads) {
      const uint32_t k = weight_key(w[i]);
      if (shift == 32 - kSelBits || k >> (shift + kSelBits) == prefix) atomicAdd(&s_hist[(k >> shift) & (kSelBins - 1)], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int b = kSelBins - 1, left = rest;
      while (s_hist[b] < left) left -= s_hist[b--];
      s_prefix = prefix << kSelBits | static_cast<uint32_t>(b);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    rest = s_need;
  }
  // ascending: all above the key, and the first `rest` equal to it
  int before = 0, equal = 0;
  for (int base = lo; base < hi; base += kSelThreads) {
    const int i = base + threadIdx.x;
    const uint32_t k = i < hi ? weight_key(w[i]) : 0u;
    const bool gt = i < hi && k > prefix, eq = i < hi && k == prefix;
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) {
      s_warp[0][warp] = __popc(mg);
      s_warp[1][warp] = __popc(me);
    }
    __syncthreads();
    int g = before, e = equal;
    for (int k2 = 0; k2 < kSelWarps; ++k2) {
      if (k2 == warp) {
        const int at_e = e + __popc(me & ((1u << lane) - 1u)), at_g = g + __popc(mg & ((1u << lane) - 1u));
        if (gt || (eq && at_e < rest)) out[lo + at_g + min(at_e, rest)] = i;
      }
      g += s_warp[0][k2];
      e += s_warp[1][k2];
    }
    before = g;
    equal = e;
  }
}

// --------------------------------------------------------------- compact --
struct CompactArgs {
  specfold_paged_cache cache;
  specfold_kept_tokens kept;
  specfold_token_weights w;
  const int32_t* lengths;
  const int32_t* new_len;
  uint32_t* status;
  int n_kv, row16;  // 16-byte pieces of a row
};

constexpr int kMoveThreads = 256;

// One block a (sequence, head, keys or values).  kept ascends strictly, so that
// kept[i] >= i: a chunk's tokens, read before any of them is written, are never a
// later chunk's destinations' sources that are gone.
__global__ void __launch_bounds__(kMoveThreads) kv_compact_kernel(const __grid_constant__ CompactArgs p) {
  constexpr int CH = 64;  // tokens of a chunk
  __shared__ int s_from[CH], s_to[CH], s_stop;
  __shared__ float s_w[CH];
  pdl_wait();
  pdl_trigger();
  const bool is_v = blockIdx.x & 1;
  const int h = (blockIdx.x >> 1) % p.n_kv, s = (blockIdx.x >> 1) / p.n_kv;
  const int len = p.lengths[s], n = p.new_len[s];
  const bool weights = p.w.ptr && !is_v && h < p.kept.n_sets;
  const bool reports = p.status && threadIdx.x == 0;
  if (n < 0 || n > len || n > p.kept.cap || (p.w.ptr && len > p.w.tokens)) {
    if (reports) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
    return;
  }
  if (n == len) return;
  const int set = p.kept.n_sets == 1 ? 0 : h;
  const int32_t* kept = p.kept.ptr + s * p.kept.seq_stride + set * p.kept.set_stride;
  const specfold_paged_cache& c = p.cache;
  const int32_t* table = c.block_table + s * c.table_stride;
  float* w = weights ? p.w.ptr + s * p.w.seq_stride + h * p.w.head_stride : nullptr;
  const int bytes = p.row16 * 16;
  (void)bytes;
  uint4* pool = reinterpret_cast<uint4*>(is_v ? c.v : c.k);
  const int e16 = p.row16;  // pieces of a row; strides in pieces come with the call
  const long long ts = is_v ? c.v_token_stride : c.k_token_stride, hs = is_v ? c.v_head_stride : c.k_head_stride;
  pool += h * hs;
  auto slot = [&](int tok) {
    const unsigned pg = static_cast<unsigned>(tok) / static_cast<unsigned>(c.page_size);
    if (pg < static_cast<unsigned>(c.table_pages)) {
      const int page = table[pg];
      if (page >= 0 && page < c.num_pages) return page * c.page_size + (tok - static_cast<int>(pg) * c.page_size);
    }
    if (p.status) atomicOr(p.status, SPECFOLD_DEV_BAD_PAGE);
    return -1;
  };
  for (int i0 = 0; i0 < n; i0 += CH) {
    const int m = min(CH, n - i0);
    __syncthreads();
    if (threadIdx.x == 0) s_stop = m;
    __syncthreads();
    if (threadIdx.x < m) {
      const int i = i0 + threadIdx.x, src = kept[i], last = i > 0 ? kept[i - 1] : -1;
      const bool good = src > last && src < len && last >= i - 1;
      if (!good) atomicMin(&s_stop, static_cast<int>(threadIdx.x));
      s_to[threadIdx.x] = s_from[threadIdx.x] = -1;
      if (good && src != i) {
        const int a = slot(i), b = slot(src);
        s_to[threadIdx.x] = b < 0 ? -1 : a;
        s_from[threadIdx.x] = b;
        if (w) s_w[threadIdx.x] = w[src];
      }
    }
    __syncthreads();
    const int stop = s_stop;
    constexpr int MOST = CH * 32 / kMoveThreads;  // pieces a thread: rows of at most 512 bytes
    uint4 v[MOST];
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      const int x = threadIdx.x + k * kMoveThreads, t = x / e16;
      if (t < stop && s_to[t] >= 0) v[k] = pool[s_from[t] * ts + x % e16];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      const int x = threadIdx.x + k * kMoveThreads, t = x / e16;
      if (t < stop && s_to[t] >= 0) pool[s_to[t] * ts + x % e16] = v[k];
    }
    if (w && threadIdx.x < stop) {
      const int i = i0 + threadIdx.x;
      if (kept[i] != i) w[i] = s_w[threadIdx.x];
    }
    if (stop < m) {
      if (reports) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
      return;
    }
  }
}

}  // namespace

int launch_kv_select(const KvSelectCall& c, cudaStream_t st) {
  SelectArgs a{c.w, c.kept, c.lengths, c.new_len, c.status, c.keep, c.sinks, c.recent};
  launch_k(kv_select_kernel, dim3(c.n_seqs * c.kept.n_sets), dim3(kSelThreads), 0, st, a);
  count_launch();
  return check_launch();
}

int launch_kv_compact(const KvCompactCall& c, cudaStream_t st) {
  CompactArgs a{c.cache, c.kept, c.w, c.lengths, c.new_len, c.status, c.n_kv, 0};
  const int e = c.dtype == SPECFOLD_BF16 ? 2 : 4;
  a.row16 = c.hd * e / 16;
  // strides in 16-byte pieces (they are multiples of 8 elements)
  for (int64_t* x : {&a.cache.k_token_stride, &a.cache.k_head_stride, &a.cache.v_token_stride, &a.cache.v_head_stride})
    *x = *x * e / 16;
  launch_k(kv_compact_kernel, dim3(2 * c.n_seqs * c.n_kv), dim3(kMoveThreads), 0, st, a);
  count_launch();
  return check_launch();
}

}  // namespace sf
