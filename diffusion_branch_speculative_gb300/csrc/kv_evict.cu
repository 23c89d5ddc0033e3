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
  int blocks, held;  // blocks of a cluster; keys of a slice that shared memory holds
};

// Weights in their order as unsigned numbers: NaN below all, the zeros alike.
SF_DEV uint32_t weight_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (u << 1 > 0xff000000u) return 0u;
  if (u << 1 == 0u) u = 0u;
  return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;           // of a pass over 11, 11 and 10 bits of the keys
constexpr int kSelCap = 48 * 1024;       // keys of a block's slice that shared memory holds
constexpr int kSelMaxCluster = 8;
constexpr int kSelSlice = 4096;          // tokens that are worth a block more

SF_DEV int ld_dsmem_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
SF_DEV int4 ld_dsmem_s32x4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// One cluster a (sequence, set); its blocks have a slice each of the tokens between
// the first and the latest ones, its keys in shared memory.  Three passes find the
// smallest chosen key by its digits (a histogram a block, added up over the cluster),
// then every warp writes what it has of its run of the slice, behind what lies before.
template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const __grid_constant__ SelectArgs p) {
  extern __shared__ uint32_t s_key[];
  __shared__ __align__(16) int s_hist[3][kSelBins];  // a pass each: read by the cluster while the next is filled
  __shared__ int s_warp[2][kSelWarps], s_found[3], s_total[2];
  pdl_wait();
  pdl_trigger();
  const int blocks = CLUSTER ? p.blocks : 1, rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = static_cast<int>(blockIdx.x) / blocks;
  const int set = unit % p.kept.n_sets, s = unit / p.kept.n_sets;
  const int len = p.lengths[s];
  int32_t* out = p.kept.ptr + s * p.kept.seq_stride + set * p.kept.set_stride;
  const bool tells = threadIdx.x == 0 && rank == 0 && set == 0;
  const int tid = rank * kSelThreads + threadIdx.x, threads = blocks * kSelThreads;  // of the cluster
  if (len < 0 || len > p.w.tokens) {
    if (tells) {
      p.new_len[s] = -1;
      if (p.status) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
    }
    return;
  }
  if (tells) p.new_len[s] = min(len, p.keep);
  if (len <= p.keep) {
    for (int i = tid; i < len; i += threads) out[i] = i;
    return;
  }
  // of the tokens [lo, hi) the `need` largest; there are more
  const int lo = p.sinks, hi = len - p.recent, need = p.keep - p.sinks - p.recent;
  for (int i = tid; i < lo; i += threads) out[i] = i;
  for (int i = tid; i < p.recent; i += threads) out[lo + need + i] = hi + i;
  if (need == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = ((hi - lo - 1) / blocks + 1 + 31) & ~31;
  const int from = min(hi, lo + rank * slice), n = min(hi - from, slice);  // this block's
  const float* w = p.w.ptr + s * p.w.seq_stride + set * p.w.head_stride + from;
  const bool held = n <= p.held;
  auto all_sync = [] {
    if constexpr (CLUSTER)
      cluster_sync_all();
    else
      __syncthreads();
  };
  for (int i = threadIdx.x; i < 3 * kSelBins; i += kSelThreads) (&s_hist[0][0])[i] = 0;
  __syncthreads();
  // the keys, and the first pass
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const uint32_t k = weight_key(w[i]);
    if (held) s_key[i] = k;
    atomicAdd(&s_hist[0][k >> 21], 1);
  }
  auto key = [&](int i) { return held ? s_key[i] : weight_key(w[i]); };
  uint32_t prefix = 0u;
  int rest = need, shift = 21;
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    all_sync();
    // bins from the largest down, four a thread: the one with the rest-th key
    static_assert(kSelBins == 4 * kSelThreads, "four bins a thread");
    const int bin = kSelBins - 4 - 4 * static_cast<int>(threadIdx.x);
    int4 h;
    if constexpr (CLUSTER) {
      const uint32_t at = smem_u32(&s_hist[pass][bin]);
      h = make_int4(0, 0, 0, 0);
#pragma unroll
      for (int k0 = 0; k0 < kSelMaxCluster; k0 += 4) {
        int4 x[4];  // four asked for before any is added
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = k0 + k < blocks ? ld_dsmem_s32x4(dsmem_addr(at, k0 + k)) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) h = make_int4(h.x + x[k].x, h.y + x[k].y, h.z + x[k].z, h.w + x[k].w);
      }
    } else {
      h = *reinterpret_cast<const int4*>(&s_hist[pass][bin]);
    }
    int upto = (h.x + h.y) + (h.z + h.w);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    if (lane == 31) s_warp[0][warp] = upto;
    __syncthreads();
    int before = lane < warp ? s_warp[0][lane] : 0;
    before = __reduce_add_sync(0xffffffffu, before);
    upto += before;
    int left = rest - (upto - (h.x + h.y) - (h.z + h.w));  // less the keys above these bins
    if (left > 0 && rest <= upto) {
      const int have[4] = {h.w, h.z, h.y, h.x};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (left > 0 && left <= have[k]) {
          s_found[0] = bin + 3 - k;
          s_found[1] = left;
          s_found[2] = have[k];
        }
        left -= have[k];
      }
    }
    __syncthreads();
    const int digit = s_found[0], count = s_found[2];
    rest = s_found[1];
    prefix = pass == 0 ? digit : prefix << (pass == 1 ? 11 : 10) | static_cast<uint32_t>(digit);
    if (pass == 2 || count == rest) break;  // (all of that bin: no further digit counts)
    const int next = pass == 0 ? 10 : 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      const uint32_t k = key(i);
      if (k >> shift == prefix) atomicAdd(&s_hist[pass + 1][(k >> next) & (pass == 0 ? 2047u : 1023u)], 1);
    }
    shift = next;
  }
  // ascending: all above the digits found, and the first `rest` of those that have them
  const int run = (slice / 32 + kSelWarps - 1) / kSelWarps * 32, i0 = warp * run, i1 = min(n, i0 + run);
  int above = 0, equal = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = key(i) >> shift;
    above += k > prefix;
    equal += k == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    s_warp[0][warp] = above;  // (pass's own values have been read, see its last barrier)
    s_warp[1][warp] = equal;
  }
  __syncthreads();
  int b0 = lane < kSelWarps ? s_warp[0][lane] : 0, b1 = lane < kSelWarps ? s_warp[1][lane] : 0;
  if constexpr (CLUSTER) {
    const int t0 = __reduce_add_sync(0xffffffffu, b0), t1 = __reduce_add_sync(0xffffffffu, b1);
    if (threadIdx.x == 0) {
      s_total[0] = t0;
      s_total[1] = t1;
    }
    cluster_sync_all();
  }
  b0 = __reduce_add_sync(0xffffffffu, lane < warp ? b0 : 0);
  b1 = __reduce_add_sync(0xffffffffu, lane < warp ? b1 : 0);
  if constexpr (CLUSTER) {
    int c0 = 0, c1 = 0;
    if (lane < rank) {  // the blocks before
      c0 = ld_dsmem_s32(dsmem_addr(smem_u32(&s_total[0]), lane));
      c1 = ld_dsmem_s32(dsmem_addr(smem_u32(&s_total[1]), lane));
    }
    b0 += __reduce_add_sync(0xffffffffu, c0);
    b1 += __reduce_add_sync(0xffffffffu, c1);
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i = i0; i < i1; i += 32) {
    const bool there = i + lane < i1;
    const uint32_t k = there ? key(i + lane) >> shift : 0u;
    const bool gt = there && k > prefix, eq = there && k == prefix;
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    const int at_e = b1 + __popc(me & below);
    if (gt || (eq && at_e < rest)) out[lo + b0 + __popc(mg & below) + min(at_e, rest)] = from + i + lane;
    b0 += __popc(mg);
    b1 += __popc(me);
  }
  if constexpr (CLUSTER) cluster_sync_all();  // no block ends while another reads its shared memory
}

// --------------------------------------------------------------- compact --
struct CompactArgs {
  specfold_paged_cache cache;  // strides in 16-byte pieces
  specfold_kept_tokens kept;
  specfold_token_weights w;
  const int32_t* lengths;
  const int32_t* new_len;
  uint32_t* status;
  int n_kv, slices, blocks;  // 128-byte slices of a row, blocks of a cluster
};

constexpr int kMovePieces = 4;  // of 16 bytes, a thread and round
constexpr int kMoveRow = 8;     // of a slice
constexpr int move_tokens(int threads) { return threads * kMovePieces / kMoveRow; }  // of a block's round
constexpr int kMoveAlone = 128, kMoveCluster = 256;  // threads of a block

// One cluster a (sequence, head, keys or values, slice of the row).  In a round each
// block has a run of destinations: all sources of a round are read before any of its
// destinations is written.  An entry is no less than its own index, so a later round
// reads nothing that an earlier one has written.
template <int kMoveThreads, bool CLUSTER>
__global__ void __launch_bounds__(kMoveThreads) kv_compact_kernel(const __grid_constant__ CompactArgs p) {
  constexpr int kMoveTokens = move_tokens(kMoveThreads);
  static_assert(2 * kMoveTokens <= kMoveThreads, "a thread a source and a destination");
  __shared__ int s_from[2][kMoveTokens], s_to[2][kMoveTokens];
  pdl_wait();
  pdl_trigger();
  const int blocks = CLUSTER ? p.blocks : 1, rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  int unit = static_cast<int>(blockIdx.x) / blocks;
  const int slice = unit % p.slices;
  unit /= p.slices;
  const bool is_v = unit & 1;
  unit >>= 1;
  const int h = unit % p.n_kv, s = unit / p.n_kv;
  const int len = p.lengths[s], n = p.new_len[s];
  const bool tells = p.status && slice == 0 && !is_v;
  if (n < 0 || n > len || n > p.kept.cap || (p.w.ptr && len > p.w.tokens)) {
    if (tells && threadIdx.x == 0) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
    return;
  }
  if (n == len) return;
  const int32_t* kept = p.kept.ptr + s * p.kept.seq_stride + (p.kept.n_sets == 1 ? 0 : h) * p.kept.set_stride;
  const specfold_paged_cache& c = p.cache;
  const int32_t* table = c.block_table + s * c.table_stride;
  const bool weighs = p.w.ptr && slice == 0 && !is_v && h < p.kept.n_sets;
  float* w = weighs ? p.w.ptr + s * p.w.seq_stride + h * p.w.head_stride : nullptr;
  uint4* pool = reinterpret_cast<uint4*>(is_v ? c.v : c.k) + h * (is_v ? c.v_head_stride : c.k_head_stride) +
                slice * kMoveRow + threadIdx.x % kMoveRow;
  const long long ts = is_v ? c.v_token_stride : c.k_token_stride;
  const int mine = threadIdx.x / kMoveRow;  // and every kMoveThreads / kMoveRow-th token behind it
  const bool dest = threadIdx.x >= kMoveTokens;
  const int token = threadIdx.x % kMoveTokens;
  // a round's pool tokens: the sources by the first threads, the destinations by the others
  auto locate = [&](int first, int buf) {
    if (threadIdx.x >= 2 * kMoveTokens) return;
    const int i = first + token;
    int at = -1;
    if (i < n) {
      const int src = kept[i];
      const bool good = src >= i && src < len;
      if (!good && tells) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
      if (good && src != i) {
        const int tok = dest ? i : src;
        const unsigned pg = static_cast<unsigned>(tok) / static_cast<unsigned>(c.page_size);
        int page = -1;
        if (pg < static_cast<unsigned>(c.table_pages)) page = table[pg];
        if (page >= 0 && page < c.num_pages)
          at = page * c.page_size + (tok - static_cast<int>(pg) * c.page_size);
        else if (tells)
          atomicOr(p.status, SPECFOLD_DEV_BAD_PAGE);
      }
    }
    (dest ? s_to : s_from)[buf][token] = at;
  };
  const int step = blocks * kMoveTokens;
  locate(rank * kMoveTokens, 0);
  __syncthreads();
  int buf = 0;
  for (int first = rank * kMoveTokens, round0 = 0; round0 < n; round0 += step, first += step, buf ^= 1) {
    uint4 v[kMovePieces];
    int to[kMovePieces];
#pragma unroll
    for (int k = 0; k < kMovePieces; ++k) {
      const int t = mine + k * (kMoveThreads / kMoveRow), from = s_from[buf][t];
      to[k] = from < 0 ? -1 : s_to[buf][t];
      if (to[k] >= 0) v[k] = pool[from * ts];
    }
    float moved = 0.f;
    bool moves = false;
    if (w && threadIdx.x < kMoveTokens && first + token < n) {
      const int src = kept[first + token];
      moves = src > first + token && src < len;
      if (moves) moved = w[src];
    }
    if (round0 + step < n) locate(first + step, buf ^ 1);
    if constexpr (CLUSTER)
      cluster_sync_all();
    else
      __syncthreads();
#pragma unroll
    for (int k = 0; k < kMovePieces; ++k)
      if (to[k] >= 0) pool[to[k] * ts] = v[k];
    if (moves) w[first + token] = moved;
  }
}

}  // namespace

int launch_kv_select(const KvSelectCall& c, cudaStream_t st) {
  SelectArgs a{c.w, c.kept, c.lengths, c.new_len, c.status, c.keep, c.sinks, c.recent, 1, 0};
  // Blocks a cluster: more while that leaves two a SM, and slices of some length.
  const long long units = static_cast<long long>(c.n_seqs) * c.kept.n_sets;
  while (a.blocks < kSelMaxCluster && c.w.tokens / a.blocks > kSelSlice && units * a.blocks * 2 <= 2LL * num_sms()) a.blocks *= 2;
  const int slice = ((c.w.tokens - 1) / a.blocks + 1 + 31) / 32 * 32;
  a.held = slice < kSelCap ? slice : kSelCap;
  const int smem = a.held * 4;
  auto kernel = a.blocks > 1 ? kv_select_kernel<true> : kv_select_kernel<false>;
  if (const int rc = smem_limit_once(kernel, kSelCap * 4)) return rc;
  if (units * a.blocks > 0x7fffffffLL) return SPECFOLD_ECAPACITY;
  const dim3 grid(static_cast<unsigned>(units * a.blocks));
  if (a.blocks > 1)
    launch_kc(kernel, grid, dim3(kSelThreads), smem, st, a.blocks, a);
  else
    launch_k(kernel, grid, dim3(kSelThreads), smem, st, a);
  count_launch();
  return check_launch();
}

int launch_kv_compact(const KvCompactCall& c, cudaStream_t st) {
  CompactArgs a{c.cache, c.kept, c.w, c.lengths, c.new_len, c.status, c.n_kv, 0, 1};
  const int e = c.dtype == SPECFOLD_BF16 ? 2 : 4;
  a.slices = c.hd * e / 128;
  // strides in 16-byte pieces (they are multiples of 8 elements)
  for (int64_t* x : {&a.cache.k_token_stride, &a.cache.k_head_stride, &a.cache.v_token_stride, &a.cache.v_head_stride})
    *x = *x * e / 16;
  const long long units = 2LL * c.n_seqs * c.n_kv * a.slices;
  while (a.blocks < 8 && a.blocks * move_tokens(kMoveCluster) < c.kept.cap && units * a.blocks < 5LL * num_sms()) a.blocks *= 2;
  if (units * a.blocks > 0x7fffffffLL) return SPECFOLD_ECAPACITY;
  const dim3 grid(static_cast<unsigned>(units * a.blocks));
  if (a.blocks > 1)
    launch_kc(kv_compact_kernel<kMoveCluster, true>, grid, dim3(kMoveCluster), 0, st, a.blocks, a);
  else
    launch_k(kv_compact_kernel<kMoveAlone, false>, grid, dim3(kMoveAlone), 0, st, a);
  count_launch();
  return check_launch();
}

}  // namespace sf
