// What stays in a paged cache, and closing its gaps: the choice of a sequence's
// tokens by their weights (specfold_kv_select) and the move of the kept ones to the
// front of its pages, in place (specfold_kv_compact).
#include "sf_device.cuh"
#include "sf_internal.h"

#include <algorithm>
#include <type_traits>

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
constexpr int kSelGroups = kSelBins / 32;
constexpr int kSelCap = 48 * 1024;       // keys of a block's slice that shared memory holds (longer ones are read each pass)
constexpr int kSelMaxCluster = 8;
constexpr int kSelSlice = 4096;          // tokens that are worth a block more
constexpr int kSelStep = 1024;           // keys of a warp's step, 32 a lane

SF_DEV void st_dsmem_s32(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Two of 64 counts a lane (h.x, h.y: those at 62 - 2 lane and 63 - 2 lane): the place, from the
// last down, of the one with the left-th; left: which of its own that is.
SF_DEV int find_from_last(int2 h, int lane, int& left) {
  int upto = h.x + h.y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, upto >= left)) - 1;
  const int in = left - (upto - h.x - h.y);  // less those above these two
  const bool upper = in <= h.y;
  left = __shfl_sync(0xffffffffu, upper ? in : in - h.y, src);
  return __shfl_sync(0xffffffffu, 62 - 2 * lane + (upper ? 1 : 0), src);
}

// One cluster a (sequence, set); its blocks have a slice each of the tokens between
// the first and the latest ones, its keys in shared memory.  Three passes find the
// smallest chosen key by its digits: a histogram a block, added up over the cluster
// in two steps, the groups of 32 bins and then the bins of one, which the blocks write
// to each other (reading all bins of eight blocks took 2 to 5 us a pass, reading
// groups and bins 4).  Then every warp writes what it has of its run of the slice, behind
// what lies before.  Latency bounds it: the chain of reads, passes and exchanges.  3
// sequences of up to 131071 tokens and 8 sets, 10 MB, take 18.9 us (21 cold), 64 of 8192
// 16.2, 64 of 2080 9.4, one of 2080 8.4 with the call, where the bytes need 1.5, 2.4, 0.9
// and 0.01.  Those weights spread over some twenty octaves; where they meet in few bins
// the counting waits: 64 of 8192 within three octaves 17.6, within one bin of the first
// pass 18.1, all equal 20.5; 64 of 60000 102, 119, 122, 145.  1024 threads were slower
// with eight blocks a cluster; 32 registers a thread (a block alone spills 4 bytes) let an
// SM have four blocks (64 x 8192: 16.0 us, 17.5 with three).
template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, 4) kv_select_kernel(const __grid_constant__ SelectArgs p) {
  extern __shared__ __align__(16) uint32_t s_key[];
  __shared__ int s_hist[2][kSelBins];
  __shared__ __align__(8) int s_group[2][kSelMaxCluster][kSelGroups];  // the blocks' sums of this pass
  __shared__ int s_bin[2][kSelMaxCluster][32];                         // and their bins of the group found
  __shared__ int s_warp[kSelWarps][2], s_found[3], s_total[kSelMaxCluster][2];
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
  const int slice = (hi - lo - 1) / blocks / kSelStep * kSelStep + kSelStep;
  const int from = min(static_cast<long long>(hi), lo + static_cast<long long>(rank) * slice);
  const int n = min(hi - from, slice);  // this block's (none, for some, of a short sequence)
  const float* w = p.w.ptr + s * p.w.seq_stride + set * p.w.head_stride + from;
  auto all_sync = [] {
    if constexpr (CLUSTER)
      cluster_sync_all();
    else
      __syncthreads();
  };
  // v to all blocks' copies of a place in shared memory, a lane a block
  auto tell = [&](int* at, int v) {
    if constexpr (CLUSTER) {
      if (lane < blocks) st_dsmem_s32(dsmem_addr(smem_u32(at), lane), v);
    } else {
      if (lane == 0) *at = v;
    }
  };
  for (int i = threadIdx.x; i < kSelBins; i += kSelThreads) s_hist[0][i] = s_hist[1][i] = 0;
  all_sync();  // (and the cluster's blocks have all begun)
  auto choose = [&](auto held) {
    constexpr bool kHeld = decltype(held)::value;
    // Keys in pieces of four, piece c of eight at c ^ (the eight's number mod 8): a warp reads
    // 32 pieces side by side or eight apart without conflicts.  Zeros past the end.
    auto place = [](int i) { return i ^ ((i >> 5 & 7) << 2); };
    auto keys = [&](int i, uint32_t (&k)[4]) {  // held: i .. i + 3, i a multiple of four
      const uint4 u = *reinterpret_cast<const uint4*>(s_key + place(i));
      k[0] = u.x, k[1] = u.y, k[2] = u.z, k[3] = u.w;
    };
    // the keys, and the first pass
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      const uint32_t k = weight_key(w[i]);
      if constexpr (kHeld) s_key[place(i)] = k;
      atomicAdd(&s_hist[0][k >> 21], 1);
    }
    if constexpr (kHeld) {
      for (int i = max(n, 0) + threadIdx.x; i < (max(n, 0) + kSelStep - 1) / kSelStep * kSelStep; i += kSelThreads) s_key[place(i)] = 0u;
    }
    uint32_t prefix = 0u;
    int rest = need, shift = 21;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      int* hist = s_hist[pass & 1];
      __syncthreads();
      for (int g = warp; g < kSelGroups; g += kSelWarps)
        tell(&s_group[pass & 1][rank][g], __reduce_add_sync(0xffffffffu, hist[g * 32 + lane]));
      all_sync();
      int left = rest, group = 0;
      if (warp == 0) {
        int2 h = make_int2(0, 0);
        for (int k = 0; k < blocks; ++k) {
          const int2 x = *reinterpret_cast<const int2*>(&s_group[pass & 1][k][62 - 2 * lane]);
          h = make_int2(h.x + x.x, h.y + x.y);
        }
        group = find_from_last(h, lane, left);
        const int mine = hist[group * 32 + lane];
        if constexpr (CLUSTER) {
          for (int k = 0; k < blocks; ++k) st_dsmem_s32(dsmem_addr(smem_u32(&s_bin[pass & 1][rank][lane]), k), mine);
        } else {
          s_bin[pass & 1][0][lane] = mine;
        }
      }
      all_sync();
      if (warp == 0) {
        // the group's bins as the upper 32 of 64, two a lane
        int2 h = make_int2(0, 0);
        if (lane < 16)
          for (int k = 0; k < blocks; ++k) {
            h.x += s_bin[pass & 1][k][30 - 2 * lane];
            h.y += s_bin[pass & 1][k][31 - 2 * lane];
          }
        const int digit = find_from_last(h, lane, left) - 32;
        const int count = __shfl_sync(0xffffffffu, digit & 1 ? h.y : h.x, (31 - digit) / 2);
        if (lane == 0) {
          s_found[0] = group * 32 + digit;
          s_found[1] = left;
          s_found[2] = count;
        }
      }
      __syncthreads();
      const int digit = s_found[0], count = s_found[2];
      rest = s_found[1];
      prefix = pass == 0 ? digit : prefix << (pass == 1 ? 11 : 10) | static_cast<uint32_t>(digit);
      if (pass == 2 || count == rest) break;  // (all of that bin: no further digit counts)
      const int next = pass == 0 ? 10 : 0;
      const uint32_t mask = pass == 0 ? 2047u : 1023u;
      int* to = s_hist[(pass + 1) & 1];
      if (pass == 1) {  // the first pass's
        for (int i = threadIdx.x; i < kSelBins; i += kSelThreads) to[i] = 0;
        __syncthreads();
      }
      if constexpr (kHeld) {
#pragma unroll 2
        for (int i = 4 * threadIdx.x; i < n; i += 4 * kSelThreads) {
          uint32_t k[4];
          keys(i, k);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (k[j] >> shift == prefix && i + j < n) atomicAdd(&to[(k[j] >> next) & mask], 1);
        }
      } else {
#pragma unroll 8
        for (int i = threadIdx.x; i < n; i += kSelThreads) {
          const uint32_t k = weight_key(w[i]);
          if (k >> shift == prefix) atomicAdd(&to[(k >> next) & mask], 1);
        }
      }
      shift = next;
    }
    // ascending: all above the digits found, and the first `rest` of those that have them.
    // A warp has a run of steps of 1024 keys, a lane 32 of them side by side.
    const int steps = max(0, n + kSelStep - 1) / kSelStep, run = (steps + kSelWarps - 1) / kSelWarps;
    const int st0 = min(steps, warp * run), st1 = min(steps, st0 + run);
    uint32_t gt = 0u, eq = 0u;  // of the lane's keys in a step
    auto marks = [&](int st) {
      gt = eq = 0u;
      const int i = st * kSelStep + 32 * lane;
      if constexpr (kHeld) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t k[4];
          keys(i + 4 * c, k);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            gt |= (k[j] >> shift > prefix ? 1u : 0u) << (4 * c + j);
            eq |= (k[j] >> shift == prefix ? 1u : 0u) << (4 * c + j);
          }
        }
      } else {  // read side by side, a word of marks a lane
#pragma unroll 8
        for (int c = 0; c < 32; ++c) {
          const int at = st * kSelStep + 32 * c + lane;
          const uint32_t k = at < n ? weight_key(w[at]) : 0u;
          const uint32_t g = __ballot_sync(0xffffffffu, k >> shift > prefix), e = __ballot_sync(0xffffffffu, k >> shift == prefix);
          if (lane == c) gt = g, eq = e;
        }
      }
      const int there = n - i;  // (what lies past the end is a key of zero)
      if (there < 32) eq &= there <= 0 ? 0u : (1u << there) - 1u;
    };
    int above = 0, equal = 0;
    for (int st = st0; st < st1; ++st) {
      marks(st);
      above += __popc(gt);
      equal += __popc(eq);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
      s_warp[warp][0] = above;
      s_warp[warp][1] = equal;
    }
    __syncthreads();
    int b0 = lane < kSelWarps ? s_warp[lane][0] : 0, b1 = lane < kSelWarps ? s_warp[lane][1] : 0;
    if constexpr (CLUSTER) {
      const int t0 = __reduce_add_sync(0xffffffffu, b0), t1 = __reduce_add_sync(0xffffffffu, b1);
      if (warp == 0) {
        tell(&s_total[rank][0], t0);
        tell(&s_total[rank][1], t1);
      }
      cluster_sync_all();  // the last exchange: a block may end from here on
    }
    b0 = __reduce_add_sync(0xffffffffu, lane < warp ? b0 : 0);
    b1 = __reduce_add_sync(0xffffffffu, lane < warp ? b1 : 0);
    if constexpr (CLUSTER) {  // the blocks before
      b0 += __reduce_add_sync(0xffffffffu, lane < rank ? s_total[lane][0] : 0);
      b1 += __reduce_add_sync(0xffffffffu, lane < rank ? s_total[lane][1] : 0);
    }
    for (int st = st0; st < st1; ++st) {
      if (run > 1) marks(st);
      const int mine = __popc(gt) + (__popc(eq) << 16);
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
      }
      const int g = b0 + ((upto - mine) & 0xffff), e = b1 + ((upto - mine) >> 16);
      for (uint32_t m = gt | eq; m; m &= m - 1u) {
        const int bit = __ffs(m) - 1;
        const uint32_t below = (1u << bit) - 1u;
        const int at_e = e + __popc(eq & below);
        if ((gt >> bit & 1u) || at_e < rest) out[lo + g + __popc(gt & below) + min(at_e, rest)] = from + st * kSelStep + 32 * lane + bit;
      }
      upto = __shfl_sync(0xffffffffu, upto, 31);
      b0 += upto & 0xffff;
      b1 += upto >> 16;
    }
  };
  if (slice <= p.held)  // the same in all of the cluster
    choose(std::true_type{});
  else
    choose(std::false_type{});
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

constexpr int kMoveRow = 8;  // 16-byte pieces of a slice
template <bool CLUSTER>
struct Move {
  static constexpr int THREADS = CLUSTER ? 256 : 128;
  static constexpr int PIECES = 4;                                   // a thread and round
  static constexpr int TOKENS = THREADS * PIECES / kMoveRow;         // of a block's round
};

// One cluster a (sequence, head, keys or values, slice of the row).  In a round each
// block has a run of destinations: all sources of a round are read before any of its
// destinations is written.  An entry is no less than its own index, so a later round
// reads nothing that an earlier one has written.  Slices of 128 bytes, not whole rows,
// for more streams and shorter rounds.  Where a cache loses a few tokens, a move is a copy:
// 64 sequences of up to 2080 tokens, 4 heads of 128, 543 MB in 92.7 us, 5860 GB/s, 0.87 of the
// copy rate.  Where prompts lose most, the sources are single rows far apart: 3 prompts
// of up to 32700 tokens to 4096, 8 heads, 102 MB in
// 24.2 us, 4200 GB/s, DRAM 35 % busy; 8 pieces a thread, 512 threads and slices of 256
// bytes are no faster.  Few long streams pay their rounds: 16000 of 32700 tokens of one
// sequence of 4 heads take 39.8 us where the bytes need 9.8.
template <bool CLUSTER>
__global__ void __launch_bounds__(Move<CLUSTER>::THREADS) kv_compact_kernel(const __grid_constant__ CompactArgs p) {
  constexpr int THREADS = Move<CLUSTER>::THREADS, PIECES = Move<CLUSTER>::PIECES, TOKENS = Move<CLUSTER>::TOKENS;
  constexpr int WEIGHTS = (TOKENS + THREADS - 1) / THREADS;  // a thread and round
  __shared__ int s_at[2][2][TOKENS];  // [round][source, destination]
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
  const int mine = threadIdx.x / kMoveRow;  // and every THREADS / kMoveRow-th token behind it
  // a round's pool tokens, -1 for a token that stays
  auto locate = [&](int first, int buf) {
#pragma unroll
    for (int x = threadIdx.x; x < 2 * TOKENS; x += THREADS) {
      const bool dest = x >= TOKENS;
      const int token = x % TOKENS, i = first + token;
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
      s_at[buf][dest][token] = at;
    }
  };
  const int step = blocks * TOKENS;
  locate(rank * TOKENS, 0);
  __syncthreads();
  int buf = 0;
  for (int first = rank * TOKENS, round0 = 0; round0 < n; round0 += step, first += step, buf ^= 1) {
    uint4 v[PIECES];
    int to[PIECES];
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      const int t = mine + k * (THREADS / kMoveRow), from = s_at[buf][0][t];
      to[k] = from < 0 ? -1 : s_at[buf][1][t];
      if (to[k] >= 0) v[k] = pool[from * ts];
    }
    float moved[WEIGHTS];
    bool moves[WEIGHTS];
#pragma unroll
    for (int k = 0; k < WEIGHTS; ++k) {
      // a token's weight goes where its keys and values go: one that stays keeps its own
      const int token = threadIdx.x + k * THREADS;
      moves[k] = w && token < TOKENS && s_at[buf][0][token] >= 0 && s_at[buf][1][token] >= 0;
      if (moves[k]) moved[k] = w[kept[first + token]];
    }
    if (round0 + step < n) locate(first + step, buf ^ 1);
    if constexpr (CLUSTER)
      cluster_sync_all();
    else
      __syncthreads();
#pragma unroll
    for (int k = 0; k < PIECES; ++k)
      if (to[k] >= 0) pool[to[k] * ts] = v[k];
#pragma unroll
    for (int k = 0; k < WEIGHTS; ++k)
      if (moves[k]) w[first + threadIdx.x + k * THREADS] = moved[k];
  }
}

}  // namespace

int launch_kv_select(const KvSelectCall& c, cudaStream_t st) {
  SelectArgs a{c.w, c.kept, c.lengths, c.new_len, c.status, c.keep, c.sinks, c.recent, 1, 0};
  // Blocks a cluster: more while slices are of some length and either the blocks are no more
  // than the SMs or a slice's keys leave an SM no second block (64 sequences of 60000 tokens and
  // 8 sets: 109 us with slices of 15000, 123 with 7500, 127 with 30000, 184 with one block a unit,
  // which cannot hold its keys; 32 of 120000: 116 with slices of 15000, 263 with one block).
  // The rule knows the room of the weights, not the lengths: with room for four times as many
  // tokens 64 of 8192 take 40 us, not 16.2, 64 of 60000 356, not 102, 3 of 131071 24.5, not 19.2,
  // one of 2080 11.5, not 8.6.
  const long long units = static_cast<long long>(c.n_seqs) * c.kept.n_sets;
  while (a.blocks < kSelMaxCluster && c.w.tokens / a.blocks > kSelSlice &&
         (units * a.blocks * 2 <= 2LL * num_sms() || c.w.tokens / a.blocks > kSelCap / 2))
    a.blocks *= 2;
  const int slice = (c.w.tokens - 1) / a.blocks / kSelStep * kSelStep + kSelStep;
  a.held = slice < kSelCap ? slice : kSelCap;
  const int smem = a.held * 4;
  auto kernel = a.blocks > 1 ? kv_select_kernel<true> : kv_select_kernel<false>;
  if (const int rc = smem_limit_once(kernel, kSelCap * 4)) return rc;
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
  while (a.blocks < 8 && a.blocks * Move<true>::TOKENS < c.kept.cap && units * a.blocks < 5LL * num_sms()) a.blocks *= 2;
  const dim3 grid(static_cast<unsigned>(units * a.blocks));
  if (a.blocks > 1)
    launch_kc(kv_compact_kernel<true>, grid, dim3(Move<true>::THREADS), 0, st, a.blocks, a);
  else
    launch_k(kv_compact_kernel<false>, grid, dim3(Move<false>::THREADS), 0, st, a);
  count_launch();
  return check_launch();
}

}  // namespace sf
