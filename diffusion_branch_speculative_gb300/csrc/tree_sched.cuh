// The decomposition of a batch of tree attentions, shared by its kernels.
//
// A unit is (sequence, key/value head, tile of query rows) and its work the
// blocks of kb keys of that sequence.  All units' blocks in one line, sequence
// by sequence, head by head, tile by tile, are cut into equal runs, one per CTA:
// the lengths are known on the device only, and one rule serves a single long
// sequence and a ragged batch of short ones.  A run's piece that covers its
// whole unit writes the output; any other writes an unnormalised partial (o,
// running max m in log2 units, sum l), at most the run's first and last piece
// (slots 2c and 2c + 1 of CTA c), which the combine kernel merges in order, so
// results do not depend on timing.
#pragma once

#include "sf_device.cuh"
#include "sf_internal.h"

namespace sf {

struct TreeArgs {
  const void* q;
  void* o;
  long long q_rs, q_hs, o_rs, o_hs;
  specfold_paged_cache cache;
  const int32_t* parent;
  SeqBatch batch;
  int max_nodes, n_kv, g;
  int tile_rows;  // query rows of a tile: row m is node m / g, head m % g of the group
  int kb;         // keys per block
  float sl2;               // scale * log2(e)
  uint32_t* status;
  int4* desc;              // [2 * grid]: the unit cut at CTA c's start, see tree_describe
  float* part_o;           // [2 * grid][tile_rows][hd]
  float* part_ml;          // [2 * grid][tile_rows][2]
};

// One sequence: rows n behind ctx cached tokens, nb blocks of keys, tiles of
// query rows.  An invalid one has none.
struct TreeSeq {
  int row0, n, ctx, nb, tiles;
  bool bad;
  SF_DEV long long items(int n_kv) const { return static_cast<long long>(nb) * tiles * n_kv; }
};

// Weight of a partial with maximum m in a merge with maximum M: 1 where they
// are equal, -inf included (a partial that saw nothing holds zeros, and one
// whose scores are NaN keeps its NaN).
SF_DEV float merge_weight(float m, float M) { return m == M ? 1.f : ex2(m - M); }
// The factor of a row with sum l: zeros where nothing was seen.
SF_DEV float merge_scale(float l) { return l == 0.f ? 0.f : 1.f / l; }

SF_DEV TreeSeq tree_seq(const TreeArgs& p, int s) {
  TreeSeq q;
  q.row0 = p.batch.row_start[s];
  const int end = p.batch.row_start[s + 1];
  q.ctx = p.batch.ctx_len[s];
  q.bad = q.row0 < 0 || end < q.row0 || end > p.batch.T || end - q.row0 > p.max_nodes || q.ctx < 0 ||
          q.ctx > 0x7fffffff - 2 * SPECFOLD_MAX_TREE;
  q.n = q.bad ? 0 : end - q.row0;
  q.nb = q.n > 0 ? (q.ctx + q.n - 1) / p.kb + 1 : 0;
  q.tiles = (q.n * p.g + p.tile_rows - 1) / p.tile_rows;
  return q;
}

// A CTA's walk along its run: the current unit u (head u / tiles, tile u %
// tiles) of sequence s from block b0 on, `left` blocks to go.
struct TreeWalk {
  int s, u, b0;
  long long left;
  TreeSeq q;
  SF_DEV int head() const { return u / q.tiles; }
  SF_DEV int tile() const { return u % q.tiles; }
  SF_DEV int blocks() const {  // of the current piece
    const long long rest = q.nb - b0;
    return static_cast<int>(rest < left ? rest : left);
  }
  SF_DEV bool whole() const { return b0 == 0 && blocks() == q.nb; }
  SF_DEV void next(const TreeArgs& p) {
    left -= blocks();
    b0 = 0;
    if (++u < q.tiles * p.n_kv) return;
    u = 0;
    while (left > 0) {
      if (++s >= p.batch.n_seqs) {  // lengths that changed under the call
        left = 0;
        break;
      }
      q = tree_seq(p, s);
      if (q.n > 0) break;
    }
  }
};

// Scratch of tree_locate in shared memory.
struct TreeLocate {
  long long warp_sum[32];
  long long per, lo, hi, off;
  int s;
};

// This CTA's run: every thread counts a contiguous share of the sequences, a
// block-wide scan gives the total and finds the sequence that holds the run's
// first block.  Called by all THREADS threads; `w` is the same in all of them.
// Returns false for a CTA without work.
template <int THREADS>
SF_DEV bool tree_locate(const TreeArgs& p, TreeLocate& sh, TreeWalk& w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int W = THREADS / 32;
  const int share = (p.batch.n_seqs + THREADS - 1) / THREADS;
  const int s_lo = min(tid * share, p.batch.n_seqs), s_hi = min(s_lo + share, p.batch.n_seqs);
  long long mine = 0;
  bool bad = false;
  for (int s = s_lo; s < s_hi; ++s) {
    const TreeSeq q = tree_seq(p, s);
    mine += q.items(p.n_kv);
    bad = bad || q.bad;
  }
  if (bad && blockIdx.x == 0) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh.warp_sum[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const long long v = sh.warp_sum[i];
    if (i < warp) before += v;
    total += v;
  }
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long lo = per * blockIdx.x;
  const long long hi = min(lo + per, total);
  if (lo >= hi) return false;  // the same in every thread
  long long at = before + inc - mine;
  if (lo >= at && lo < at + mine) {
    for (int s = s_lo; s < s_hi; ++s) {
      const long long it = tree_seq(p, s).items(p.n_kv);
      if (lo < at + it) {
        sh.s = s;
        sh.off = lo - at;
        break;
      }
      at += it;
    }
  }
  __syncthreads();
  w.s = sh.s;
  w.q = tree_seq(p, w.s);
  w.u = static_cast<int>(sh.off / w.q.nb);
  w.b0 = static_cast<int>(sh.off % w.q.nb);
  w.left = hi - lo;
  if (tid == 0) {
    sh.per = per;
    sh.lo = lo;
  }
  return true;
}

// The partial slot of a run's piece.
SF_DEV int tree_slot(bool first) { return 2 * static_cast<int>(blockIdx.x) + (first ? 0 : 1); }

// Rows of the current unit's tile: the first one and how many.
SF_DEV int tree_m0(const TreeArgs& p, const TreeWalk& w) { return w.tile() * p.tile_rows; }
SF_DEV int tree_tile_rows(const TreeArgs& p, const TreeWalk& w) {
  return min(p.tile_rows, w.q.n * p.g - tree_m0(p, w));
}

// By one thread of every CTA: the unit that this CTA's start cuts, if this is
// the first cut in it, for the combine kernel: {rows, row0, m0, head},
// {first CTA, last CTA, the first CTA's slot, 0}; rows 0: nothing to merge.
SF_DEV void tree_describe_none(const TreeArgs& p) { p.desc[2 * blockIdx.x] = make_int4(0, 0, 0, 0); }
SF_DEV void tree_describe(const TreeArgs& p, const TreeWalk& w, long long per, long long lo) {
  const int c = blockIdx.x;
  const long long beg = lo - w.b0, end = beg + w.q.nb;
  if (w.b0 == 0 || beg < lo - per) {
    tree_describe_none(p);
    return;
  }
  p.desc[2 * c] = make_int4(tree_tile_rows(p, w), w.q.row0, tree_m0(p, w), w.head());
  p.desc[2 * c + 1] = make_int4(c - 1, static_cast<int>((end - 1) / per), 2 * (c - 1) + (beg == lo - per ? 0 : 1), 0);
}

// Pool token of a sequence's token, or -1 (flagged) where the table has none.
SF_DEV int tree_pool_token(const TreeArgs& p, int s, int tok) {
  const specfold_paged_cache& c = p.cache;
  const int pg = static_cast<int>(static_cast<unsigned>(tok) / static_cast<unsigned>(c.page_size));
  if (pg < c.table_pages) {
    const int page = c.block_table[s * c.table_stride + pg];
    if (page >= 0 && page < c.num_pages) return page * c.page_size + (tok - pg * c.page_size);
  }
  atomicOr(p.status, SPECFOLD_DEV_BAD_PAGE);
  return -1;
}

// 16-byte asynchronous copy global -> shared of `bytes` (16 or 0, the rest
// zero-filled), and the group waits.
SF_DEV void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
SF_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SF_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- host ----
// Many rows a head group, bf16 (tree_attn_tc.cu): tiles of 256 rows, blocks of
// 128 keys, one CTA per SM.
constexpr int kTreeTcRows = 256, kTreeTcKeys = 128;
int launch_tree_tc(const TreeArgs& a, int hd, int grid, cudaStream_t st);

}  // namespace sf
