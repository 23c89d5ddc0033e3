// The decomposition of a batch of tree attentions, shared by its kernels.
//
// A unit is (sequence, key/value head, tile of query rows) and its work the
// blocks of kb keys of that sequence.  All units' blocks in one line, sequence
// by sequence, head by head, tile by tile, are cut into equal runs, one per CTA:
// the lengths are known on the device only, and one rule serves a single long
// sequence and a ragged batch of short ones.  Starting a unit costs a CTA as
// much as some blocks (its queries, an output to write): a unit counts unit_cost
// places more than its blocks, in front of them, so that a CTA that starts more
// units gets fewer blocks.  A cut inside these places is one at the unit's start.  A run's piece that covers its
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
  int unit_cost;  // a unit's start, in blocks
  float sl2;               // scale * log2(e)
  uint32_t* status;
  int4* desc;              // [2 * grid]: the unit cut at CTA c's start, see tree_describe
  float* part_o;           // [2 * grid][tile_rows][hd], or [2 * grid][hd / 4][tile_rows][4] (tree_attn_tc.cu)
  float* part_ml;          // [2 * grid][tile_rows][2]
};

// One sequence: rows n behind ctx cached tokens, nb blocks of keys, tiles of
// query rows.  An invalid one has none.
struct TreeSeq {
  int row0, n, ctx, nb, tiles;
  bool bad;
  SF_DEV long long items(const TreeArgs& p) const {  // its places in the line
    return static_cast<long long>(nb + (n > 0 ? p.unit_cost : 0)) * tiles * p.n_kv;
  }
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
// tiles) of sequence s from block b0 on, `left` places to go (the unit's start
// not counted when b0 > 0).
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
  // Enter the current unit at its start: its places are paid for, or, where the
  // run ends among them, it is left to the next CTA.
  SF_DEV void enter(const TreeArgs& p) {
    b0 = 0;
    left = left > p.unit_cost ? left - p.unit_cost : 0;
  }
  SF_DEV void next(const TreeArgs& p) {
    left -= blocks();
    if (++u >= q.tiles * p.n_kv) {
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
    enter(p);
  }
};

// Quotient of numbers that hardly ever need more than 32 bits.
SF_DEV long long div_ll(long long a, unsigned b) {
  return a >> 32 ? a / b : static_cast<long long>(static_cast<unsigned>(a) / b);
}

SF_DEV TreeSeq tree_seq_or_none(const TreeArgs& p, int s) {
  if (s < p.batch.n_seqs) return tree_seq(p, s);
  TreeSeq q;
  q.row0 = q.n = q.ctx = q.nb = q.tiles = 0;
  q.bad = false;
  return q;
}

SF_DEV long long warp_prefix(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// This CTA's run, found by every warp on its own (a lane a sequence, 32 at a
// time: no block-wide barrier, one round trip for up to 32 sequences).  lo: the
// run's first block, per: the blocks of a run.  Returns false for a CTA without
// work; the walk is the same in all threads.
SF_DEV bool tree_locate(const TreeArgs& p, TreeWalk& w, long long& lo, long long& per) {
  const int lane = threadIdx.x & 31, n = p.batch.n_seqs;
  TreeSeq q = tree_seq_or_none(p, lane);
  bool bad = q.bad;
  long long inc = warp_prefix(q.items(p), lane);
  long long total = __shfl_sync(0xffffffffu, inc, 31);
  for (int c = 32; c < n; c += 32) {
    const TreeSeq r = tree_seq_or_none(p, c + lane);
    bad = bad || r.bad;
    total += __shfl_sync(0xffffffffu, warp_prefix(r.items(p), lane), 31);
  }
  if (bad && blockIdx.x == 0 && threadIdx.x < 32) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
  per = div_ll(total + gridDim.x - 1, gridDim.x);
  lo = per * blockIdx.x;
  const long long hi = min(lo + per, total);
  if (lo >= hi) return false;
  long long base = 0;
  int c = 0;
  while (lo >= base + __shfl_sync(0xffffffffu, inc, 31)) {
    base += __shfl_sync(0xffffffffu, inc, 31);
    c += 32;
    q = tree_seq_or_none(p, c + lane);
    inc = warp_prefix(q.items(p), lane);
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, lo < base + inc)) - 1;
  const long long off = lo - base - __shfl_sync(0xffffffffu, inc - q.items(p), src);
  w.s = c + src;
  w.q.row0 = __shfl_sync(0xffffffffu, q.row0, src);
  w.q.n = __shfl_sync(0xffffffffu, q.n, src);
  w.q.ctx = __shfl_sync(0xffffffffu, q.ctx, src);
  w.q.nb = __shfl_sync(0xffffffffu, q.nb, src);
  w.q.tiles = __shfl_sync(0xffffffffu, q.tiles, src);
  w.q.bad = false;
  const int places = w.q.nb + p.unit_cost;
  w.u = static_cast<int>(div_ll(off, places));
  const int at = static_cast<int>(off - static_cast<long long>(w.u) * places);
  w.left = hi - lo;
  if (at <= p.unit_cost) {  // at the unit's start
    w.left += at;
    w.enter(p);
  } else {
    w.b0 = at - p.unit_cost;
  }
  return w.left > 0;
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
SF_DEV void tree_describe(const TreeArgs& p, const TreeWalk& w, bool work, long long lo, long long per) {
  const int c = blockIdx.x;
  int4 a = make_int4(0, 0, 0, 0);
  if (work && w.b0 > 0) {
    // the unit's places are [beg, end), its first block's place beg + unit_cost
    const long long beg = lo - w.b0 - p.unit_cost, end = beg + p.unit_cost + w.q.nb, before = lo - per;
    if (beg + p.unit_cost >= before) {  // CTA c - 1 has the first block
      a = make_int4(tree_tile_rows(p, w), w.q.row0, tree_m0(p, w), w.head());
      // per < 2^32: a run of more 64-key blocks than that is no cache's
      p.desc[2 * c + 1] = make_int4(c - 1, static_cast<int>(div_ll(end - 1, static_cast<unsigned>(per))),
                                    2 * (c - 1) + (beg <= before ? 0 : 1), 0);
    }
  }
  p.desc[2 * c] = a;
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
