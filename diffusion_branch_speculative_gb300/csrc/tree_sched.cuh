// The decomposition of a batch of tree attentions, shared by its kernels.
//
// A unit is (sequence, key/value head, tile of query rows) and its work the
// blocks of kb keys of that sequence.  All units' blocks in one line, sequence
// by sequence, head by head, tile by tile, are cut into equal runs, one per CTA:
// the lengths are known on the device only, and one rule serves a single long
// sequence and a ragged batch of short ones.  Starting a unit costs a CTA as
// much as some blocks (its queries, an output to write): a unit counts unit_cost
// blocks more than it has, in front of them, so that a CTA that starts more
// units gets fewer blocks.  A block counts as many places as its tile weighs: one
// with at most half its rows may cost less.  A cut inside a block's places is one
// before it, a cut inside a unit's start one before the unit.  A run's piece that covers its
// whole unit writes the output; any other writes an unnormalised partial (o,
// running max m in log2 units, sum l), at most the run's first and last piece
// (slots 2c and 2c + 1 of CTA c), which the combine kernel merges in order, so
// results do not depend on timing.
#pragma once

#include "sf_device.cuh"
#include "sf_internal.h"
#include "warp_ops.cuh"

namespace sf {

// Blocks that a call may count, head by head: what the header states.  Nothing here
// needs the bound (at 10^8 blocks a call reads 1.6 TB and more, a quarter of a second
// at the copy rate, once for every tile of rows); it turns lengths that cannot be meant
// into an error.
constexpr unsigned kTreeMaxBlocks = 100000000u;

struct TreeArgs {
  const void* q;
  void* o;
  long long q_rs, q_hs, o_rs, o_hs;
  specfold_paged_cache cache;
  const int32_t* parent;
  SeqBatch batch;
  int max_nodes, n_kv, g;
  unsigned most_tokens;  // a sequence's tokens, its rows among them, at most
  int tile_rows;  // query rows of a tile: row m is node m / g, head m % g of the group
  int kb;         // keys per block
  int unit_cost;  // a unit's start, in blocks
  int w_full, w_half;  // places of a block: of a tile with more, with at most half its rows
  float sl2;               // scale * log2(e)
  uint32_t* status;
  int4* desc;              // [2 * grid]: the unit cut at CTA c's start, see tree_describe
  float* part_o;           // [2 * grid][tile_rows][hd], or [2 * grid][hd / 4][tile_rows][4] (tree_attn_tc.cu)
  float* part_ml;          // [2 * grid][tile_rows][2]
};

// One sequence: rows n behind ctx cached tokens, nb blocks of keys, tiles of
// query rows (the last one's rows may be at most half a tile's).  An invalid one
// has none.
struct TreeSeq {
  int row0, n, ctx, nb, tiles;
  bool half, bad;
  SF_DEV unsigned weight(const TreeArgs& p, int tile) const { return half && tile == tiles - 1 ? p.w_half : p.w_full; }
  // places in the line of all its tiles of one head
  template <typename Places>
  SF_DEV Places head_places(const TreeArgs& p) const {
    return static_cast<Places>(nb + p.unit_cost) * static_cast<unsigned>(tiles * p.w_full - (half ? p.w_full - p.w_half : 0));
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
          q.ctx > 0x7fffffff - 2 * SPECFOLD_MAX_TREE ||
          static_cast<unsigned>(q.ctx) + static_cast<unsigned>(end - q.row0) > p.most_tokens;
  q.n = q.bad ? 0 : end - q.row0;
  q.nb = q.n > 0 ? (q.ctx + q.n - 1) / p.kb + 1 : 0;
  q.tiles = (q.n * p.g + p.tile_rows - 1) / p.tile_rows;
  q.half = 2 * (q.n * p.g - (q.tiles - 1) * p.tile_rows) <= p.tile_rows;
  return q;
}

// A CTA's walk along its run: the current piece, blocks b0 .. b0 + n - 1 of
// (sequence s, head, tile), and the places left from there on.  All of this is
// executed once or twice a launch, mostly on cold instruction caches: it is kept
// short (few divisions; 32 bits within a run).
struct TreeWalk {
  int s, head, tile, b0, n;
  unsigned left;
  unsigned past;  // places of block b0 before the run's first, where the run starts in it
  TreeSeq q;
  SF_DEV bool whole() const { return n == q.nb; }
  SF_DEV void cut(unsigned wt) {  // n, from b0 and left
    n = q.nb - b0;
    if (left < n * wt) n = left / wt;
  }
  // The current unit from its start on, whose start is paid for, or, where the
  // run ends before its first block does, is left to the next CTA.
  SF_DEV void enter(const TreeArgs& p) {
    const unsigned wt = q.weight(p, tile), start = p.unit_cost * wt;
    b0 = n = 0;
    if (left < start + wt) return;
    left -= start;
    cut(wt);
  }
  SF_DEV void next(const TreeArgs& p) {
    const bool ends = b0 + n < q.nb;  // the run does
    left -= n * q.weight(p, tile);
    b0 = n = 0;
    if (ends || left == 0) return;
    if (++tile == q.tiles) {
      tile = 0;
      if (++head == p.n_kv) {
        head = 0;
        do {
          if (++s >= p.batch.n_seqs) return;  // lengths that changed under the call
          q = tree_seq(p, s);
        } while (q.n == 0);
      }
    }
    enter(p);
  }
};

// This CTA's run, found by every warp on its own (a lane a sequence, 32 at a
// time: no block-wide barrier, one round trip for up to 32 sequences).  per: the
// places of a run.  False for a CTA without work; the walk is the same in all threads.
//
// Places is 64 bits where the line may be longer than 32 bits hold (10^8 blocks times
// up to 4096 tiles of a head group's rows; a run's places fit always: 4.1 10^11 over
// the fp32 kernel's 456 CTAs, 6.4 10^10 over the tcgen05 kernel's 152), and that form
// alone asks for the limit.  With it for every call the tcgen05 kernel took 1 to 2 us more.
template <typename Places>
SF_DEV bool tree_locate_in(const TreeArgs& p, TreeWalk& w, unsigned& per) {
  constexpr bool kLong = sizeof(Places) == 8;
  const int lane = threadIdx.x & 31, n_seqs = p.batch.n_seqs;
  TreeSeq q;
  Places inc = 0;
  float size = 0.f;  // this lane's part of the line, in places, which cannot wrap
  Places blocks = 0;
  // 32 sequences from c on: q this lane's, inc the places up to and with its own
  auto take = [&](int c) {
    q = tree_seq(p, min(c + lane, n_seqs - 1));
    const bool mine = c + lane < n_seqs && q.n > 0;
    const Places places = mine ? q.head_places<Places>(p) * p.n_kv : 0;
    if constexpr (kLong)
      blocks += mine ? static_cast<Places>(q.nb) * p.n_kv : 0;
    else
      size += mine ? static_cast<float>(q.nb + p.unit_cost) * q.tiles * p.w_full * p.n_kv : 0.f;
    inc = places;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Places u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    return places;
  };
  Places total = 0, places = 0;
  bool bad = false;
#pragma unroll 1
  for (int c = (n_seqs - 1) & ~31; c >= 0; c -= 32) {  // the first 32 last: they stay
    places = take(c);
    total += __shfl_sync(0xffffffffu, inc, 31);
    bad = bad || q.bad;
  }
  bool too_long = false;
  if constexpr (kLong) {
    // (a lane's count is cut where it is too much by itself, so that 32 of them fit)
    const unsigned cut = static_cast<unsigned>(min(blocks, static_cast<Places>(kTreeMaxBlocks) + 1));
    too_long = __reduce_add_sync(0xffffffffu, cut) > kTreeMaxBlocks;
  } else if (__any_sync(0xffffffffu, size > kTreeMaxBlocks / 32)) {  // else no more than that in all
    return tree_locate_in<unsigned long long>(p, w, per);
  }
  const Places run = max((total + gridDim.x - 1) / gridDim.x, static_cast<Places>(p.w_full));  // a block at least
  if (kLong && run > 0x7fffffffu) too_long = true;  // (not on a grid of a hundred CTAs)
  if ((bad || too_long) && blockIdx.x == 0 && threadIdx.x < 32) atomicOr(p.status, SPECFOLD_DEV_BAD_SEQ);
  per = static_cast<unsigned>(run);
  const Places lo = run * blockIdx.x;  // where the run starts in the line
  if (too_long || lo >= total) return false;
  Places before = 0;
  int c = 0;
#pragma unroll 1
  while (true) {
    const Places sum = __shfl_sync(0xffffffffu, inc, 31);
    if (lo < before + sum) break;
    before += sum;
    c += 32;
    if (c >= n_seqs) return false;  // lengths that changed under the call
    places = take(c);
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, lo < before + inc)) - 1;
  const Places off = lo - before - __shfl_sync(0xffffffffu, inc - places, src);
  w.s = c + src;
  w.q.row0 = __shfl_sync(0xffffffffu, q.row0, src);
  w.q.n = __shfl_sync(0xffffffffu, q.n, src);
  w.q.ctx = __shfl_sync(0xffffffffu, q.ctx, src);
  w.q.nb = __shfl_sync(0xffffffffu, q.nb, src);
  w.q.tiles = __shfl_sync(0xffffffffu, q.tiles, src);
  w.q.half = __shfl_sync(0xffffffffu, q.half, src);
  const Places hp = w.q.head_places<Places>(p);
  const unsigned tp = static_cast<unsigned>(w.q.nb + p.unit_cost) * p.w_full;
  w.head = static_cast<int>(off / hp);
  const Places in_head = off - w.head * hp;
  w.tile = min(static_cast<int>(in_head / tp), w.q.tiles - 1);
  const unsigned at = static_cast<unsigned>(in_head - static_cast<Places>(w.tile) * tp);
  const unsigned wt = w.q.weight(p, w.tile), v = at / wt;  // blocks, the start's among them, before the cut
  w.left = static_cast<unsigned>(min(run, total - lo));
  if (static_cast<int>(v) <= p.unit_cost) {  // before the unit
    w.left += at;
    w.enter(p);
  } else {
    w.past = at - v * wt;
    w.left += w.past;
    w.b0 = v - p.unit_cost;
    w.cut(wt);
  }
  return w.n > 0;
}
SF_DEV bool tree_locate(const TreeArgs& p, TreeWalk& w, unsigned& per) { return tree_locate_in<unsigned>(p, w, per); }

// The partial slot of a run's piece.
SF_DEV int tree_slot(bool first) { return 2 * static_cast<int>(blockIdx.x) + (first ? 0 : 1); }

// Rows of the current unit's tile: the first one and how many.
SF_DEV int tree_m0(const TreeArgs& p, const TreeWalk& w) { return w.tile * p.tile_rows; }
SF_DEV int tree_tile_rows(const TreeArgs& p, const TreeWalk& w) {
  return min(p.tile_rows, w.q.n * p.g - tree_m0(p, w));
}

// By one thread of every CTA: the unit that this CTA's start cuts, if this is
// the first cut in it, for the combine kernel: {rows, row0, m0, head},
// {first CTA, last CTA, the first CTA's slot, 0}; rows 0: nothing to merge.
SF_DEV void tree_describe(const TreeArgs& p, const TreeWalk& w, bool work, unsigned per) {
  const int c = blockIdx.x;
  int4 a = make_int4(0, 0, 0, 0);
  if (work && w.b0 > 0) {
    // Where the unit begins and ends, from where its block b0 does, in places from the cut
    // on; a block is its last place's owner's.
    const unsigned wt = w.q.weight(p, w.tile);
    const unsigned begins = w.past + (w.b0 + p.unit_cost) * wt, ends = (w.q.nb - w.b0) * wt - w.past;  // before, behind the cut
    if (begins - (p.unit_cost + 1) * wt < per) {  // CTA c - 1 has the first block
      a = make_int4(tree_tile_rows(p, w), w.q.row0, tree_m0(p, w), w.head);
      p.desc[2 * c + 1] = make_int4(c - 1, c + (ends - 1) / per, 2 * (c - 1) + (begins >= per ? 0 : 1), 0);
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

// ---- host ----
// Many rows a head group, bf16 (tree_attn_tc.cu): tiles of 256 rows, blocks of
// 128 keys, one CTA per SM.
constexpr int kTreeTcRows = 256, kTreeTcKeys = 128;
int launch_tree_tc(const TreeArgs& a, int hd, int grid, cudaStream_t st);

}  // namespace sf
