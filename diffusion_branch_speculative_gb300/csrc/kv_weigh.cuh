// What the kernels of specfold_kv_weigh share.
//
// Two launches (few rows often need but one: weigh_unit_kernel), each over a line of
// work as tree_sched.cuh has it.  The first
// finds every row's maximum m (in log2 units) and sum l over the keys it sees: a
// piece that is its whole unit leaves its rows' own in row_ml, any other in its slot
// (2c or 2c + 1 of CTA c: a run's first or last piece), and the CTA with a unit's
// first block notes which slots the unit's pieces have.  The second merges them, in
// order, and adds up every token's 2^(x - m) / l over the rows.
#pragma once

#include "tree_sched.cuh"

namespace sf {

struct WeighArgs {
  TreeArgs t;           // the launch's line; parent, o, desc and the partials of o are not used
  const int32_t* rows;  // null: row t takes q's row t
  int n_src;
  float decay;
  specfold_token_weights w;
  int stat_rows;        // rows of a tile of the first launch
  int stat_tiles;       // its tiles a head, at most
  int4* span;           // [n_seqs][n_kv][stat_tiles]: a unit's first and last CTA, the first one's slot (-1: whole)
  float2* part;         // [2 * grid of the first launch][stat_rows]: m, l
  float2* row_ml;       // [T][n_kv * g]: m, l
  float* scores;        // [n_seqs][n_kv][w.tokens][score_rows] in log2 units, or null
  int score_rows;
  int blocks, spread;   // of a cluster, where one holds a unit; blocks a unit that fill the SMs
};

// q's row for row t of the batch; -1: there is none (reported).
SF_DEV int weigh_src(const WeighArgs& p, int t) {
  const int r = p.rows ? p.rows[t] : t;
  if (r >= 0 && r < p.n_src) return r;
  atomicOr(p.t.status, SPECFOLD_DEV_BAD_SEQ);
  return -1;
}

// Whether row t of a batch with `rows` has one (not reported).  A row without is given q's row 0 to work
// on, whose scores, and those with an infinite key, may be anything: it sees no token, so that all its
// scores are -inf.
SF_DEV bool weigh_has_src(const WeighArgs& p, int t) { return p.rows[t] >= 0 && p.rows[t] < p.n_src; }

SF_DEV size_t weigh_unit(const WeighArgs& p, const TreeWalk& w, int tile) {
  return (static_cast<size_t>(w.s) * p.t.n_kv + w.head) * p.stat_tiles + tile;
}

// By one thread, for a piece with its unit's first block.
SF_DEV void weigh_note_span(const WeighArgs& p, const TreeWalk& w, bool first, unsigned per) {
  const int c = blockIdx.x;
  int last = c;
  if (!w.whole()) {
    const unsigned wt = w.q.weight(p.t, w.tile);
    // places of the unit behind this run (a block is its last place's owner's)
    const unsigned beyond = static_cast<unsigned>(w.q.nb - w.n) * wt - (w.left - static_cast<unsigned>(w.n) * wt);
    last = c + 1 + static_cast<int>((beyond - 1) / per);
  }
  p.span[weigh_unit(p, w, w.tile)] = make_int4(c, last, w.whole() ? -1 : tree_slot(first), 0);
}

// Where row m of a head's group has its own.
SF_DEV float2* weigh_row_ml(const WeighArgs& p, int row0, int head, int m) {
  return p.row_ml + static_cast<size_t>(row0 + m / p.t.g) * (p.t.n_kv * p.t.g) + head * p.t.g + m % p.t.g;
}
// Row r of the current piece's tile: whole or partial.
SF_DEV void weigh_leave(const WeighArgs& p, const TreeWalk& w, bool first, int r, float2 v) {
  const int m = tree_m0(p.t, w) + r;
  if (r >= tree_tile_rows(p.t, w)) return;
  if (weigh_src(p, w.q.row0 + m / p.t.g) < 0) v = make_float2(INFINITY, 0.f);  // weighs nothing: 2^(x - inf) = 0
  if (w.whole())
    *weigh_row_ml(p, w.q.row0, w.head, m) = v;
  else
    p.part[static_cast<size_t>(tree_slot(first)) * p.stat_rows + r] = v;
}

// Two partials of a row as one.
SF_DEV float2 weigh_merge(float2 a, float2 b) {
  const float M = fmaxf(a.x, b.x);
  return make_float2(M, fmaf(merge_weight(a.x, M), a.y, merge_weight(b.x, M) * b.y));
}

// Whether a row's weights are no numbers: a score of it is NaN or +inf, or all are -inf.  (One
// that weighs nothing has m = +inf, l = 0.)
SF_DEV bool weigh_no_number(float2 v) { return v.y != v.y || v.x == -INFINITY; }

// This thread's merge of a row, the r-th of the unit's tile: the partials z0, z0 + zs, ...;
// whole: where it has its own if the unit was not cut.
SF_DEV float2 weigh_gather(const WeighArgs& p, size_t unit, const float2* whole, int r, int z0, int zs) {
  const int4 sp = p.span[unit];
  float2 v = make_float2(-INFINITY, 0.f);
  if (sp.z < 0) return z0 == 0 ? *whole : v;
#pragma unroll 4
  for (int z = sp.x + z0; z <= sp.y; z += zs)
    v = weigh_merge(v, p.part[static_cast<size_t>(z == sp.x ? sp.z : 2 * z) * p.stat_rows + r]);
  return v;
}

// Host: many rows a head group, bf16 (kv_weigh_tc.cu).
constexpr int kWeighTcRows = 256, kWeighTcKeys = 128;
int launch_weigh_tc(WeighArgs& a, int hd, int grid, cudaStream_t st);

}  // namespace sf
