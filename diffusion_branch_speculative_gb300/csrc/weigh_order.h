// The order of the products of weigh_tokens_tc_kernel, the same in all of its roles, and
// what becomes of them where a wait runs out.  Plain C++: the tests compile it for the host.
#pragma once

#ifdef __CUDACC__
#define SF_ORDER __host__ __device__ __forceinline__
#else
#define SF_ORDER inline
#endif

namespace sf {

// Of a piece of n blocks: groups of `group` blocks, each passed by all tiles of rows, back
// and forth.
struct WItems {
  int n, tiles, group;
  int g0 = 0, tile_at = 0, dir = 1, done = 0;  // group's first block, tile now, its step, tiles of the group so far
  SF_ORDER WItems(int blocks, int tiles_, int ring) : n(blocks), tiles(tiles_), group(tiles_ > 1 ? ring : blocks) {}
  SF_ORDER int blocks() const { return group < n - g0 ? group : n - g0; }
  SF_ORDER bool last() const { return done == tiles - 1; }
  // to the next tile or group; true: another tile's queries are needed
  SF_ORDER bool next() {
    if (++done < tiles) {
      tile_at += dir;
      return true;
    }
    done = 0;
    dir = -dir;
    g0 += group;
    return false;
  }
};

// One half's way through a piece whose first block is the run's it-th: it takes every
// second block, x (0 or 1) those whose number in the run is even or odd.
//   tile(q, ok)   the halves meet there; false once either's ok is
//   block(q, b)   block b of the group; false where a wait ran out
// A wait that ran out is remembered in ok: a product that completes after all would be
// taken for another block's.  No further block is worked on, but the half comes to the
// next tile, which ends the other half as well.  Returns whether both go on.
template <typename Tile, typename Block>
SF_ORDER bool half_pass(WItems q, int it, int x, bool& ok, Tile tile, Block block) {
  for (bool fresh = true; q.g0 < q.n; fresh = q.next()) {
    if (fresh && !(ok = tile(q, ok))) return false;
    for (int b = (x ^ (it + q.g0)) & 1; ok && b < q.blocks(); b += 2) ok = block(q, b);
  }
  return true;
}

}  // namespace sf
