"""The order of the products that weigh many rows (csrc/weigh_order.h), compiled for the
host: every block of every tile once, and nothing more once a wait has run out (CPU only)."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "diffusion_branch_speculative_gb300", "csrc")

SOURCE = r"""
#include "weigh_order.h"
using namespace sf;

// The issuing warp's order: (tile, block of the piece), `buffer` the half that takes it.
extern "C" int issued(int n, int tiles, int ring, int it, int* out) {
  int k = 0;
  for (WItems q(n, tiles, ring); q.g0 < q.n; q.next())
    for (int b = 0; b < q.blocks(); ++b, ++k) {
      out[3 * k] = q.tile_at;
      out[3 * k + 1] = q.g0 + b;
      out[3 * k + 2] = (it + q.g0 + b) & 1;
    }
  return k;
}

// A half's way through `pieces` pieces: its fails-th wait runs out (-1: none), all others are
// satisfied.  Returns the blocks worked on, out[0] the tiles it came to, out[1] whether it came to
// the last one with its wait run out, out[2] whether it went through all.
extern "C" int taken(int pieces, int n, int tiles, int ring, int x, int fails, int* out, int* blocks) {
  int waits = 0, worked = 0, it = 0;
  bool ok = true;
  out[0] = out[1] = 0;
  out[2] = 1;
  for (int i = 0; i < pieces; ++i) {
    auto tile = [&](const WItems&, bool mine) {
      ++out[0];
      out[1] = !mine;
      return mine;
    };
    auto block = [&](const WItems& q, int b) {
      if (waits++ == fails) return false;
      blocks[2 * worked] = q.tile_at;
      blocks[2 * worked + 1] = q.g0 + b;
      ++worked;
      return true;
    };
    if (!half_pass(WItems(n, tiles, ring), it, x, ok, tile, block)) {
      out[2] = 0;
      break;
    }
    it += n;
  }
  return worked;
}
"""


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("order")
    (d / "order.cpp").write_text(SOURCE)
    lib = str(d / "order.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(d / "order.cpp"),
                    "-o", lib], check=True)
    return ctypes.CDLL(lib)


SHAPES = [(1, 1), (7, 1), (8, 1), (1, 2), (3, 2), (4, 3), (9, 2), (10, 3), (17, 5)]   # blocks, tiles


def taken(L, pieces, n, tiles, ring, x, fails):
    out, blocks = (ctypes.c_int * 3)(), (ctypes.c_int * (2 * pieces * n * tiles + 2))()
    k = L.taken(pieces, n, tiles, ring, x, fails, out, blocks)
    return [(blocks[2 * i], blocks[2 * i + 1]) for i in range(k)], list(out)


@pytest.mark.parametrize("ring", [4, 8])
@pytest.mark.parametrize("n,tiles", SHAPES)
@pytest.mark.parametrize("it", [0, 3])
def test_every_block_of_every_tile_once(L, n, tiles, ring, it):
    out = (ctypes.c_int * (3 * n * tiles))()
    assert L.issued(n, tiles, ring, it, out) == n * tiles
    order = [tuple(out[3 * i:3 * i + 3]) for i in range(n * tiles)]
    assert sorted((t, b) for t, b, _ in order) == [(t, b) for t in range(tiles) for b in range(n)]
    at = {}
    for i, (t, b, _) in enumerate(order):       # a group's blocks leave the ring before the next one's come
        at.setdefault(b, []).append(i)
    if tiles > 1:
        for b in range(ring, n):
            assert max(at[b - ring]) < min(at[b])


@pytest.mark.parametrize("ring", [4, 8])
@pytest.mark.parametrize("n,tiles", SHAPES)
def test_the_halves_take_what_is_issued(L, n, tiles, ring):
    out = (ctypes.c_int * (3 * n * tiles))()
    L.issued(n, tiles, ring, 0, out)
    for x in (0, 1):
        want = [(out[3 * i], out[3 * i + 1]) for i in range(n * tiles) if out[3 * i + 2] == x]
        got, (met, missed, through) = taken(L, 1, n, tiles, ring, x, -1)
        assert got == want and through == 1 and not missed
        groups = 1 if tiles == 1 else -(-n // ring)
        assert met == 1 + groups * (tiles - 1)      # a group begins with the tile that the one before ended with


@pytest.mark.parametrize("n,tiles", [(3, 1), (9, 2), (10, 3), (17, 5)])
def test_nothing_is_worked_on_behind_a_wait_that_ran_out(L, n, tiles):
    ring = 4
    for x in (0, 1):
        whole, _ = taken(L, 3, n, tiles, ring, x, -1)
        for fails in range(len(whole)):
            got, (met, missed, through) = taken(L, 3, n, tiles, ring, x, fails)
            assert got == whole[:fails]             # later waits are satisfied, and yet
            # the half comes to the next tile there is, and ends there
            assert (missed and not through) or (through and fails >= len(whole) - 4 * ring)
