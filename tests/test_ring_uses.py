"""Which phases of a ring's barriers a CTA that gave up waits for
(csrc/ring_uses.h), compiled for the host (CPU only)."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "diffusion_branch_speculative_gb300", "csrc")

SOURCE = r"""
#include "ring_uses.h"
extern "C" int last_uses(int last, int ring, int* out) {
  int k = 0;
  sf::each_last_use(last, ring, [&](int slot, unsigned parity) {
    out[2 * k] = slot;
    out[2 * k++ + 1] = static_cast<int>(parity);
  });
  return k;
}
"""


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(SOURCE)
    lib = str(d / "ring.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(d / "ring.cpp"),
                    "-o", lib], check=True)
    return ctypes.CDLL(lib)


@pytest.mark.parametrize("ring", [1, 2, 3, 4, 8])
def test_every_copy_in_flight_is_waited_for(L, ring):
    """Whatever order the copies land in: of uses 0 .. last, any of the last `ring` may be in flight (a slot is used
    again only once its use before is done with)."""
    for last in range(-1, 5 * ring):
        out = (ctypes.c_int * (2 * ring))()
        n = L.last_uses(last, ring, out)
        waits = {(out[2 * i], out[2 * i + 1]) for i in range(n)}
        flight = {(i % ring, i // ring % 2) for i in range(max(last - ring + 1, 0), last + 1)}
        assert waits == flight and n == len(flight)


def test_no_waits_without_a_use(L):
    assert L.last_uses(-1, 4, (ctypes.c_int * 8)()) == 0
