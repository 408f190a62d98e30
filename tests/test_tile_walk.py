"""The order in which the tensor-core products take their tiles (csrc/tile_walk.h), on the CPU: every tile of every
range exactly once, whatever their numbers."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compensated_bit_reproducible_gb300", "csrc")
SOURCE = """
#include "tile_walk.h"
using namespace repro;
extern "C" long long walk(int m, int n, int tn, int splits, int band, unsigned step, int* out, long long room) {
  const TileShape sh{m, n, 64, tn, splits, 0, 0, band};
  long long seen = 0;
  for (unsigned first = 0; first < step; ++first)
    for (TileWalk w(sh, first, step); w.more(); w.next()) {
      if (seen < room) out[3 * seen] = w.m, out[3 * seen + 1] = w.n, out[3 * seen + 2] = w.split;
      ++seen;
    }
  return seen;
}
extern "C" long long tiles(int m, int n, int tn, int splits) { return TileShape{m, n, 64, tn, splits, 0, 0, 8}.tiles(); }
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    at = tmp_path_factory.mktemp("walk")
    src, so = at / "walk.cpp", at / "walk.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.walk.restype = lib.tiles.restype = ctypes.c_longlong
    lib.walk.argtypes = [ctypes.c_int] * 5 + [ctypes.c_uint, ctypes.c_void_p, ctypes.c_longlong]
    return lib


@pytest.mark.parametrize("band", [1, 8, 1 << 22, 0x7fffffff])
@pytest.mark.parametrize("nt", [1, 2, 10, 1023, 1024, 1025, 2047, 2048, 4096])
@pytest.mark.parametrize("mt,splits,step", [(1, 1, 1), (1, 1, 76), (2, 3, 76), (5, 1, 7), (8, 1, 76), (19, 2, 76)])
def test_every_tile_once(walk, mt, nt, splits, step, band):
    for tn, cut in ((256, 0), (256, 255), (96, 31)):
        m, n = mt * 256 - (37 if mt > 1 else 0), nt * tn - cut
        room = mt * nt * splits
        assert walk.tiles(m, n, tn, splits) == room
        out = np.empty((room, 3), np.int32)
        assert walk.walk(m, n, tn, splits, band, step, out.ctypes.data, room) == room
        assert out.min() >= 0 and np.all(out.max(0) < [mt, nt, splits])
        flat = (out[:, 2].astype(np.int64) * mt + out[:, 0]) * nt + out[:, 1]
        assert np.array_equal(np.sort(flat), np.arange(room))


def test_tiles_at_the_largest_shapes(walk):
    """Counts in 64 bits, for the refusal of what 32 do not hold."""
    assert walk.tiles((1 << 30), (1 << 30), 32, 16) == (1 << 22) * (1 << 25) * 16
    assert walk.tiles(0x7fffffff, 1, 256, 1) == 1 << 23
