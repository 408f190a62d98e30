// Which tiles of a product a pair of blocks works on, and in which order.  Plain
// arithmetic, callable on the host as well.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define REPRO_HD __host__ __device__ __forceinline__
#else
#define REPRO_HD inline
#endif

namespace repro {

constexpr int TG_M = 256, TG_N = 256, TG_K = 64;

struct TileShape {
  int m, n, k;      // rows of A, rows of B, inner dimension
  int tn, splits;   // columns of a tile, ranges of the inner dimension
  int bn0, bk0;     // B's first row and first inner index within its tensor map
  int band;         // order of the tiles, see TileWalk
  REPRO_HD int mt() const { return (int)(((unsigned)m + TG_M - 1) / TG_M); }
  REPRO_HD int nt() const { return (int)(((unsigned)n + (unsigned)tn - 1) / (unsigned)tn); }
  REPRO_HD int64_t tiles() const { return (int64_t)mt() * nt() * splits; }
};

// The walk counts tiles in 32 bits, and steps past the last one by at most a
// step.
constexpr int64_t TILES_MAX = 0x7fffffff;

// The tiles of a pair, every step-th of them: within a range of the inner
// dimension, bands of `band` tiles of m; in a band m fastest, then n.  With 8,
// the tiles in flight form a block of about 8 x 10, which reads fewer different
// rows of A and B at a time than a column of all m does.  A band is at most all
// of m, so that its tiles are no more than the range's.
struct TileWalk {
  int m, n, split, mt, nt, splits, width;
  unsigned at, step;
  REPRO_HD TileWalk(const TileShape& sh, unsigned first, unsigned stride)
      : mt(sh.mt()), nt(sh.nt()), splits(sh.splits), width(sh.band < mt ? sh.band : mt), at(first), step(stride) {
    place();
  }
  REPRO_HD void place() {
    const unsigned flat = (unsigned)mt * (unsigned)nt, s = at / flat, in = at - s * flat;
    const unsigned wide = (unsigned)nt * (unsigned)width, band = in / wide, r = in - band * wide;
    const unsigned left = (unsigned)mt - band * (unsigned)width;
    const unsigned high = left < (unsigned)width ? left : (unsigned)width;
    split = (int)s;
    n = (int)(r / high);
    m = (int)(band * (unsigned)width + r % high);
  }
  REPRO_HD bool more() const { return split < splits; }
  REPRO_HD void next() {
    at += step;
    place();
  }
};

}  // namespace repro
