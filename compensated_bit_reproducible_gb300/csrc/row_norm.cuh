// Rows of a matrix through shared memory, several to a block: what the layer
// norm's two directions share.
#pragma once
#include <atomic>
#include "elem.cuh"
#include "launch.h"
#include "mbarrier.cuh"

namespace repro {


// Threads of a block that takes a row of any length alone.
constexpr int LN_LONG_T = 1024;

// A row of `cols` columns is held by WARPS warps, N elements per thread as U
// packs of V: pack u of thread t starts at column (u * threads + t) * V.  A
// block of fewer than eight such warps holds ROWS rows at a time.
template <int V, int WARPS>
struct RowShape {
  static constexpr int N = 16, U = N / V, T = 32 * WARPS, COLS = T * N;
  static constexpr int ROWS = WARPS < 8 ? 8 / WARPS : 1, BLOCK = T * ROWS;
};
// Elements per thread.  Rows come through shared memory, so a thread's registers
// hold only what it works on.
constexpr int ROW_N = 16;
// How rows lie in memory: every row on 16 bytes; rows of 16-bit elements that
// start on a word or between two, alike in all matrices of the call; anything.
// An access to shared memory takes 16 bytes or four, or the elements apart.
enum { WIDE, ALIKE, APART };
template <typename T, int MODE> struct Access { static constexpr int V = MODE == WIDE ? Vec16<T>::N : 4 / (int)sizeof(T); };

// Element k of a thread's packs.
template <typename T, int V, int U>
__device__ __forceinline__ float elem(const Pack<T, V> (&p)[U], int k) {
  return to_f32<T>(p[k / V].e[k % V]);
}
template <typename T, int V, int U>
__device__ __forceinline__ F2 elem2(const Pack<T, V> (&p)[U], int h) {
  if constexpr (V > 1) return get2(p[2 * h / V], h % (V / 2));
  else return pk2(elem(p, 2 * h), elem(p, 2 * h + 1));
}
template <typename T, int V, int U>
__device__ __forceinline__ void put2(Pack<T, V> (&p)[U], int h, F2 v) {
  if constexpr (V > 1) {
    set2(p[2 * h / V], h % (V / 2), v);
  } else {
    float a, b;
    up2(v, a, b);
    p[2 * h].e[0] = from_f32<T>(a);
    p[2 * h + 1].e[0] = from_f32<T>(b);
  }
}

// Sums over the row's threads, the same bits in every thread: butterfly in the
// warp, then the warps' values in order.  The row's warps meet at a barrier of
// their own; `buf` may be written again once another row_sum of the row, in
// another buffer, has passed.
template <int WARPS, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float (*buf)[WARPS], int warp, int lane, int row) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  if (WARPS == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) buf[i][warp] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(row + 1), "n"(32 * WARPS) : "memory");
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (WARPS % 4 == 0) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; w += 4) {
        const Pack<float, 4> q = load_pack<float, 4>(&buf[i][w]);
        s += (q.e[0] + q.e[1]) + (q.e[2] + q.e[3]);
      }
      v[i] = s;
    } else {
      float s = buf[i][0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) s += buf[i][w];
      v[i] = s;
    }
  }
}
__device__ __forceinline__ float across(F2 v) {
  float a, b;
  up2(v, a, b);
  return a + b;
}

// A ring of bulk copies into shared memory, one barrier a stage.  Waits are
// bounded: one that runs out (about two seconds) marks `error` and lets every
// later one of its thread pass, so the block ends with values that mean nothing.
// The thread that fills the ring stops then (the next row to fill is put past the
// last) and leaves its copies time to land, before the block can end or use the
// ring for something else.  All of it where a wait runs out: a test in the rows'
// loop or after it costs the large layer norm 1%.
constexpr int RING_MAX = 4;
constexpr int64_t NO_ROW = 1ll << 62;
struct Ring {
  uint64_t* full;
  int stages, s;
  uint32_t phase;
  bool dead;
  TileError error;
  __device__ __forceinline__ Ring(uint64_t* f, int n, TileError e)
      : full(f), stages(n), s(0), phase(0), dead(false), error(e) {}
  __device__ __forceinline__ void init() {
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&full[i]), 1 + error.never);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __device__ __forceinline__ void expect(int stage, uint32_t bytes) { mbar_expect(smem_u32(&full[stage]), bytes); }
  __device__ __forceinline__ void copy(void* dst, const void* src, uint32_t bytes, int stage) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(&full[stage]))
        : "memory");
  }
  // `ahead`: how far ahead of the row waited for the thread fills.
  __device__ __forceinline__ void wait(int64_t& ahead) {
    const uint32_t b = smem_u32(&full[s]);
    if (dead || mbar_try(b, phase)) return;
    const uint64_t t0 = now_ns();
    while (!mbar_try(b, phase)) {
      if (now_ns() - t0 > error.limit_ns) {
        dead = true;
        *(volatile int*)error.device = 1;
        *(volatile int*)error.host = 1;
        __threadfence_system();
        ahead = NO_ROW;
        pause_ns(WAIT_DRAIN_NS);
        return;
      }
    }
  }
  __device__ __forceinline__ void next() {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

// A pack of a row from column c.  Pairs of 16-bit elements go out as whole words:
// ALIKE, their columns are chosen so that they are words; APART, where the row
// starts between words, each lane's word is its neighbour's second element and
// its own first.  (Every lane of the warp calls, with neighbouring packs.)
template <typename T, int V, int MODE>
__device__ __forceinline__ void store_in_row(T* row, int c, int cols, int lane, const Pack<T, V>& v) {
  if constexpr (V == 2 && sizeof(T) == 2) {
    if (MODE == ALIKE || ((uintptr_t)row & 2) == 0) {
      if (c >= 0 && c + 1 < cols) {
        store_pack<T, V>(row + c, v);
      } else {
        if (c >= 0 && c < cols) row[c] = v.e[0];
        if (c < 0) row[0] = v.e[1];
      }
    } else {
      const unsigned own = *reinterpret_cast<const unsigned*>(&v);
      const unsigned before = __shfl_up_sync(0xffffffffu, own, 1);
      if (c < cols) {
        if (lane) *reinterpret_cast<unsigned*>(row + c - 1) = __funnelshift_r(before, own, 16);
        else row[c] = v.e[0];
      }
      // the last element of the warp, or of the row, has no neighbour to take it
      if (c + 1 < cols && (lane == 31 || c + 2 >= cols)) row[c + 1] = v.e[1];
    }
  } else {
    if (c < cols) store_pack<T, V>(row + c, v);
  }
}

// Whether the rows of a slot start between words.  Its rows are an even number
// apart (row_step), so that all of them do or none.
template <typename T, int MODE>
__device__ __forceinline__ int first_shift(const T* x, int64_t ldx, int slot, int held) {
  if (MODE != ALIKE || sizeof(T) != 2) return 0;
  return (int)(((uintptr_t)(x + ((int64_t)blockIdx.x * held + slot) * ldx) >> 1) & 1);
}

// A row vector kept in shared memory (the rings leave the L1 cache too small for
// it), or ones or zeros for a null one; `front` places before it.
template <typename T>
__device__ __forceinline__ void keep_vector(const T* __restrict__ v, T* to, int cols, T otherwise, int front) {
  constexpr int V = Vec16<T>::N;
  if (threadIdx.x < front) to[threadIdx.x] = otherwise;
  to += front;
  const int packed = v && !front && ((uintptr_t)v & 15) == 0 ? cols / V * V : 0;
  for (int c = threadIdx.x * V; c < packed; c += blockDim.x * V) store_pack<T, V>(to + c, load_pack<T, V>(v + c));
  for (int c = packed + threadIdx.x; c < cols; c += blockDim.x) to[c] = v ? v[c] : otherwise;
}

// Bytes of a row's place in a ring, and of a kept vector: with room for the
// bytes around a row that starts and ends anywhere.
__host__ __device__ inline uint32_t row_place(int64_t cols, int size, int mode) {
  return (uint32_t)((cols * size + 15) / 16 * 16 + (mode == WIDE ? 0 : 16));
}

// Bytes of a vector kept beside the ring, and how many copies of it (see the
// kernels).
__host__ __device__ inline uint32_t vector_place(int64_t cols, int size, int mode) {
  return (uint32_t)(((cols + 2) * size + 15) / 16 * 16);
}
inline int vector_copies(int size, int mode) { return mode == ALIKE && size == 2 ? 2 : 1; }

// Copies of a slot's rows, one after another, into places of its ring.  A row that
// does not start and end on 16 bytes is copied with the bytes around it; the
// matrix's first and last row (and rows shorter than 16 bytes), around which
// there may be nothing, with their own first and last elements apart.  Only the
// thread that fills keeps one: it is on the way of every row, so a copy costs an
// addition, two roundings and a comparison.
template <typename T, int MODE>
struct RowCopies {
  uintptr_t at, step, first, last;   // the next row, to the one after it; the matrix's first and last row
  uint32_t size;
  bool tiny;
  __device__ __forceinline__ RowCopies(const T* m, int64_t ld, int64_t rows, int cols, int64_t row, int64_t rows_on) {
    at = (uintptr_t)(m + row * ld);
    step = (uintptr_t)(rows_on * ld) * sizeof(T);
    first = (uintptr_t)m;
    last = (uintptr_t)(m + (rows - 1) * ld);
    size = (uint32_t)cols * sizeof(T);
    tiny = ld * (int64_t)sizeof(T) < 16;
  }
  __device__ __forceinline__ bool apart() const {
    return MODE != WIDE && (at == first || at == last || tiny);
  }
  // What the bulk copy takes.
  __device__ __forceinline__ uintptr_t lo() const {
    return MODE == WIDE ? at : apart() ? (at + 15) & ~(uintptr_t)15 : at & ~(uintptr_t)15;
  }
  __device__ __forceinline__ uint32_t bytes() const {
    if (MODE == WIDE) return size;
    const uintptr_t from = lo(), to = apart() ? (at + size) & ~(uintptr_t)15 : (at + size + 15) & ~(uintptr_t)15;
    return to > from ? (uint32_t)(to - from) : 0;
  }
  // Elements apart: before the copy is announced, so that the announcement
  // publishes them.
  __device__ __noinline__ static void ends(uintptr_t at, uint32_t size, unsigned char* to) {
    const T* from = (const T*)at;
    T* p = (T*)(to + (at & 15));
    const uint32_t n = size / sizeof(T), up = (uint32_t)((16 - (at & 15)) & 15) / sizeof(T);
    const uint32_t head = up < n ? up : n, middle = (n - head) * sizeof(T) / 16 * 16 / sizeof(T);
    for (uint32_t i = 0; i < head; ++i) p[i] = from[i];
    for (uint32_t i = head + middle; i < n; ++i) p[i] = from[i];
  }
  __device__ __forceinline__ void prepare(unsigned char* to) const {
    if (apart()) ends(at, size, to);
  }
  __device__ __forceinline__ void start(Ring& q, unsigned char* to, int stage) {
    const uint32_t b = bytes();
    const uintptr_t from = lo();
    if (MODE == WIDE || b) q.copy(to + (from - (at & ~(uintptr_t)15)), (const void*)from, b, stage);
    at += step;
  }
};
// Where a row's elements are in its place.
template <typename T, int MODE>
__device__ __forceinline__ const T* row_at(const unsigned char* place, const T* m, int64_t ld, int64_t row) {
  return (const T*)(MODE == WIDE ? place : place + (uint32_t)((uintptr_t)(m + row * ld) & 15));
}
// A pack of the row from column c, elements outside it as `past`; `all`: none
// of the row's packs in this place is.
template <typename T, int V, int MODE>
__device__ __forceinline__ Pack<T, V> row_pack(const T* p, int c, int cols, T past, bool all) {
  Pack<T, V> v;
  if constexpr (V == 2 && MODE == ALIKE) {
    // (the word of column -1 or `cols` lies inside the row's place)
    if (all) return load_pack<T, V>(p + c);
    v.e[0] = v.e[1] = past;
    if (c < cols) {
      const Pack<T, V> q = load_pack<T, V>(p + c);
      if (c >= 0) v.e[0] = q.e[0];
      if (c + 1 < cols) v.e[1] = q.e[1];
    }
  } else if constexpr (V == 2) {
    v.e[0] = c < cols ? p[c] : past;
    v.e[1] = c + 1 < cols ? p[c + 1] : past;
  } else if constexpr (V * sizeof(T) == 16) {
    // by words: a choice per element would take 16-bit ones apart
    Pack<T, 4 / sizeof(T)> two;
#pragma unroll
    for (int i = 0; i < 4 / (int)sizeof(T); ++i) two.e[i] = past;
    const unsigned f = *reinterpret_cast<const unsigned*>(&two);
    uint4 q = make_uint4(f, f, f, f);
    if (c < cols) q = *reinterpret_cast<const uint4*>(p + c);
    *reinterpret_cast<uint4*>(&v) = q;
  } else {
    v.e[0] = c < cols ? p[c] : past;
  }
  return v;
}

// Warps that hold a row: the fewest that give each thread at most ROW_N
// elements; 0 where a row is too long for 32.
static int row_warps(int64_t cols) {
  for (int w : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32})
    if (cols <= (int64_t)32 * w * ROW_N) return w;
  return 0;
}

// Ring depth of a block whose rows take `row_bytes` a stage, beside `kept` more
// bytes, and blocks per SM: at most `most`, fewer where their shares of the
// shared memory would not hold two stages; 0 stages: not even one block's does.
constexpr int RING_BYTES = 220 << 10;
struct RingFit {
  int stages, per_sm;
};
static RingFit ring_fit(int64_t row_bytes, int rows, int64_t kept, int most) {
  for (int per_sm = most; per_sm >= 1; --per_sm) {
    const int64_t s = (RING_BYTES / per_sm - kept) / (row_bytes * rows);
    if (s >= 2) return {s < RING_MAX ? (int)s : RING_MAX, per_sm};
  }
  return {0, 1};
}

// Lets a kernel have the largest ring, once per device.
template <typename K>
static cudaError_t ring_smem(K kernel, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load()) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES);
  if (e == cudaSuccess) done[dev].store(true);
  return e;
}

// Rows a step apart that every block takes: even, so that a slot's rows all lie
// alike (first_shift).
static unsigned row_blocks(int64_t need, int64_t cap, int held, int mode) {
  int64_t g = need < cap ? need : cap;
  if (mode == ALIKE && g * held % 2) g = g + 1 <= cap || g == 1 ? g + 1 : g - 1;
  return (unsigned)g;
}

// How the rows of a call's matrices lie (see the modes above).
struct Rows {
  const void* p;
  int64_t ld;
};
static int row_mode(const Rows* m, int count, int64_t rows, int64_t cols, int size) {
  bool wide = true, alike = true;
  for (int i = 0; i < count; ++i) {
    wide &= rows_vec16(m[i].p, m[i].ld, cols, size);
    alike &= (((uintptr_t)m[i].p ^ (uintptr_t)m[0].p) & 2) == 0 && ((m[i].ld ^ m[0].ld) & 1) == 0;
  }
  return wide ? WIDE : size == 4 || alike ? ALIKE : APART;
}

}  // namespace repro
