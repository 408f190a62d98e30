// Gradient of the layer norm of each row, with h = (x - mean) rstd and
// g = dy weight:
//
//   dx = rstd (g - sum(g) / n - h sum(g h) / n)
//   dweight = sum over rows of dy h,   dbias = sum over rows of dy
//
// Sums are float32 on a topology fixed by the shape and the alignment (lanes,
// then warps, then blocks in order): no atomics, so the bits do not depend on
// scheduling.
#include "chain.cuh"
#include "row_norm.cuh"

namespace repro {

// A block walks its share of the rows; its threads keep their columns, so the
// weight's and bias's sums stay in registers and leave the block once, as one
// partial row each.  The number of blocks depends on the shape alone
// (ln_grad_shape), and so do the bits.
template <typename T, int MODE, int WARPS>
struct Backward {
  static constexpr int V = Access<T, MODE>::V;
  typedef RowShape<V, WARPS> RS;
  static constexpr int N = RS::N, U = RS::U;
  F2 aw[N / 2], ab[N / 2], hh[N / 2], g[N / 2];
  int t, slot, lane, warp, cols, shift;   // shift: see Forward
  float inv_n;

  __device__ __forceinline__ Backward(int c, const T* x, int64_t ldx) : cols(c), inv_n(1.0f / (float)c) {
    t = threadIdx.x % RS::T;
    slot = threadIdx.x / RS::T;
    lane = t & 31;
    warp = t >> 5;
    shift = first_shift<T, MODE>(x, ldx, slot, RS::ROWS);
#pragma unroll
    for (int h = 0; h < N / 2; ++h) aw[h] = ab[h] = 0;
  }
  __device__ __forceinline__ int col(int u) const { return (u * RS::T + t) * V - (MODE == ALIKE ? shift : 0); }
  __device__ __forceinline__ bool whole(int u) const { return (u + 1) * RS::T * V <= cols && (u > 0 || !shift); }
  // One pair: x and dy are zero outside the row, and with dy all its products.
  // (g feeds sums here and in store(): with its own rounding or, contracted,
  // without it; either is within the sums' error.)
  __device__ __forceinline__ void pair(int h, F2 x, F2 d, F2 w, F2 level, F2 width, F2& s0, F2& s1) {
    hh[h] = mul2(sub2(x, level), width);
    g[h] = mul2(d, w);
    s0 = add2(s0, g[h]);
    s1 = fma2(g[h], hh[h], s1);
    aw[h] = fma2(d, hh[h], aw[h]);
    ab[h] = add2(ab[h], d);
  }
  __device__ __forceinline__ void store(float s0, float s1, float rs, T* __restrict__ o) {
    const float a = s0 * inv_n, b = -(s1 * inv_n);
    const F2 ma = pk2(a, a), mb = pk2(b, b), width = pk2(rs, rs);
    Pack<T, V> out[U];
#pragma unroll
    for (int h = 0; h < N / 2; ++h) put2(out, h, mul2(fma2(hh[h], mb, sub2(g[h], ma)), width));
#pragma unroll
    for (int u = 0; u < U; ++u) store_in_row<T, V, MODE>(o, col(u), cols, lane, out[u]);
  }
  // The block's partial rows: weight's at 2 * blockIdx, bias's after it; its
  // rows' sums are added in order through `sum` ([2][COLS], unused for one row).
  __device__ __forceinline__ void leave(float* __restrict__ part, float* sum) {
    float* po = part + (size_t)blockIdx.x * 2 * cols;
#pragma unroll 1
    for (int k = 0; k < RS::ROWS; ++k) {
      if (slot == k) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int c = col(j / V) + j % V;
          if (c < 0) continue;
          float a0, a1, b0, b1;
          up2(aw[j / 2], a0, a1);
          up2(ab[j / 2], b0, b1);
          float a = j & 1 ? a1 : a0, b = j & 1 ? b1 : b0;
          if (k > 0) {
            a += sum[c];
            b += sum[RS::COLS + c];
          }
          if (k + 1 < RS::ROWS) {
            sum[c] = a;
            sum[RS::COLS + c] = b;
          } else if (c < cols) {
            po[c] = a;
            po[cols + c] = b;
          }
        }
      }
      if (RS::ROWS > 1) __syncthreads();
    }
  }
};

// x and dy side by side in a stage of the ring.
//
// Bound by DRAM and by the row's latency (one sum, two blocks per SM at 125
// registers: the columns' sums, h and g stay in registers).  32768 x 4096
// bfloat16: 136 us, 5.9 TB/s; 4096 x 4096 float32: 44 us, 4.6 TB/s with the 10 MB
// of partial rows written and read again, which the second kernel does in 3 us.
// Rows through registers 299 us, the weight read through the L1 cache 178.
template <typename T, int WARPS, int MODE>
__global__ void __launch_bounds__(RowShape<1, WARPS>::BLOCK, RowShape<1, WARPS>::BLOCK <= 256 ? 2 : 1)
    ln_backward(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                const T* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd, T* __restrict__ dx,
                int64_t lddx, float* __restrict__ part, int stages, TileError error) {
  chain_begin();
  constexpr int V = Access<T, MODE>::V;
  typedef RowShape<V, WARPS> RS;
  constexpr int U = RS::U;
  extern __shared__ __align__(128) unsigned char ring_bytes[];
  __shared__ __align__(16) float buf[2][RS::ROWS][2][WARPS];
  __shared__ __align__(8) uint64_t full[RS::ROWS][RING_MAX];
  Backward<T, MODE, WARPS> k(cols, x, ldx);
  const int64_t step = (int64_t)gridDim.x * RS::ROWS;
  int64_t r = (int64_t)blockIdx.x * RS::ROWS + k.slot;
  const uint32_t place = row_place(cols, sizeof(T), MODE);
  unsigned char* ring = ring_bytes + (size_t)k.slot * stages * 2 * place;
  Ring q(full[k.slot], stages, error);
  if (k.t == 0) q.init();
  T* vector = (T*)(ring_bytes + (size_t)RS::ROWS * stages * 2 * place);
  constexpr int FRONT = MODE == ALIKE && sizeof(T) == 2 ? 1 : 0;
  keep_vector(w, vector, cols, from_f32<T>(1.0f), FRONT);
  if (FRONT) {
    T* other = (T*)((unsigned char*)vector + vector_place(cols, sizeof(T), MODE));
    keep_vector(w, other, cols, from_f32<T>(1.0f), 0);
    vector = k.shift ? vector + 1 : other;
  }
  __syncthreads();
  RowCopies<T, MODE> nx(x, ldx, rows, cols, r, step), ny(dy, lddy, rows, cols, r, step);
  auto fill = [&](int s) {
    unsigned char* to = ring + s * 2 * place;
    nx.prepare(to);
    ny.prepare(to + place);
    q.expect(s, nx.bytes() + ny.bytes());
    nx.start(q, to, s);
    ny.start(q, to + place, s);
  };
  if (k.t == 0)
    for (int s = 0; s < stages && r + s * step < rows; ++s) fill(s);
  int64_t ahead = stages * step;
  int par = 0;
  float mu = 0.0f, rs = 0.0f;
  if (r < rows) mu = mean[r], rs = rstd[r];
  const T zero = from_f32<T>(0.0f);
  for (; r < rows; r += step, par ^= 1) {
    q.wait(ahead);
    const unsigned char* at = ring + q.s * 2 * place;
    const T *p = row_at<T, MODE>(at, x, ldx, r), *g = row_at<T, MODE>(at + place, dy, lddy, r);
    F2 s0 = 0, s1 = 0;
    const float rsr = rs;
    const F2 level = pk2(mu, mu), width = pk2(rs, rs);
    constexpr int UP = V > 1 ? 1 : 2;
#pragma unroll
    for (int u = 0; u < U; u += UP) {
      Pack<T, V> px[UP], py[UP], pw[UP];
#pragma unroll
      for (int i = 0; i < UP; ++i) {
        const int c = k.col(u + i);
        const bool all = k.whole(u + i);
        px[i] = row_pack<T, V, MODE>(p, c, cols, zero, all);
        py[i] = row_pack<T, V, MODE>(g, c, cols, zero, all);
        // (outside the row dy is zero, and the weight has to be finite)
        pw[i] = row_pack<T, V, MODE>(vector, c, cols, zero, all);
      }
#pragma unroll
      for (int j = 0; j < UP * V / 2; ++j)
        k.pair(u * V / 2 + j, elem2(px, j), elem2(py, j), elem2(pw, j), level, width, s0, s1);
    }
    if (r + step < rows) mu = mean[r + step], rs = rstd[r + step];
    float s[2] = {across(s0), across(s1)};
    row_sum<WARPS, 2>(s, buf[par][k.slot], k.warp, k.lane, k.slot);
    if (k.t == 0 && r + ahead < rows) fill(q.s);
    q.next();
    k.store(s[0], s[1], rsr, dx + r * lddx);
  }
  __syncthreads();
  // every copy has been waited for: the ring is free
  k.leave(part, (float*)ring_bytes);
}

// Rows longer than the ring holds (float32 past 11,260 columns, 16-bit past
// 16,384): a block per row, read twice, its column sums in global memory, one
// element an access.  Bound by the accesses: 2048 x 12288 float32 202 us, 1.5
// TB/s (2048 x 8192 with the ring 43, 4.7); 4096 x 32768 bfloat16 1342 us, 0.6 TB/s.
template <typename T>
__global__ void __launch_bounds__(LN_LONG_T)
    ln_backward_long(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, int64_t rows,
                     int64_t cols, const T* __restrict__ w, const float* __restrict__ mean,
                     const float* __restrict__ rstd, T* __restrict__ dx, int64_t lddx, float* __restrict__ part) {
  chain_begin();
  __shared__ __align__(16) float buf[2][2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float n = (float)cols;
  float* pw = part + (size_t)blockIdx.x * 2 * cols;
  int par = 0;
  bool any = false;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, par ^= 1) {
    const float mu = mean[r], rs = rstd[r];
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < cols; c += LN_LONG_T) {
      const float d = to_f32<T>(dy[r * lddy + c]), h = (to_f32<T>(x[r * ldx + c]) - mu) * rs;
      const float g = d * (w ? to_f32<T>(w[c]) : 1.0f);
      s[0] += g;
      s[1] = fmaf(g, h, s[1]);
      pw[c] = any ? fmaf(d, h, pw[c]) : d * h;
      pw[cols + c] = any ? pw[cols + c] + d : d;
    }
    any = true;
    row_sum<32, 2>(s, buf[par], warp, lane, 0);
    const float a = s[0] / n, b = s[1] / n;
    for (int64_t c = threadIdx.x; c < cols; c += LN_LONG_T) {
      const float d = to_f32<T>(dy[r * lddy + c]), h = (to_f32<T>(x[r * ldx + c]) - mu) * rs;
      const float g = d * (w ? to_f32<T>(w[c]) : 1.0f);
      dx[r * lddx + c] = from_f32<T>(rs * (fmaf(-h, b, g - a)));
    }
  }
}

// dweight and dbias from the blocks' partial rows: 32 columns and LN_SUM
// strands of rows per block, each strand in order, then the strands in order.
constexpr int LN_SUM = 16;

template <typename T>
__global__ void __launch_bounds__(32 * LN_SUM)
    ln_reduce(const float* __restrict__ part, int blocks, int64_t cols, T* __restrict__ dw, T* __restrict__ db) {
  chain_begin();
  __shared__ float buf[LN_SUM][33];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;   // columns of dweight, then of dbias
  float s = 0.0f;
  if (c < 2 * cols) {
#pragma unroll 4
    for (int p = k; p < blocks; p += LN_SUM) s += part[(size_t)p * 2 * cols + c];
  }
  buf[k][lane] = s;
  __syncthreads();
  if (k == 0 && c < 2 * cols) {
#pragma unroll
    for (int j = 1; j < LN_SUM; ++j) s += buf[j][lane];
    if (c < cols) {
      if (dw) dw[c] = from_f32<T>(s);
    } else if (db) {
      db[c - cols] = from_f32<T>(s);
    }
  }
}

// The gradient's grid: warps that hold a row (0: the long kernel), ring stages
// and blocks: a full GPU of 152 SMs, or fewer so that a block has about four
// rows for each that it holds at a time (a partial row costs as much to write
// and read as a row of the input).
struct LnGrad {
  int warps, stages;
  size_t ring;
  int64_t blocks;
};
static LnGrad ln_grad_shape(int mode, int64_t rows, int64_t cols, int size) {
  LnGrad g = {row_warps(cols + (mode == ALIKE && size == 2)), 0, 0, 0};
  int held = g.warps && g.warps < 8 ? 8 / g.warps : 1, per_sm = 1;
  if (g.warps) {
    const int64_t place = row_place(cols, size, mode);
    const int64_t kept = (int64_t)vector_copies(size, mode) * vector_place(cols, size, mode);
    const RingFit fit = ring_fit(2 * place, held, kept, 32 * g.warps * held <= 256 ? 2 : 1);
    per_sm = fit.per_sm;
    g.stages = fit.stages;
    g.ring = (size_t)g.stages * held * 2 * place + kept;
    // the ring also holds the block's sums of its rows
    const size_t sums = held > 1 ? (size_t)2 * 32 * g.warps * ROW_N * sizeof(float) : 0;
    if (g.ring < sums) g.ring = sums;
    if (!g.stages) g.warps = 0, held = per_sm = 1;
  }
  const int64_t most = 152 * per_sm, want = (rows + 4 * held - 1) / (4 * held);
  // (the long kernel has no slots that need an even step, and leaves a partial row for each block only if each has a row)
  g.blocks = g.warps ? row_blocks(want, most, held, mode) : want < most ? want : most;
  return g;
}

template <typename T, int MODE>
static cudaError_t ln_backward_pick(const T* dy, int64_t lddy, const T* x, int64_t ldx, int64_t rows, int64_t cols,
                                    const T* w, const float* mean, const float* rstd, T* dx, int64_t lddx, float* part,
                                    T* dw, T* db, TileError error, cudaStream_t s) {
  const LnGrad g = ln_grad_shape(MODE, rows, cols, sizeof(T));
  const unsigned blocks = (unsigned)g.blocks;
  Chain chain(s);
  cudaError_t e = cudaSuccess;
#define CASE(W)                                                                                              \
  case W: {                                                                                                  \
    static std::atomic<bool> done[64];                                                                       \
    if ((e = ring_smem(ln_backward<T, W, MODE>, done)) != cudaSuccess) return e;                             \
    e = chain.launch(ln_backward<T, W, MODE>, blocks, RowShape<1, W>::BLOCK, g.ring, dy, lddy, x, ldx, rows, \
                     (int)cols, w, mean, rstd, dx, lddx, part, g.stages, error);                             \
    break;                                                                                                   \
  }
  switch (g.warps) {
    CASE(1) CASE(2) CASE(3) CASE(4) CASE(6) CASE(8) CASE(12) CASE(16) CASE(24) CASE(32)
    default:
      e = chain.launch(ln_backward_long<T>, blocks, LN_LONG_T, 0, dy, lddy, x, ldx, rows, cols, w, mean, rstd, dx, lddx,
                       part);
  }
#undef CASE
  if (e != cudaSuccess) return e;
  return chain.launch(ln_reduce<T>, (unsigned)((2 * cols + 31) / 32), 32 * LN_SUM, 0, part, (int)g.blocks, cols, dw, db);
}

template <typename T>
static int ln_grad_mode(const T* dy, int64_t lddy, const T* x, int64_t ldx, int64_t rows, int64_t cols, const T* dx,
                        int64_t lddx) {
  const Rows m[3] = {{x, ldx}, {dy, lddy}, {dx, lddx}};
  return row_mode(m, 3, rows, cols, sizeof(T));
}

template <typename T>
size_t layer_norm_grad_workspace_bytes(const T* dy, int64_t lddy, const T* x, int64_t ldx, int64_t rows, int64_t cols,
                                       const T*, const T* dx, int64_t lddx) {
  const int mode = ln_grad_mode(dy, lddy, x, ldx, rows, cols, dx, lddx);
  return (size_t)ln_grad_shape(mode, rows, cols, sizeof(T)).blocks * 2 * (size_t)cols * sizeof(float);
}

template <typename T>
cudaError_t launch_layer_norm_grad(const T* dy, int64_t lddy, const T* x, int64_t ldx, int64_t rows, int64_t cols,
                                   const T* w, const float* mean, const float* rstd, T* dx, int64_t lddx, T* dw, T* db,
                                   float* part, TileError error, cudaStream_t s) {
  const int mode = ln_grad_mode(dy, lddy, x, ldx, rows, cols, dx, lddx);
  if (mode == WIDE)
    return ln_backward_pick<T, WIDE>(dy, lddy, x, ldx, rows, cols, w, mean, rstd, dx, lddx, part, dw, db, error, s);
  if constexpr (sizeof(T) == 2)
    if (mode == APART)
      return ln_backward_pick<T, APART>(dy, lddy, x, ldx, rows, cols, w, mean, rstd, dx, lddx, part, dw, db, error, s);
  return ln_backward_pick<T, ALIKE>(dy, lddy, x, ldx, rows, cols, w, mean, rstd, dx, lddx, part, dw, db, error, s);
}

#define INSTANTIATE(T)                                                                                             \
  template size_t layer_norm_grad_workspace_bytes<T>(const T*, int64_t, const T*, int64_t, int64_t, int64_t,       \
                                                     const T*, const T*, int64_t);                                 \
  template cudaError_t launch_layer_norm_grad<T>(const T*, int64_t, const T*, int64_t, int64_t, int64_t, const T*, \
                                                 const float*, const float*, T*, int64_t, T*, T*, float*,          \
                                                 TileError, cudaStream_t);
INSTANTIATE(float)
INSTANTIATE(__half)
INSTANTIATE(__nv_bfloat16)
#undef INSTANTIATE

}  // namespace repro
