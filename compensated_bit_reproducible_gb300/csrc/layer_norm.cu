// Layer norm of each row, and its gradient.
//
// Forward, the variance kernel's steps on a row held in registers: shift by
// the first element, local centring, two-term correction.
//
//   y = x - x[0];  m = sum(y) / n;  d = y - m
//   s1 = sum(d);   s2 = sum(d d);   var = max(s2 / n - (s1 / n)^2, 0)
//   mean = x[0] + m + s1 / n;       rstd = 1 / sqrt(var + eps)
//   out = (d - s1 / n) rstd weight + bias
//
// The shift keeps a row whose level is far above its width accurate: the sums
// see differences, which are exact within a factor of two of x[0].
//
// Sums are float32 on a topology fixed by the shape and the alignment (lanes,
// then warps in order): the bits do not depend on scheduling.
#include "row_norm.cuh"

namespace repro {

__device__ __forceinline__ float inverse_root(float v) {
  if (!(v > 0.0f) || v == INFINITY) return 1.0f / sqrtf(v);
  // one Newton step on the approximation: within an ulp
  const float r = rsqrtf(v);
  return fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
}

// The rest of a row once its shifted elements d = x - x0 and their sum are
// there; `in` is -1 where an element is inside the row and 0 past it.
template <typename T, int MODE, int WARPS>
struct Forward {
  static constexpr int V = Access<T, MODE>::V;
  typedef RowShape<V, WARPS> RS;
  static constexpr int N = RS::N, U = RS::U, INS = V > 1 ? U : N / 2;
  F2 in[INS];
  int t, slot, lane, warp, cols;
  int shift;   // ALIKE: 1 where this thread's rows start between words: its columns are one lower
  float inv_n;

  __device__ __forceinline__ Forward(int c, const T* x, int64_t ldx) : cols(c), inv_n(1.0f / (float)c) {
    t = threadIdx.x % RS::T;
    slot = threadIdx.x / RS::T;
    lane = t & 31;
    warp = t >> 5;
    shift = first_shift<T, MODE>(x, ldx, slot, RS::ROWS);
#pragma unroll
    for (int u = 0; u < INS; ++u) {
      // (V == 1: the pair's elements are packs 2 u and 2 u + 1)
      const int c0 = V > 1 ? col(u) : 2 * u * RS::T + t, c1 = V > 1 ? c0 + (V == 2) : c0 + RS::T;
      in[u] = pk2(c0 >= 0 && c0 < cols ? -1.0f : 0.0f, c1 < cols ? -1.0f : 0.0f);
    }
  }
  __device__ __forceinline__ int col(int u) const { return (u * RS::T + t) * V - (MODE == ALIKE ? shift : 0); }
  __device__ __forceinline__ bool whole(int u) const { return (u + 1) * RS::T * V <= cols && (u > 0 || !shift); }
  __device__ __forceinline__ F2 inside(int h) const { return in[V > 1 ? 2 * h / V : h]; }
  __device__ __forceinline__ void finish(F2 (&d)[N / 2], float sum, float x0, int64_t r, const T* w, const T* b,
                                         float eps, T* __restrict__ o,
                                         float* __restrict__ mean, float* __restrict__ rstd, float (*buf2)[WARPS]) {
    const float m = sum * inv_n;
    const F2 mm = pk2(m, m);
    F2 q1 = 0, q2 = 0;
#pragma unroll
    for (int h = 0; h < N / 2; ++h) {
      d[h] = fma2(inside(h), mm, d[h]);
      q1 = add2(q1, d[h]);
      q2 = fma2(d[h], d[h], q2);
    }
    float q[2] = {across(q1), across(q2)};
    row_sum<WARPS, 2>(q, buf2, warp, lane, slot);
    const float m1 = q[0] * inv_n;
    float var = fmaf(q[1], inv_n, -m1 * m1);
    if (var < 0.0f) var = 0.0f;   // a NaN stays
    const float rs = inverse_root(var + eps);
    if (t == 0) {
      mean[r] = x0 + (m + m1);
      rstd[r] = rs;
    }
    const F2 scale = pk2(rs, rs), off = pk2(-m1 * rs, -m1 * rs);
    // a pack at a time (single elements: a pair)
    constexpr int UP = V > 1 ? 1 : 2;
#pragma unroll
    for (int u0 = 0; u0 < U; u0 += UP) {
      Pack<T, V> pw[UP], pb[UP], out[UP];
#pragma unroll
      for (int k = 0; k < UP; ++k) {
        // (ALIKE: the vectors are kept so that column -shift is on a word)
        const int c = ((u0 + k) * RS::T + t) * V;
        if (c < cols + 1) {
          pw[k] = load_pack<T, V>(w + c);
          pb[k] = load_pack<T, V>(b + c);
        }
      }
#pragma unroll
      for (int j = 0; j < UP * V / 2; ++j)
        put2(out, j, fma2(fma2(d[u0 * V / 2 + j], scale, off), elem2(pw, j), elem2(pb, j)));
#pragma unroll
      for (int k = 0; k < UP; ++k) store_in_row<T, V, MODE>(o, col(u0 + k), cols, lane, out[k]);
    }
  }
};

// Each of the block's rows has a ring of `stages` rows in shared memory, filled
// by bulk copies.  A stage is free once its row's threads have met at the first
// sum's barrier.
//
// Bound by instruction issue (67% busy) and the two sums' latency: 320
// instructions a warp and row of 512 elements, of which about 110 for the sums.
// 32768 x 4096 bfloat16: 101 us, 5.3 TB/s; 4096 x 4096 float32: 27 us, 5.0 TB/s;
// without its sums the kernel reads and writes at 5.9 TB/s.  With 32 elements a
// thread 101 us too (half the warps, but fewer rows at a time); with 5 or 6
// blocks per SM 146 and 148 (spills); weight and bias read through the L1 cache
// 110; rows through registers 137, with 8 elements a thread 220.
template <typename T, int WARPS, int MODE>
__global__ void __launch_bounds__(RowShape<1, WARPS>::BLOCK,
                                  RowShape<1, WARPS>::BLOCK > 512 ? 1 : 1024 / RowShape<1, WARPS>::BLOCK)
    ln_forward(const T* __restrict__ x, int64_t ldx, int64_t rows, int cols, const T* __restrict__ w,
               const T* __restrict__ b, float eps,
               T* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd, int stages,
               TileError error) {
  constexpr int V = Access<T, MODE>::V;
  typedef RowShape<V, WARPS> RS;
  constexpr int N = RS::N, U = RS::U;
  extern __shared__ __align__(128) unsigned char ring_bytes[];
  __shared__ __align__(16) float buf1[RS::ROWS][1][WARPS], buf2[RS::ROWS][2][WARPS];
  __shared__ __align__(8) uint64_t full[RS::ROWS][RING_MAX];
  Forward<T, MODE, WARPS> f(cols, x, ldx);
  const int64_t step = (int64_t)gridDim.x * RS::ROWS;
  int64_t r = (int64_t)blockIdx.x * RS::ROWS + f.slot;
  const uint32_t place = row_place(cols, sizeof(T), MODE);
  unsigned char* ring = ring_bytes + (size_t)f.slot * stages * place;
  unsigned char* vectors = ring_bytes + (size_t)RS::ROWS * stages * place;
  Ring q(full[f.slot], stages, error);
  if (f.t == 0) q.init();
  // ALIKE: rows that start between words use the vectors one element on
  constexpr int FRONT = MODE == ALIKE && sizeof(T) == 2 ? 1 : 0;
  const uint32_t kept = vector_place(cols, sizeof(T), MODE);
  keep_vector(w, (T*)vectors, cols, from_f32<T>(1.0f), FRONT);
  keep_vector(b, (T*)(vectors + kept), cols, from_f32<T>(0.0f), FRONT);
  if (FRONT) {
    // and the others a copy of their own
    keep_vector(w, (T*)(vectors + 2 * kept), cols, from_f32<T>(1.0f), 0);
    keep_vector(b, (T*)(vectors + 3 * kept), cols, from_f32<T>(0.0f), 0);
    if (!f.shift) vectors += 2 * kept;
  }
  const T *w_at = (const T*)vectors, *b_at = (const T*)(vectors + kept);
  __syncthreads();
  RowCopies<T, MODE> next(x, ldx, rows, cols, r, step);
  auto fill = [&](int s) {
    unsigned char* to = ring + s * place;
    next.prepare(to);
    q.expect(s, next.bytes());
    next.start(q, to, s);
  };
  if (f.t == 0)
    for (int s = 0; s < stages && r + s * step < rows; ++s) fill(s);
  int64_t ahead = stages * step;
  for (; r < rows; r += step) {
    q.wait(ahead);
    const T* p = row_at<T, MODE>(ring + q.s * place, x, ldx, r);
    const T first = p[0];
    const float x0 = to_f32<T>(first);
    const F2 shift = pk2(x0, x0);
    F2 d[N / 2], acc = 0;
    // (an element past the row repeats the first: a zero after the shift)
    constexpr int UP = V > 1 ? 1 : 2;
#pragma unroll
    for (int u = 0; u < U; u += UP) {
      Pack<T, V> raw[UP];
#pragma unroll
      for (int k = 0; k < UP; ++k)
        raw[k] = row_pack<T, V, MODE>(p, f.col(u + k), cols, first, f.whole(u + k));
#pragma unroll
      for (int j = 0; j < UP * V / 2; ++j) {
        const int h = u * V / 2 + j;
        d[h] = sub2(elem2(raw, j), shift);
        acc = add2(acc, d[h]);
      }
    }
    float s[1] = {across(acc)};
    row_sum<WARPS, 1>(s, buf1[f.slot], f.warp, f.lane, f.slot);
    if (f.t == 0 && r + ahead < rows) fill(q.s);
    q.next();
    f.finish(d, s[0], x0, r, w_at, b_at, eps, y + r * ldy, mean, rstd, buf2[f.slot]);
  }
}

// Rows longer than the ring or the registers hold (float32 past 14,076 columns,
// 16-bit past 16,384): one block per row, the row read three times (from L2 after
// the first), one element an access.  2048 x 16384 float32: 77 us, 3.5 TB/s (2048 x
// 12288 with the ring 41, 5.0); 4096 x 32768 bfloat16: 224 us, 2.4 TB/s.
template <typename T>
__global__ void __launch_bounds__(LN_LONG_T)
    ln_forward_long(const T* __restrict__ x, int64_t ldx, int64_t rows, int cols, const T* __restrict__ w,
                    const T* __restrict__ b, float eps, T* __restrict__ y, int64_t ldy, float* __restrict__ mean,
                    float* __restrict__ rstd) {
  __shared__ __align__(16) float buf1[1][32], buf2[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float n = (float)cols;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* p = x + r * ldx;
    const float x0 = to_f32<T>(p[0]);
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < cols; c += LN_LONG_T) s[0] += to_f32<T>(p[c]) - x0;
    row_sum<32, 1>(s, buf1, warp, lane, 0);
    const float m = s[0] / n;
    float q[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < cols; c += LN_LONG_T) {
      const float d = (to_f32<T>(p[c]) - x0) - m;
      q[0] += d;
      q[1] = fmaf(d, d, q[1]);
    }
    row_sum<32, 2>(q, buf2, warp, lane, 0);
    const float m1 = q[0] / n;
    float var = q[1] / n - m1 * m1;
    if (var < 0.0f) var = 0.0f;
    const float rs = 1.0f / sqrtf(var + eps);
    if (threadIdx.x == 0) {
      mean[r] = x0 + (m + m1);
      rstd[r] = rs;
    }
    T* o = y + r * ldy;
    for (int64_t c = threadIdx.x; c < cols; c += LN_LONG_T) {
      const float g = w ? to_f32<T>(w[c]) : 1.0f, h = b ? to_f32<T>(b[c]) : 0.0f;
      o[c] = from_f32<T>(fmaf((((to_f32<T>(p[c]) - x0) - m) - m1) * rs, g, h));
    }
  }
}

template <typename T, int MODE>
static cudaError_t ln_forward_pick(const T* x, int64_t ldx, int64_t rows, int64_t cols, const T* w, const T* b,
                                   float eps, T* y, int64_t ldy, float* mean, float* rstd, int sms, TileError error,
                                   cudaStream_t s) {
  const int64_t place = row_place(cols, sizeof(T), MODE);
  const int64_t kept = (int64_t)2 * vector_copies(sizeof(T), MODE) * vector_place(cols, sizeof(T), MODE);
#define CASE(W)                                                                                                      \
  case W: {                                                                                                          \
    typedef RowShape<1, W> RS;                                                                                       \
    const RingFit fit = ring_fit(place, RS::ROWS, kept, RS::BLOCK > 512 ? 1 : 1024 / RS::BLOCK);                     \
    if (!fit.stages) break;                                                                                          \
    static std::atomic<bool> done[64];                                                                               \
    cudaError_t e = ring_smem(ln_forward<T, W, MODE>, done);                                                         \
    if (e != cudaSuccess) return e;                                                                                  \
    const unsigned grid = row_blocks((rows + RS::ROWS - 1) / RS::ROWS, (int64_t)sms * fit.per_sm, RS::ROWS, MODE);   \
    ln_forward<T, W, MODE><<<grid, RS::BLOCK, fit.stages * RS::ROWS * place + kept, s>>>(                            \
        x, ldx, rows, (int)cols, w, b, eps, y, ldy, mean, rstd, fit.stages, error);                                  \
    return cudaGetLastError();                                                                                       \
  }
  // (an element more than the row where it starts between words)
  switch (row_warps(cols + (MODE == ALIKE && sizeof(T) == 2))) {
    CASE(1) CASE(2) CASE(3) CASE(4) CASE(6) CASE(8) CASE(12) CASE(16) CASE(24) CASE(32)
  }
#undef CASE
  const int64_t most = 2 * (int64_t)sms;
  ln_forward_long<T><<<(unsigned)(rows < most ? rows : most), LN_LONG_T, 0, s>>>(x, ldx, rows, (int)cols, w, b, eps, y,
                                                                             ldy, mean, rstd);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_layer_norm(const T* x, int64_t ldx, int64_t rows, int64_t cols, const T* w, const T* b, float eps,
                              T* y, int64_t ldy, float* mean, float* rstd, int sms, TileError error, cudaStream_t s) {
  const Rows m[2] = {{x, ldx}, {y, ldy}};
  const int mode = row_mode(m, 2, rows, cols, sizeof(T));
  if (mode == WIDE)
    return ln_forward_pick<T, WIDE>(x, ldx, rows, cols, w, b, eps, y, ldy, mean, rstd, sms, error, s);
  if constexpr (sizeof(T) == 2)
    if (mode == APART)
      return ln_forward_pick<T, APART>(x, ldx, rows, cols, w, b, eps, y, ldy, mean, rstd, sms, error, s);
  return ln_forward_pick<T, ALIKE>(x, ldx, rows, cols, w, b, eps, y, ldy, mean, rstd, sms, error, s);
}

#define INSTANTIATE(T)                                                                                          \
  template cudaError_t launch_layer_norm<T>(const T*, int64_t, int64_t, int64_t, const T*, const T*, float, T*, \
                                            int64_t, float*, float*, int, TileError, cudaStream_t);
INSTANTIATE(float)
INSTANTIATE(__half)
INSTANTIATE(__nv_bfloat16)
#undef INSTANTIATE

}  // namespace repro
