// Softmax cross entropy of a linear layer over a large vocabulary, and its
// gradient, in pieces of the vocabulary: the logits are never kept.
//
//   z = h weight^T                              [n, vocab]
//   lse[t] = log sum_v exp z[t, v],   loss[t] = lse[t] - z[t, label[t]]
//   g[t, v] = (exp(z[t, v] - lse[t]) - [v = label[t]]) dloss[t]
//   dh = g weight,   dweight = g^T h
//
// Forward: tiles of z stay in tensor memory; each thread reduces 128 columns
// of one row to (maximum, sum of exponentials), and a second kernel joins the pieces
// of a row in order.  Gradient, for each piece of the vocabulary: the tiles of
// z again, turned into g in 16 bits, then the two products that read it.  g is
// held for dloss over the largest |dloss|, times 2^14, so that it keeps its
// precision in half's range and equal dloss are exactly 1 (see xent_scale); the
// products are scaled back.
//
// Bound by the tensor cores and, over milliseconds, by the power limit: loss and
// gradient of 8192 x 32768 x 2048 bfloat16 take 2.73 to 2.83 ms for four products
// (the logits twice), 1.55 to 1.61 PFLOP/s.  A half of the vocabulary (16384 columns): g 304
// us, dh 351 (256 tiles are 3.4 rounds of 76 pairs), dweight 306.
//
// Every tile's inner dimension is walked in order and nothing is added by
// atomics: the bits depend on values and shapes alone.  Statistics, products
// and the sums over pieces are float32; g is the only value rounded to 16 bits
// on the way, which is what the tensor cores multiply, and costs the gradients
// about as much as their own final rounding.
#include <atomic>
#include "elem.cuh"
#include "launch.h"
#include "tile_gemm.cuh"

namespace repro {

constexpr float LOG2E = 1.44269504088896341f;

// ------------------------------------------------------------- epilogues
// Their instructions are not free although they run beside the products: at
// full rate the GPU is at its power limit, and what they draw the tensor cores
// lack.  So: pairs, the hardware's exponential alone, rare cases apart.

// 2^x, relative error below 2^-22; 0 below 2^-126 (a share of less than that in
// a sum of at least 1, or a gradient below any type's range).
__device__ __forceinline__ float power2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ F2 power2(F2 x) {
  float a, b;
  up2(x, a, b);
  return pk2(power2(a), power2(b));
}
__device__ __forceinline__ float lane_of(const F2* v, int i) {
  float a, b;
  up2(v[i / 2], a, b);
  return i & 1 ? b : a;
}

// Maximum m and sum of exp(z - m) of half a tile's columns.  The difference is
// taken before the factor of 2^x: it is exact near the maximum, so the largest
// logit's share is exactly 1 whatever its size, and a sum at least 1.  (With one
// fma for both, m log2(e) is rounded: the loss of a sure row is then that rounding,
// and logits past 2^31 give an infinite lse.  4096 x 32768 x 1024 bfloat16: 165 us
// with the fma, 166.5 so.)
struct EpiStats {
  const int64_t* label;
  float2* part;      // [halves of tiles][n]
  float* zlabel;     // [n]: the label's logit
  int n, vocab;
  struct State {
    int64_t label;
    float m, s;
  };
  __device__ __forceinline__ void row(int row, State& st) const {
    st.label = row < n ? label[row] : -1;
    st.m = -INFINITY;
    st.s = 0.0f;
  }
  __device__ __forceinline__ void chunk(int row, int col, F2* v, State& st, const Place&) const {
    if (col + 32 > vocab)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = pk2(col + 2 * i < vocab ? lane_of(v, 2 * i) : -INFINITY,
                   col + 2 * i + 1 < vocab ? lane_of(v, 2 * i + 1) : -INFINITY);
    if (st.label >= col && st.label < col + 32) {
      const int at = (int)(st.label - col);
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (at == i) z = lane_of(v, i);
      if (st.label < vocab) zlabel[row] = z;
    }
    float m[2] = {lane_of(v, 0), lane_of(v, 1)};
#pragma unroll
    for (int i = 1; i < 16; ++i) m[i & 1] = fmaxf(fmaxf(m[i & 1], lane_of(v, 2 * i)), lane_of(v, 2 * i + 1));
    const float top = fmaxf(st.m, fmaxf(m[0], m[1]));
    const float base = top == -INFINITY ? 0.0f : top;   // nothing but -inf so far: 2^(-inf - 0) = 0
    const F2 scale = pk2(LOG2E, LOG2E), off = pk2(base, base);
    F2 s[2] = {pk2(st.s * power2((st.m - base) * LOG2E), 0.0f), 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i & 1] = add2(s[i & 1], power2(mul2(sub2(v[i], off), scale)));
    float a, b;
    up2(add2(s[0], s[1]), a, b);
    st.s = a + b;
    st.m = top;
  }
  __device__ __forceinline__ void done(int row, State& st, const Place& at) const {
    if (row < n) part[(size_t)(2 * at.tile + at.half) * n + row] = make_float2(st.m, st.s);
  }
};

// g of one piece of the vocabulary, in 16 bits.
template <typename T>
struct EpiGrad {
  const int64_t* label;
  const float* lse;
  const float* dloss;
  const float* scale;   // [0]: the largest finite |dloss|, [1]: a power of two
  T* g;                 // [n][ldg]
  int64_t ldg;
  int n, width, v0, vocab;   // columns of the piece, its first token
  struct State {
    float lse, d;
    int at;   // the label's column in the piece, or -1
  };
  __device__ __forceinline__ void row(int row, State& st) const {
    st.lse = 0.0f;
    st.d = 0.0f;
    st.at = -1;
    if (row < n) {
      const int64_t l = label[row];
      if (l >= 0) {
        st.lse = lse[row];
        st.d = l < vocab ? __fdiv_rn(dloss[row], scale[0]) * scale[1] : __uint_as_float(0x7fc00000u);
        st.at = l >= v0 && l < v0 + (int64_t)width ? (int)(l - v0) : -1;
      } else {
        st.at = -2;   // no label: the row of g is zero whatever the logits are
      }
    }
  }
  __device__ __forceinline__ void chunk(int, int col, F2* v, State& st, const Place& at) const {
    if (col >= width) return;
    // (the difference first, as in the loss: a rounding of lse log2(e) would be an exponent's error past 2^24)
    const F2 scale = pk2(LOG2E, LOG2E), off = pk2(st.lse, st.lse), d = pk2(st.d, st.d);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = power2(mul2(sub2(v[i], off), scale));
    const int hit = st.at - col;
    if (hit >= 0 && hit < 32)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = pk2(lane_of(v, 2 * i) - (hit == 2 * i ? 1.0f : 0.0f),
                   lane_of(v, 2 * i + 1) - (hit == 2 * i + 1 ? 1.0f : 0.0f));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = mul2(v[i], d);
    // ldg is a multiple of 32: whole runs fit, what lies past the piece is never read
    put_rows<T>(v, at.stage, at.lane, g, ldg, at.row0, n, col, (int)ldg, true, st.at == -2 ? 0u : ~0u);
  }
  __device__ __forceinline__ void done(int, State&, const Place&) const {}
};

// Rows of a gradient: rounded to the output, or float32 sums of a range of the
// inner dimension, over the pieces of the vocabulary.
template <typename T>
struct EpiOut {
  float* sum;           // [splits][rows][lds] or null
  int64_t lds;          // a multiple of 32
  int add;              // sum holds earlier pieces
  const float* scale;   // [0]: the largest finite |dloss|, [2]: the inverse power of two
  T* out;
  int64_t ldo;
  int rows, cols, wide;   // wide: rows of out are 16-byte aligned
  struct State {
    float inv, top;
  };
  __device__ __forceinline__ void row(int, State& st) const {
    st.inv = sum ? 1.0f : scale[2];
    st.top = sum ? 1.0f : scale[0];
  }
  __device__ __forceinline__ void chunk(int row, int col, F2* v, State& st, const Place& at) const {
    if (col >= cols) return;
    if (!sum) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = mul2(mul2(v[i], pk2(st.inv, st.inv)), pk2(st.top, st.top));
      put_rows<T>(v, at.stage, at.lane, out, ldo, at.row0, rows, col, cols, wide);
      return;
    }
    if (row >= rows) return;
    float* p = sum + ((size_t)at.split * rows + row) * lds + col;
    if (add)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Pack<float, 4> q = load_pack<float, 4>(p + 4 * j);
        v[2 * j] = add2(v[2 * j], get2(q, 0));
        v[2 * j + 1] = add2(v[2 * j + 1], get2(q, 1));
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      Pack<float, 4> q;
      set2(q, 0, v[2 * j]);
      set2(q, 1, v[2 * j + 1]);
      store_pack<float, 4>(p + 4 * j, q);
    }
  }
  __device__ __forceinline__ void done(int, State&, const Place&) const {}
};

// --------------------------------------------------------- small kernels
// The pieces of each row joined: strand k of a row takes pieces k, k + 8, ...,
// the strands are joined in order.  *error (a tile gave up) makes NaN.
__global__ void __launch_bounds__(256) xent_join(const float2* __restrict__ part, int slots, int n, int vocab,
                                                 const int64_t* __restrict__ label, const float* __restrict__ zlabel,
                                                 float* __restrict__ loss, float* __restrict__ lse,
                                                 const int* error) {
  chain_begin();
  __shared__ float2 buf[8][33];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.0f;
  auto join = [&](float2 p) {
    const float top = fmaxf(m, p.x), base = top == -INFINITY ? 0.0f : top;
    s = s * exp2f((m - base) * LOG2E) + p.y * exp2f((p.x - base) * LOG2E);
    m = top;
  };
  if (row < n)
#pragma unroll 4
    for (int i = k; i < slots; i += 8) join(part[(size_t)i * n + row]);
  buf[k][lane] = make_float2(m, s);
  __syncthreads();
  if (k || row >= n) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) join(buf[j][lane]);
  const bool ok = !*(volatile const int*)error;
  const float nan = __uint_as_float(0x7fc00000u), above = ok ? logf(s) : nan;   // lse - m, at least 0
  lse[row] = m + above;
  const int64_t id = label[row];
  // (not lse - z: that has lost what is small beside m)
  loss[row] = id < 0 ? 0.0f : id >= vocab ? nan : (m - zlabel[row]) + above;
}

// scale[0] = the largest finite |dloss|, scale[1] = 2^14, scale[2] = 2^-14; 1
// where there is nothing to scale by.  (An infinity or a NaN stays one at any
// scale, and the other rows keep theirs.)  The largest itself, not a power of two near it:
// where all rows have the same dloss (a mean) their quotient is exactly 1, the
// label's element p - 1 is off by p at most in 16 bits, and no rounding of dloss
// is shared by all rows.
__global__ void __launch_bounds__(1024) xent_scale(const float* __restrict__ dloss, const int64_t* __restrict__ label,
                                                   int n, float* __restrict__ scale) {
  chain_begin();
  __shared__ unsigned top[32];
  unsigned m = 0;
  for (int i = threadIdx.x; i < n; i += 1024)
    if (label[i] >= 0) {
      const unsigned a = __float_as_uint(fabsf(dloss[i]));
      if (a < 0x7f800000u) m = max(m, a);
    }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 32; ++i) m = max(m, top[i]);
    const bool any = m != 0;
    scale[0] = any ? __uint_as_float(m) : 1.0f;
    scale[1] = any ? 0x1p14f : 1.0f;
    scale[2] = any ? 0x1p-14f : 1.0f;
  }
}

// Rows copied to a base and stride that TMA takes: a thread writes eight
// elements, read as the five aligned words that hold them.
template <typename T>
__global__ void __launch_bounds__(256) xent_pack(const T* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                                                 T* __restrict__ y, int ldy) {
  chain_begin();
  const int vpr = ldy / 8;
  const int64_t packs = rows * vpr;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < packs; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / vpr;
    const int c = (int)(i - r * vpr) * 8;
    const T* p = x + r * ldx + c;
    Pack<T, 8> v = {};
    if (c + 8 <= cols) {
      const unsigned odd = ((uintptr_t)p >> 1) & 1;
      const unsigned* q = (const unsigned*)((uintptr_t)p & ~(uintptr_t)3);
      unsigned w[5];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = q[k];
      w[4] = odd ? q[4] : 0;   // holds the last element only of an odd start
      unsigned* o = (unsigned*)&v;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(w[k], w[k + 1], odd * 16);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < cols) v.e[k] = p[k];
    }
    store_pack<T, 8>(y + r * ldy + c, v);
  }
}

// out = the splits' sums, added in order, with g's scale taken out.
template <typename T>
__global__ void __launch_bounds__(256) xent_sum(const float* __restrict__ sum, int splits, int64_t rows, int cols,
                                                int64_t lds, const float* __restrict__ scale, T* __restrict__ out,
                                                int64_t ldo) {
  chain_begin();
  const float top = scale[0], inv = scale[2];
  const int64_t quads = lds / 4, all = rows * quads;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / quads;
    const int c = (int)(i - r * quads) * 4;
    if (c >= cols) continue;
    Pack<float, 4> v = load_pack<float, 4>(sum + r * lds + c);
    for (int s = 1; s < splits; ++s) {
      const Pack<float, 4> q = load_pack<float, 4>(sum + ((size_t)s * rows + r) * lds + c);
#pragma unroll
      for (int k = 0; k < 4; ++k) v.e[k] += q.e[k];
    }
    T* o = out + r * ldo + c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < cols) o[k] = from_f32<T>(v.e[k] * inv * top);
  }
}

// --------------------------------------------------------------- host side
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// Map of a row-major matrix whose boxes are 64 columns by `box_rows` rows.
template <typename T>
static cudaError_t make_map(CUtensorMap* map, const T* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorSymbolNotFound;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * sizeof(T)};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
  const CUtensorMapDataType dt =
      std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(map, dt, 2, (void*)p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <typename T, bool AMN, bool BMN, typename E>
static cudaError_t run_tiles(const CUtensorMap& a, const CUtensorMap& b, const TileShape& sh, const E& epi, TileError error,
                             Chain& chain) {
  auto kernel = tile_gemm<std::is_same<T, __nv_bfloat16>::value, AMN, BMN, E>;
  static std::atomic<int> pairs[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!pairs[dev].load()) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TG_SMEM)) != cudaSuccess)
      return e;
    // as many pairs as can be resident: the tiles are dealt out to them
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(TG_THREADS);
    cfg.dynamicSmemBytes = TG_SMEM;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int c = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&c, kernel, &cfg)) != cudaSuccess) return e;
    if (c < 1) return cudaErrorInvalidConfiguration;
    pairs[dev].store(c);
  }
  const int64_t tiles = sh.tiles(), all = pairs[dev].load(), use = tiles < all ? tiles : all;
  if (tiles > TILES_MAX) return cudaErrorInvalidValue;
  return chain.launch(kernel, (unsigned)(2 * use), TG_THREADS, TG_SMEM, a, b, sh, epi, error);
}

// An operand as TMA takes it: the caller's memory, or a packed copy in `ws`.
template <typename T>
struct Operand {
  const T* p;
  int64_t ld;
  bool copied;
};
template <typename T>
static Operand<T> operand(const T* p, int64_t ld, int64_t rows, int64_t cols) {
  // one row has no stride of its own: any multiple of 16 bytes will do
  if (((uintptr_t)p & 15u) == 0 && rows <= 1) return {p, (cols + 7) / 8 * 8, false};
  if (((uintptr_t)p & 15u) == 0 && ld % 8 == 0) return {p, ld, false};
  return {nullptr, (cols + 7) / 8 * 8, true};
}
template <typename T>
static cudaError_t pack_operand(Operand<T>& o, const T* p, int64_t ld, int64_t rows, int64_t cols, T* to,
                                Chain& chain) {
  const int64_t blocks = (rows * (o.ld / 8) + 255) / 256;
  o.p = to;
  return chain.launch(xent_pack<T>, (unsigned)(blocks < 152 * 32 ? blocks : 152 * 32), 256, 0, p, ld, rows, (int)cols,
                      to, (int)o.ld);
}

static size_t up1k(size_t x) { return (x + 1023) & ~(size_t)1023; }

// Columns of a piece of the vocabulary in the gradient: g takes at most
// XENT_PIECE bytes.  Pieces get narrow as rows get many, and dh's float32 sums are
// read and written once a piece: 8192 rows of 32768 x 2048 run at 1.68 PFLOP/s (6
// n vocab cols operations), 32768 rows at 1.39, 131072 rows of 32768 x 1024 at 1.03.
constexpr size_t XENT_PIECE = 256u << 20;
static int64_t piece_width(int64_t n, int64_t vocab) {
  int64_t w = (int64_t)(XENT_PIECE / 2 / (size_t)n) / 256 * 256;
  if (w < 256) w = 256;
  return w < vocab ? w : vocab;
}

static int64_t up32(int64_t x) { return (x + 31) / 32 * 32; }

// The shapes below come from the product's sizes alone, for a GPU of 76 pairs,
// so that the bits do not depend on how many are free.
constexpr int64_t PAIRS = 76;

// Columns of a tile: equal tiles of at most 256, or smaller ones where 256
// would leave pairs without work.
static int tile_cols(int64_t m, int64_t n, bool fill) {
  const int64_t mt = (m + TG_M - 1) / TG_M;
  int64_t nt = (n + TG_N - 1) / TG_N;
  if (fill && mt * nt < PAIRS) nt = PAIRS / mt > nt ? PAIRS / mt : nt;
  const int64_t tn = up32((n + nt - 1) / nt);
  return (int)(tn < TG_N ? tn : TG_N);
}

// Ranges of the inner dimension: the number that costs least, in steps of a
// tile (256 x 256 x 64, 0.27 us at 1.9 PFLOP/s of 76 pairs): rounds of tiles, each
// with a few steps of filling, and each range's float32 sums written and read
// again.  The gradient in us with one number for both its products, and by the
// rule:
//                                     1     2     4     8    16   rule
//   float16   1003 x 20011 x  777   204   214   266   426   739   137
//   bfloat16   256 x 32768 x 1024   218   294   406   388   381    85
//               64 x 50000 x  512   291   174   115    85    72    72
//             2048 x 32768 x 1024   340   395   542   860  1480   275
//             8192 x  2048 x  256    85    75    73    92   142    61
//             4096 x 32768 x 2048   953  1179  1407  1989  3293   954
static int split_count(int64_t m, int64_t n, int tn, int64_t k, bool carried) {
  const int64_t tiles = ((m + TG_M - 1) / TG_M) * ((n + tn - 1) / tn), kb = (k + TG_K - 1) / TG_K;
  const double traffic = (double)m * n * 8 / 1.6e6;   // bytes of a step's time at 6 TB/s
  int best = 1;
  double least = 0;
  for (int s = 1; s <= 16 && kb / s >= 8; ++s) {
    const double rounds = (double)((tiles * s + PAIRS - 1) / PAIRS);
    const double cost = rounds * ((double)kb / s * tn / 256 + 8) + (s > 1 || carried ? s * traffic : 0);
    if (s == 1 || cost < 0.95 * least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

// Orders of the tiles: the logits go through all rows of h for each tile of the
// vocabulary (a tile's weights are read once; 608 us against 618 for 8192 x
// 32768 x 2048), the products that read g in bands of 8 (305 against 331 us for
// half of dweight).
constexpr int BAND = 8, BAND_ALL = 0x7fffffff;

// How the gradient of one shape is computed.
struct XentPlan {
  int64_t pw, ldg, lds;     // columns of a piece, row strides of g and of the sums
  int tn, splits_h, splits_w;
  bool sum_h, sum_w;
};
static XentPlan xent_plan(int64_t n, int64_t vocab, int64_t cols) {
  XentPlan p;
  p.pw = piece_width(n, vocab);
  p.ldg = up32(p.pw);
  p.lds = up32(cols);
  p.tn = tile_cols(n, cols, false);
  p.splits_h = split_count(n, cols, p.tn, p.pw, p.pw < vocab);
  p.splits_w = split_count(p.pw, cols, p.tn, n, false);
  p.sum_h = p.splits_h > 1 || p.pw < vocab;
  p.sum_w = p.splits_w > 1;
  return p;
}

struct XentWs {
  size_t h, w, part, zlabel, scale, g, sum_h, sum_w, bytes;
};
template <typename T>
static XentWs xent_ws(const T* h, int64_t ldh, const T* w, int64_t ldw, int64_t n, int64_t vocab, int64_t cols,
                      bool grad) {
  XentWs x = {};
  size_t at = 0;
  auto take = [&](size_t b) {
    const size_t p = at;
    at += up1k(b);
    return p;
  };
  const Operand<T> oh = operand(h, ldh, n, cols), ow = operand(w, ldw, vocab, cols);
  x.h = take(oh.copied ? (size_t)n * oh.ld * sizeof(T) : 0);
  x.w = take(ow.copied ? (size_t)vocab * ow.ld * sizeof(T) : 0);
  x.scale = take(16);
  if (!grad) {
    const int64_t tn = tile_cols(n, vocab, true);
    x.part = take((size_t)(2 * ((vocab + tn - 1) / tn)) * n * sizeof(float2));
    x.zlabel = take((size_t)n * 4);
  } else {
    const XentPlan p = xent_plan(n, vocab, cols);
    x.g = take((size_t)n * p.ldg * sizeof(T));
    x.sum_h = take(p.sum_h ? (size_t)p.splits_h * n * p.lds * 4 : 0);
    x.sum_w = take(p.sum_w ? (size_t)p.splits_w * p.pw * p.lds * 4 : 0);
  }
  x.bytes = at;
  return x;
}

template <typename T>
size_t linear_xent_workspace_bytes(const T* h, int64_t ldh, const T* w, int64_t ldw, int64_t n, int64_t vocab,
                                   int64_t cols, bool grad) {
  return xent_ws<T>(h, ldh, w, ldw, n, vocab, cols, grad).bytes;
}

template <typename T>
cudaError_t launch_linear_xent(const T* h, int64_t ldh, const T* w, int64_t ldw, const int64_t* label, int64_t n,
                               int64_t vocab, int64_t cols, float* loss, float* lse, unsigned char* ws, TileError error,
                               cudaStream_t s) {
  const XentWs x = xent_ws<T>(h, ldh, w, ldw, n, vocab, cols, false);
  Operand<T> oh = operand(h, ldh, n, cols), ow = operand(w, ldw, vocab, cols);
  Chain chain(s);
  cudaError_t e;
  if (oh.copied && (e = pack_operand(oh, h, ldh, n, cols, (T*)(ws + x.h), chain)) != cudaSuccess) return e;
  if (ow.copied && (e = pack_operand(ow, w, ldw, vocab, cols, (T*)(ws + x.w), chain)) != cudaSuccess) return e;
  const int tn = tile_cols(n, vocab, true);
  CUtensorMap mh, mw;
  if ((e = make_map<T>(&mh, oh.p, n, cols, oh.ld, 128)) != cudaSuccess) return e;
  if ((e = make_map<T>(&mw, ow.p, vocab, cols, ow.ld, tn / 2)) != cudaSuccess) return e;
  EpiStats epi{label, (float2*)(ws + x.part), (float*)(ws + x.zlabel), (int)n, (int)vocab};
  const TileShape sh{(int)n, (int)vocab, (int)cols, tn, 1, 0, 0, BAND_ALL};
  if ((e = run_tiles<T, false, false>(mh, mw, sh, epi, error, chain)) != cudaSuccess) return e;
  return chain.launch(xent_join, (unsigned)((n + 31) / 32), 256, 0, epi.part, 2 * sh.nt(), (int)n, (int)vocab, label,
                      epi.zlabel, loss, lse, error.device);
}

// out from the splits' sums.
template <typename T>
static cudaError_t run_sum(const float* sum, int splits, int64_t rows, int64_t cols, int64_t lds, const float* scale,
                           T* out, int64_t ldo, Chain& chain) {
  const int64_t blocks = (rows * (lds / 4) + 255) / 256;
  return chain.launch(xent_sum<T>, (unsigned)(blocks < 152 * 16 ? blocks : 152 * 16), 256, 0, sum, splits, rows,
                      (int)cols, lds, scale, out, ldo);
}

template <typename T>
cudaError_t launch_linear_xent_grad(const float* dloss, const T* h, int64_t ldh, const T* w, int64_t ldw,
                                    const int64_t* label, const float* lse, int64_t n, int64_t vocab, int64_t cols,
                                    T* dh, int64_t lddh, T* dw, int64_t lddw, unsigned char* ws, TileError error,
                                    cudaStream_t s) {
  const XentWs x = xent_ws<T>(h, ldh, w, ldw, n, vocab, cols, true);
  Operand<T> oh = operand(h, ldh, n, cols), ow = operand(w, ldw, vocab, cols);
  Chain chain(s);
  cudaError_t e;
  if (oh.copied && (e = pack_operand(oh, h, ldh, n, cols, (T*)(ws + x.h), chain)) != cudaSuccess) return e;
  if (ow.copied && (e = pack_operand(ow, w, ldw, vocab, cols, (T*)(ws + x.w), chain)) != cudaSuccess) return e;
  float* scale = (float*)(ws + x.scale);
  if ((e = chain.launch(xent_scale, 1, 1024, 0, dloss, label, (int)n, scale)) != cudaSuccess) return e;
  const XentPlan p = xent_plan(n, vocab, cols);
  T* g = (T*)(ws + x.g);
  float* sum_h = p.sum_h ? (float*)(ws + x.sum_h) : nullptr;
  float* sum_w = p.sum_w ? (float*)(ws + x.sum_w) : nullptr;
  CUtensorMap mh, hm, wm;   // as rows of a product (128-row boxes), and as its inner dimension
  if ((e = make_map<T>(&mh, oh.p, n, cols, oh.ld, 128)) != cudaSuccess) return e;
  if ((e = make_map<T>(&hm, oh.p, n, cols, oh.ld, TG_K)) != cudaSuccess) return e;
  if ((e = make_map<T>(&wm, ow.p, vocab, cols, ow.ld, TG_K)) != cudaSuccess) return e;
  const int dh_wide = rows_vec16(dh, lddh, 8, sizeof(T)), dw_wide = rows_vec16(dw, lddw, 8, sizeof(T));
  for (int64_t v0 = 0; v0 < vocab; v0 += p.pw) {
    const int width = (int)(vocab - v0 < p.pw ? vocab - v0 : p.pw);
    const int tn = tile_cols(n, width, true);
    CUtensorMap mw, mg, gm;
    if ((e = make_map<T>(&mw, ow.p, vocab, cols, ow.ld, tn / 2)) != cudaSuccess) return e;
    if ((e = make_map<T>(&mg, g, n, width, p.ldg, 128)) != cudaSuccess) return e;
    if ((e = make_map<T>(&gm, g, n, width, p.ldg, TG_K)) != cudaSuccess) return e;
    EpiGrad<T> eg{label, lse, dloss, scale, g, p.ldg, (int)n, width, (int)v0, (int)vocab};
    const TileShape s1{(int)n, width, (int)cols, tn, 1, (int)v0, 0, BAND_ALL};
    if ((e = run_tiles<T, false, false>(mh, mw, s1, eg, error, chain)) != cudaSuccess) return e;
    EpiOut<T> e2{sum_h, p.lds, v0 > 0, scale, dh, lddh, (int)n, (int)cols, dh_wide};
    // a last piece too short for all ranges adds to the first ones only
    const int steps = (width + TG_K - 1) / TG_K, splits = p.splits_h < steps ? p.splits_h : steps;
    const TileShape s2{(int)n, (int)cols, width, p.tn, splits, 0, (int)v0, BAND};
    if ((e = run_tiles<T, false, true>(mg, wm, s2, e2, error, chain)) != cudaSuccess) return e;
    T* dwp = dw + v0 * lddw;
    EpiOut<T> e3{sum_w, p.lds, 0, scale, dwp, lddw, width, (int)cols, dw_wide};
    const TileShape s3{width, (int)cols, (int)n, p.tn, p.splits_w, 0, 0, BAND};
    if ((e = run_tiles<T, true, true>(gm, hm, s3, e3, error, chain)) != cudaSuccess) return e;
    if (sum_w && (e = run_sum<T>(sum_w, p.splits_w, width, cols, p.lds, scale, dwp, lddw, chain)) != cudaSuccess) return e;
  }
  return sum_h ? run_sum<T>(sum_h, p.splits_h, n, cols, p.lds, scale, dh, lddh, chain) : cudaSuccess;
}

#define INSTANTIATE(T)                                                                                                \
  template size_t linear_xent_workspace_bytes<T>(const T*, int64_t, const T*, int64_t, int64_t, int64_t, int64_t,     \
                                                 bool);                                                               \
  template cudaError_t launch_linear_xent<T>(const T*, int64_t, const T*, int64_t, const int64_t*, int64_t, int64_t,  \
                                             int64_t, float*, float*, unsigned char*, TileError, cudaStream_t);            \
  template cudaError_t launch_linear_xent_grad<T>(const float*, const T*, int64_t, const T*, int64_t, const int64_t*, \
                                                  const float*, int64_t, int64_t, int64_t, T*, int64_t, T*, int64_t,  \
                                                  unsigned char*, TileError, cudaStream_t);
INSTANTIATE(__half)
INSTANTIATE(__nv_bfloat16)
#undef INSTANTIATE

}  // namespace repro
