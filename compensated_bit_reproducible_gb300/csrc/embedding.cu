// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t]     = scale * weight[token[t]]
//   dweight[v] = scale * sum over {t : token[t] = v} of dy[t]
//
// A negative token is padding: a zero row, no gradient.  A token at or past
// the vocabulary gives a row of NaN and no gradient.
//
// The gradient's sums are the binned sum with K = 3 folds (adn.cuh), one per
// token and column, so their bits depend on the rows alone and not on the
// positions' order.  That is what lets the sort be an unordered one: a count
// per token and slots handed out by integer atomics.
#include "accum.cuh"
#include "chain.cuh"
#include "elem.cuh"
#include "f32x2.cuh"
#include "launch.h"

namespace repro {

// ------------------------------------------------------------------ lookup
// Bound by DRAM: one read of each row that occurs, one write of the output.
// The output is walked as one flat array of packs, LOOK_U per thread, all
// their loads in flight together.
constexpr int LOOK_T = 256, LOOK_U = 4;

template <typename T, int V>
__global__ void __launch_bounds__(LOOK_T) embed_kernel(const T* __restrict__ w, int64_t vocab, int64_t ldw,
                                                       const int64_t* __restrict__ tok, int64_t n, uint32_t vpr,
                                                       uint32_t step_rows, uint32_t step_cols, float scale,
                                                       T* __restrict__ out, int64_t ldo) {
  // this thread's first pack, then LOOK_T packs further each step
  const int64_t flat = (int64_t)blockIdx.x * (LOOK_T * LOOK_U) + threadIdx.x;
  int64_t row = flat / vpr;
  uint32_t col = (uint32_t)(flat - row * vpr);
  Pack<T, V> v[LOOK_U];
  int64_t at[LOOK_U];
  int64_t id[LOOK_U];
#pragma unroll
  for (int u = 0; u < LOOK_U; ++u) {
    const bool in = row < n;
    id[u] = in ? tok[row] : -1;
    at[u] = in ? row * ldo + (int64_t)col * V : -1;
    if (id[u] >= 0 && id[u] < vocab) v[u] = load_pack<T, V>(w + id[u] * ldw + (int64_t)col * V);
    row += step_rows;
    col += step_cols;
    if (col >= vpr) {
      col -= vpr;
      ++row;
    }
  }
#pragma unroll
  for (int u = 0; u < LOOK_U; ++u) {
    if (at[u] < 0) continue;
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float y = scale * to_f32<T>(v[u].e[i]);
      if (id[u] < 0) y = 0.0f;
      if (id[u] >= vocab) y = canonical_nan<float>();
      r.e[i] = from_f32<T>(y);
    }
    store_pack<T, V>(out + at[u], r);
  }
}

template <typename T, int V>
static cudaError_t embed_run(const T* w, int64_t vocab, int64_t ldw, const int64_t* tok, int64_t n, int64_t cols,
                             float scale, T* out, int64_t ldo, cudaStream_t s) {
  const uint32_t vpr = (uint32_t)(cols / V);
  const int64_t blocks = (n * (int64_t)vpr + LOOK_T * LOOK_U - 1) / (LOOK_T * LOOK_U);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  embed_kernel<T, V><<<(unsigned)blocks, LOOK_T, 0, s>>>(w, vocab, ldw, tok, n, vpr, LOOK_T / vpr, LOOK_T % vpr, scale,
                                                         out, ldo);
  return cudaGetLastError();
}

// Rows of at least a warp's packs: a warp per row and WIDE_U packs a lane, which
// needs few registers (32), so that twice as many rows are in flight as with the
// flat walk above.  32768 x 2048 bfloat16: 31 us, 6.5 TB/s of the bytes it cannot
// do without (flat: 39 us; WIDE_U 2 and 8: 32 and 31 us).
constexpr int WIDE_U = 4;
template <typename T>
__global__ void __launch_bounds__(256, 8) embed_wide(const T* __restrict__ w, int64_t vocab, int64_t ldw,
                                                     const int64_t* __restrict__ tok, int64_t n, int cols, int segs,
                                                     float scale, T* __restrict__ out, int64_t ldo) {
  constexpr int V = Vec16<T>::N;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t row = unit / segs;
  if (row >= n) return;
  const int c0 = ((int)(unit - row * segs) * (32 * WIDE_U) + (threadIdx.x & 31)) * V;
  const int64_t id = tok[row];
  const bool in = id >= 0 && id < vocab;
  const T* p = w + (in ? id : 0) * ldw;
  T* o = out + row * ldo;
  const float other = id < 0 ? 0.0f : canonical_nan<float>();
  const F2 s2 = pk2(scale, scale), o2 = pk2(other, other);
  Pack<T, V> v[WIDE_U];
#pragma unroll
  for (int i = 0; i < WIDE_U; ++i)
    if (in && c0 + i * 32 * V < cols) v[i] = load_pack<T, V>(p + c0 + i * 32 * V);
#pragma unroll
  for (int i = 0; i < WIDE_U; ++i) {
#pragma unroll
    for (int h = 0; h < V / 2; ++h) set2(v[i], h, in ? mul2(get2(v[i], h), s2) : o2);
    if (c0 + i * 32 * V < cols) store_pack<T, V>(o + c0 + i * 32 * V, v[i]);
  }
}

// Rows at any alignment, a warp per row and LOOK_WORDS words of 32 lanes.  The
// output goes out in whole words from its first aligned one; where a row of
// 16-bit elements starts between words relative to that, a lane's word is put
// together from its own and the next one (which hold the row's elements and at
// most one neighbour on each side, inside the same aligned words).  32768 x 2049
// bfloat16: 57 us (single elements: 124); 4 and 16 words: 63 and 61 us.
constexpr int LOOK_WORDS = 8;
template <typename T>
__global__ void __launch_bounds__(256, 6) embed_rows(const T* __restrict__ w, int64_t vocab, int64_t ldw,
                                                  const int64_t* __restrict__ tok, int64_t n, int cols, int segs,
                                                  float scale, T* __restrict__ out, int64_t ldo) {
  constexpr int E = 4 / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t row = unit / segs;
  if (row >= n) return;
  const int seg = (int)(unit - row * segs);
  const int64_t id = tok[row];
  T* o = out + row * ldo;
  const bool in = id >= 0 && id < vocab;
  const T* p = w + (in ? id : 0) * ldw;
  const float other = id < 0 ? 0.0f : canonical_nan<float>();
  const int head = E == 2 && ((uintptr_t)o & 2) ? 1 : 0, words = (cols - head) / E;
  const bool odd = E == 2 && ((uintptr_t)(p + head) & 2) != 0;
  const unsigned* q = (const unsigned*)((uintptr_t)(p + head) & ~(uintptr_t)3);
  const int k0 = seg * (32 * LOOK_WORDS) + lane;
  // (between words, the last one written needs one more)
  unsigned v[LOOK_WORDS], after = 0;
#pragma unroll
  for (int i = 0; i < LOOK_WORDS; ++i) v[i] = in && k0 + i * 32 < words + odd ? q[k0 + i * 32] : 0;
  if (in && odd && lane == 31 && k0 + LOOK_WORDS * 32 - 31 <= words) after = q[k0 + LOOK_WORDS * 32 - 31];
#pragma unroll
  for (int i = 0; i < LOOK_WORDS; ++i) {
    const int k = k0 + i * 32;
    unsigned x = v[i];
    if (odd) {
      unsigned next = __shfl_down_sync(0xffffffffu, v[i], 1);
      const unsigned turn = i + 1 < LOOK_WORDS ? __shfl_sync(0xffffffffu, v[i + 1 < LOOK_WORDS ? i + 1 : i], 0) : after;
      if (lane == 31) next = turn;
      x = __funnelshift_r(x, next, 16);
    }
    Pack<T, E> r;
    *reinterpret_cast<unsigned*>(&r) = x;
#pragma unroll
    for (int e = 0; e < E; ++e) r.e[e] = from_f32<T>(in ? scale * to_f32<T>(r.e[e]) : other);
    if (k < words) store_pack<T, E>(o + head + E * k, r);
  }
  if (E == 2 && seg == 0 && lane < 2) {
    // the elements before and after the words
    const int c = lane ? head + 2 * words : 0;
    if (lane ? c < cols : head) o[c] = from_f32<T>(in ? scale * to_f32<T>(p[c]) : other);
  }
}

template <typename T>
cudaError_t launch_embedding(const T* w, int64_t vocab, int64_t ldw, const int64_t* tok, int64_t n, int64_t cols,
                             float scale, T* out, int64_t ldo, cudaStream_t s) {
  if (rows_vec16(w, ldw, cols, sizeof(T)) && rows_vec16(out, ldo, cols, sizeof(T))) {
    constexpr int V = Vec16<T>::N;
    if (cols < 32 * V) return embed_run<T, V>(w, vocab, ldw, tok, n, cols, scale, out, ldo, s);
    const int64_t per = 32 * WIDE_U * V, segs = (cols + per - 1) / per, blocks = (n * segs + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    embed_wide<T><<<(unsigned)blocks, 256, 0, s>>>(w, vocab, ldw, tok, n, (int)cols, (int)segs, scale, out, ldo);
    return cudaGetLastError();
  }
  const int64_t per = 32 * LOOK_WORDS * 4 / sizeof(T), segs = (cols + per - 1) / per, blocks = (n * segs + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  embed_rows<T><<<(unsigned)blocks, 256, 0, s>>>(w, vocab, ldw, tok, n, (int)cols, (int)segs, scale, out, ldo);
  return cudaGetLastError();
}
template cudaError_t launch_embedding<float>(const float*, int64_t, int64_t, const int64_t*, int64_t, int64_t, float,
                                             float*, int64_t, cudaStream_t);
template cudaError_t launch_embedding<__half>(const __half*, int64_t, int64_t, const int64_t*, int64_t, int64_t, float,
                                              __half*, int64_t, cudaStream_t);
template cudaError_t launch_embedding<__nv_bfloat16>(const __nv_bfloat16*, int64_t, int64_t, const int64_t*, int64_t,
                                                     int64_t, float, __nv_bfloat16*, int64_t, cudaStream_t);

// ---------------------------------------------------------------- gradient
// Three kinds of table rows, by how often their token occurs:
//   never       zeros
//   1..FEW      one warp per token and 128 columns; the positions are listed
//               in the token's entry
//   more        one warp per CHUNK positions and 128 columns; the chunks of a
//               token leave states (exact integers), which a second kernel
//               adds
// One kernel does all three, the longest units first, every unit a warp's.  A
// unit is bound by instruction issue and the latency of its rows, the zeros by
// DRAM; the index and the conversion cost each column about 35 instructions, a
// deposit 7.5 an element.  32768 x 1024 bfloat16 over 65536 tokens (67 MB in, 134
// MB out): 59 us, of which 43 the sums (18 the chunks, 25 the entries) and 19 the
// zeros, each alone; 33 million instructions, 48% of issue.
// Measured and not kept: units taken from a counter (93 to 105 us the whole call
// against 92), blocks that begin with the zeros (74 us), zeros between a warp's
// sums (68 us), 3 or 5 blocks per SM (72 and 96 against 71 us), a block per chunk
// of 128 with its folds in shared memory (73 us for the chunks, with an earlier
// form of the deposits).
constexpr int FEW = 14, CHUNK = 64;

struct Few {
  int v, count, pos[FEW];         // 64 bytes: one load of a warp
};
struct Item {
  int v, start, count, part;      // a chunk of a token, its state's slot (< 0: the only chunk)
};
struct Heavy {
  int v, first, chunks, pad;      // a token of several chunks, its first state's slot
};

// cursor: positions handed out, entries, items, tokens of several chunks, their chunks
enum { CUR_POS, CUR_FEW, CUR_ITEM, CUR_HEAVY, CUR_PART, CUR_N = 8 };

struct EmbedWs {
  // zeroed at the start of each call
  int* cursor;      // [CUR_N]
  int* count;       // [vocab]
  size_t zero_bytes;
  // written before they are read
  int* start;       // [vocab]: the token's entry, or its positions' first slot
  int* rank;        // [n]
  int* pos;         // [n]: positions grouped by token
  Few* few;
  Item* item;
  Heavy* hv;
  int4* part;       // [chunks of heavy tokens * cols]: index | flags << 8 and three fold sums
  size_t bytes;
};

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

static EmbedWs embed_ws(unsigned char* base, int64_t n, int64_t vocab, int64_t cols) {
  EmbedWs w;
  size_t at = 0;
  auto take = [&](size_t b) {
    unsigned char* p = base + at;
    at += up256(b);
    return p;
  };
  // most a call can have: items, one per CHUNK positions and one more per token of over FEW; tokens of several
  // chunks; their items (ceil(c / CHUNK) is below 2 c / CHUNK for those)
  const int64_t items = n / CHUNK + n / (FEW + 1), heavy = n / (CHUNK + 1), parts = 2 * n / CHUNK;
  w.cursor = (int*)take(4 * CUR_N);
  w.count = (int*)take(4 * (size_t)vocab);
  w.zero_bytes = at;
  w.start = (int*)take(4 * (size_t)vocab);
  w.rank = (int*)take(4 * (size_t)n);
  w.pos = (int*)take(4 * (size_t)n);
  w.few = (Few*)take(sizeof(Few) * (size_t)(n < vocab ? n : vocab));
  w.item = (Item*)take(sizeof(Item) * (size_t)items);
  w.hv = (Heavy*)take(sizeof(Heavy) * (size_t)heavy);
  w.part = (int4*)take(heavy ? 16 * (size_t)parts * (size_t)cols : 0);
  w.bytes = at;
  return w;
}

// How often each token occurs, and each position's place among its token's
// (any order).  Lanes that hold the same token share one atomic.
__global__ void __launch_bounds__(256) embed_count(const int64_t* __restrict__ tok, int n, int64_t vocab,
                                                   int* __restrict__ count, int* __restrict__ rank) {
  chain_begin();
  const int t = blockIdx.x * 256 + threadIdx.x;
  const int lane = threadIdx.x & 31;
  int64_t id = t < n ? tok[t] : -1;
  // all that are no row become -1 (below, 32 bits of the token are compared)
  if (id < 0 || id >= vocab) id = -1;
  const unsigned same = __match_any_sync(0xffffffffu, (int)id);
  const int first = __ffs(same) - 1;
  int base = 0;
  if (id >= 0 && lane == first) base = atomicAdd(&count[id], __popc(same));
  base = __shfl_sync(0xffffffffu, base, first);
  if (t < n) rank[t] = id >= 0 ? base + __popc(same & ((1u << lane) - 1u)) : -1;
}

// A slot in a list for each lane that asks for `want` of them.
__device__ __forceinline__ int take_slots(int* cursor, int want, int lane) {
  int x = want;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  int base = 0;
  if (lane == 31 && x) base = atomicAdd(cursor, x);
  return __shfl_sync(0xffffffffu, base, 31) + x - want;
}

// An entry or slots for each token that occurs.
__global__ void __launch_bounds__(256) embed_plan(int vocab, EmbedWs w) {
  chain_begin();
  const int v = blockIdx.x * 256 + threadIdx.x, lane = threadIdx.x & 31;
  const int c = v < vocab ? w.count[v] : 0;
  if (!__any_sync(0xffffffffu, c > 0)) return;
  const bool few = c > 0 && c <= FEW, many = c > FEW;
  int start = take_slots(&w.cursor[CUR_FEW], few, lane);
  if (few) *(int2*)&w.few[start] = make_int2(v, c);
  if (__any_sync(0xffffffffu, many)) {
    const int p = take_slots(&w.cursor[CUR_POS], many ? c : 0, lane);
    if (many) start = p;
    const int chunks = many ? (c + CHUNK - 1) / CHUNK : 0;
    const int h = take_slots(&w.cursor[CUR_HEAVY], chunks > 1, lane);
    const int f = take_slots(&w.cursor[CUR_ITEM], chunks, lane);
    const int q = take_slots(&w.cursor[CUR_PART], chunks > 1 ? chunks : 0, lane);
    if (chunks > 1) w.hv[h] = Heavy{v, q, chunks, 0};
    for (int j = 0; j < chunks; ++j)
      w.item[f + j] = Item{v, p + j * CHUNK, min(CHUNK, c - j * CHUNK), chunks > 1 ? q + j : -1};
  }
  if (c > 0) w.start[v] = start;
}

__global__ void __launch_bounds__(256) embed_scatter(const int64_t* __restrict__ tok, int n, EmbedWs w) {
  chain_begin();
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= n) return;
  const int r = w.rank[t];
  if (r < 0) return;
  const int64_t id = tok[t];
  const int at = w.start[id];
  if (w.count[id] <= FEW) w.few[at].pos[r] = t;
  else w.pos[at + r] = t;
}

// Bin of a column's largest magnitude from its float exponent field: the
// index (adn.cuh: bin_index) is (255 - e) / 13, at most 18 with three folds.
__device__ __forceinline__ int bin_of_field(unsigned e) {
  const int i = (int)(((255u - e) * 5042u) >> 16);   // division by 13, exact below 256
  return i < 18 ? i : 18;
}
// The primaries of fold k at index i >= 1 start at 1.5 * 2^(140 - 13 (i + k)).
__device__ __forceinline__ float primary(int i, int k) {
  return __uint_as_float(((267u << 23) | 0x400000u) - (unsigned)(i + k) * (13u << 23));
}

// Deposits into the three primaries of two columns at once (accum.cuh:
// AccF::deposit_fp): a value with its last bit forced rounds on a primary's
// grid with ties away from zero, and P - S leaves the remainder.
__device__ __forceinline__ F2 sticky(F2 v) { return v | 0x0000000100000001ull; }
__device__ __forceinline__ void deposit3(F2* P, F2 x) {
  F2 S = add2(P[0], sticky(x));
  F2 r = add2(x, sub2(P[0], S));
  P[0] = S;
  S = add2(P[1], sticky(r));
  r = add2(r, sub2(P[1], S));
  P[1] = S;
  P[2] = add2(P[2], sticky(r));
}

// Correct rounding of three fold sums a, b, c, each an exact float: with at
// most 512 deposits they are at most 2^21 of their own grid units, the grids
// 2^13 apart.  The error e of a + b is a multiple of b's grid below 2^24 units
// of c's, so e + c is exact, and the last addition is the only rounding.
__device__ __forceinline__ F2 round3(F2 a, F2 b, F2 c) {
  const F2 s = add2(a, b);
  const F2 bb = sub2(s, a);
  const F2 e = add2(sub2(a, sub2(s, bb)), sub2(b, bb));
  return add2(s, add2(e, c));
}

// The sum of one value: itself, but rounded to the finest grid 2^-143 (only a
// float32 below 2^-120 has bits under it), +0 for either zero, the canonical
// NaN.
template <typename T>
__device__ __forceinline__ float one_value(float x) {
  if (sizeof(T) == 4 && fabsf(x) < 0x1p-120f) {
    F2 P[3] = {pk2(primary(18, 0), 0.0f), pk2(primary(18, 1), 0.0f), pk2(primary(18, 2), 0.0f)};
    deposit3(P, pk2(x, 0.0f));
    float y, z;
    up2(round3(sub2(P[0], pk2(primary(18, 0), 0.0f)), sub2(P[1], pk2(primary(18, 1), 0.0f)),
               sub2(P[2], pk2(primary(18, 2), 0.0f))),
        y, z);
    return y;
  }
  return x != x ? canonical_nan<float>() : __fadd_rn(x, 0.0f);
}

__device__ __forceinline__ float lanes_value(const Lanes<float, 3>& a) {
  W128 F[3] = {w_from(a.L[0]), w_from(a.L[1]), w_from(a.L[2])};
  return convert_fast<float, 3>(a.I, a.flags, F);
}

// Any column: values in bin 0, infinities, NaN.  As a state, or as its value.
template <typename T>
__device__ __noinline__ int4 slow_column(const T* __restrict__ dy, int64_t lddy, int64_t col,
                                         const int* __restrict__ pos, int c) {
  AccF<3> a;
  a.init(3);
  for (int j = 0; j < c; ++j) {
    float v[1] = {to_f32<T>(dy[(int64_t)pos[j] * lddy + col])};
    a.template chunk<1>(v);
  }
  a.finish();
  return make_int4(a.I | a.flags << 8, (int)a.L[0], (int)a.L[1], (int)a.L[2]);
}
__device__ __noinline__ float state_value(int4 st) {
  Lanes<float, 3> a;
  a.I = st.x & 255;
  a.flags = st.x >> 8;
  a.L[0] = st.y;
  a.L[1] = st.z;
  a.L[2] = st.w;
  return lanes_value(a);
}
// One chunk's state added to a column's sum.
__device__ __forceinline__ void join_state(Lanes<float, 3>& a, int4 st) {
  const int I = st.x & 255;
  if (I < a.I) a.raise_lanes(I);
  const int d = I - a.I;
  a.flags |= st.x >> 8;
  a.L[0] += d == 0 ? st.y : 0;
  a.L[1] += d == 0 ? st.z : d == 1 ? st.y : 0;
  a.L[2] += d == 0 ? st.w : d == 1 ? st.z : d == 2 ? st.y : 0;
}
// A warp's tile: REP runs of 32 * V columns, V adjacent ones per lane.
template <typename T, int V, int REP>
struct Tile {
  static constexpr int NC = V * REP, COLS = 32 * NC;
  int64_t c0;       // this lane's first column; run r starts 32 * V further
  int64_t cols;
  __device__ __forceinline__ bool in(int r) const { return c0 + r * 32 * V < cols; }
  __device__ __forceinline__ int64_t col(int i) const { return c0 + (i / V) * 32 * V + i % V; }
  __device__ __forceinline__ int place(int i, int lane) const { return (i / V) * 32 * V + lane * V + i % V; }
  __device__ __forceinline__ void load(const T* row, Pack<T, V>* v) const {
#pragma unroll
    for (int r = 0; r < REP; ++r) v[r] = in(r) ? load_pack<T, V>(row + c0 + r * 32 * V) : Pack<T, V>{};
  }
  __device__ __forceinline__ void store(T* row, const float* y) const {
#pragma unroll
    for (int r = 0; r < REP; ++r) {
      if (!in(r)) continue;
      Pack<T, V> v;
#pragma unroll
      for (int i = 0; i < V; ++i) v.e[i] = from_f32<T>(y[r * V + i]);
      store_pack<T, V>(row + c0 + r * 32 * V, v);
    }
  }
};

// Largest magnitudes of a lane's columns, a NaN above all: two to a register
// for the 16-bit types, so that rows stay packed until they are deposited.
template <typename T, int NC> struct Tops {
  unsigned m[NC];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NC; ++i) m[i] = 0;
  }
  template <int V> __device__ __forceinline__ void see(const Pack<T, V>* v) {
#pragma unroll
    for (int i = 0; i < NC; ++i) m[i] = max(m[i], __float_as_uint(fabsf(v[i / V].e[i % V])));
  }
  __device__ __forceinline__ unsigned bits(int i) const { return m[i]; }   // as a float's
};
template <typename T, typename T2, int NC> struct Tops16 {
  T2 m[NC / 2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) m[i] = T2{from_f32<T>(0.0f), from_f32<T>(0.0f)};
  }
  template <int V> __device__ __forceinline__ void see(const Pack<T, V>* v) {
#pragma unroll
    for (int i = 0; i < NC / 2; ++i)
      m[i] = __hmax2_nan(m[i], __habs2(T2{v[2 * i / V].e[2 * i % V], v[(2 * i + 1) / V].e[(2 * i + 1) % V]}));
  }
  __device__ __forceinline__ unsigned bits(int i) const {
    return __float_as_uint(to_f32<T>(i & 1 ? m[i / 2].y : m[i / 2].x));
  }
};
template <int NC> struct Tops<__half, NC> : Tops16<__half, __half2, NC> {};
template <int NC> struct Tops<__nv_bfloat16, NC> : Tops16<__nv_bfloat16, __nv_bfloat162, NC> {};

// The sums of a lane's columns: an index and three primaries each.
template <typename T, int V, int REP>
struct Sums {
  typedef Tile<T, V, REP> TL;
  static constexpr int NC = TL::NC;
  F2 P[NC / 2][3];
  int I[NC];
  bool fast;      // no column in bin 0, no infinity, no NaN

  __device__ __forceinline__ F2 start(int h, int k) const { return pk2(primary(I[2 * h], k), primary(I[2 * h + 1], k)); }
  __device__ __forceinline__ void first(const Tops<T, NC>& m) {
    fast = true;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      I[i] = bin_of_field((m.bits(i) >> 23) & 255u);
      fast &= I[i] >= 1;
      I[i] = max(I[i], 1);
    }
#pragma unroll
    for (int h = 0; h < NC / 2; ++h)
#pragma unroll
      for (int k = 0; k < 3; ++k) P[h][k] = start(h, k);
  }
  // A fold's sum of column i in its grid's units: within its binade a primary's
  // bits count them.
  __device__ __forceinline__ int digits(int i, int k) const {
    const unsigned p = (unsigned)(i & 1 ? P[i / 2][k] >> 32 : P[i / 2][k]);
    return (int)(p - __float_as_uint(primary(I[i], k)));
  }
  // Larger magnitudes have come: columns move to coarser indices, each fold's
  // sum d places down, the finest dropped.
  __device__ __forceinline__ void raise(const Tops<T, NC>& m) {
    int J[NC];
    bool any = false;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      J[i] = min(I[i], bin_of_field((m.bits(i) >> 23) & 255u));
      fast &= J[i] >= 1;
      J[i] = max(J[i], 1);
      any |= J[i] < I[i];
    }
    if (!any) return;
#pragma unroll
    for (int h = 0; h < NC / 2; ++h) {
      float f[2][3];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int i = 2 * h + z, d = I[i] - J[i];
        const int n0 = digits(i, 0), n1 = digits(i, 1), n2 = digits(i, 2);
        const int o0 = d == 0 ? n0 : 0, o1 = d == 0 ? n1 : d == 1 ? n0 : 0;
        const int o2 = d == 0 ? n2 : d == 1 ? n1 : d == 2 ? n0 : 0;
        f[z][0] = __uint_as_float(__float_as_uint(primary(J[i], 0)) + (unsigned)o0);
        f[z][1] = __uint_as_float(__float_as_uint(primary(J[i], 1)) + (unsigned)o1);
        f[z][2] = __uint_as_float(__float_as_uint(primary(J[i], 2)) + (unsigned)o2);
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) P[h][k] = pk2(f[0][k], f[1][k]);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) I[i] = J[i];
  }
  __device__ __forceinline__ void deposit(const Pack<T, V>* v) {
#pragma unroll
    for (int h = 0; h < NC / 2; ++h)
      deposit3(P[h], pk2(to_f32<T>(v[2 * h / V].e[2 * h % V]), to_f32<T>(v[(2 * h + 1) / V].e[(2 * h + 1) % V])));
  }
  // scale times the sums
  __device__ __forceinline__ void values(float scale, float* y) const {
#pragma unroll
    for (int h = 0; h < NC / 2; ++h) {
      float a, b;
      up2(round3(sub2(P[h][0], start(h, 0)), sub2(P[h][1], start(h, 1)), sub2(P[h][2], start(h, 2))), a, b);
      y[2 * h] = __fmul_rn(scale, a);
      y[2 * h + 1] = __fmul_rn(scale, b);
    }
  }
};

static_assert(CHUNK <= 64, "a lane holds two positions");
constexpr int RED_T = 256, RED_W = RED_T / 32, RED_PER_SM = 4;

// Sums of `count` rows, at(j) the j-th row's position, U rows in registers at a
// time: their magnitudes, the indices, their deposits.  (A load past the end
// repeats the last row, which changes no magnitude.)
template <int U, typename T, int V, int REP, typename At>
__device__ __forceinline__ void sum_rows(Sums<T, V, REP>& s, const Tile<T, V, REP>& tl, const T* __restrict__ dy,
                                         int64_t lddy, int count, At at) {
  for (int j = 0; j < count; j += U) {
    Pack<T, V> v[U][REP];
#pragma unroll
    for (int i = 0; i < U; ++i) tl.load(dy + (int64_t)at(min(j + i, count - 1)) * lddy, v[i]);
    Tops<T, V * REP> m;
    m.clear();
#pragma unroll
    for (int i = 0; i < U; ++i) m.template see<V>(v[i]);
    if (j == 0) s.first(m);
    else s.raise(m);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (j + i < count) s.deposit(v[i]);
  }
}

// A row of the table from the rows at pos[0..count) (also given by at), count
// >= 1.
template <int U, typename T, int V, int REP, typename At>
__device__ __forceinline__ void sum_to_row(const Tile<T, V, REP>& tl, const T* __restrict__ dy, int64_t lddy,
                                           int count, const int* pos, float scale, T* __restrict__ out, At at) {
  constexpr int NC = V * REP;
  float y[NC];
  if (count == 1) {
    Pack<T, V> v[REP];
    tl.load(dy + (int64_t)at(0) * lddy, v);
#pragma unroll
    for (int i = 0; i < NC; ++i) y[i] = __fmul_rn(scale, one_value<T>(to_f32<T>(v[i / V].e[i % V])));
    tl.store(out, y);
    return;
  }
  Sums<T, V, REP> s;
  sum_rows<U>(s, tl, dy, lddy, count, at);
  if (s.fast) {
    s.values(scale, y);
    tl.store(out, y);
  } else {
    for (int i = 0; i < NC; ++i) {
      const int64_t col = tl.col(i);
      if (col < tl.cols)
        out[col] = from_f32<T>(__fmul_rn(scale, state_value(slow_column<T>(dy, lddy, col, pos, count))));
    }
  }
}
template <int U, typename T, int V, int REP>
__device__ __forceinline__ void sum_to_row(const Tile<T, V, REP>& tl, const T* __restrict__ dy, int64_t lddy,
                                           int count, const int* pos, float scale, T* __restrict__ out) {
  sum_to_row<U>(tl, dy, lddy, count, pos, scale, out, [&](int j) { return pos[j]; });
}

// Units of (list entry, tile), a warp's every `step`.
struct Units {
  int it, tile, step_it, step_tile, tiles;
  __device__ __forceinline__ Units(int first, int step, int t)
      : it(first / t), tile(first % t), step_it(step / t), step_tile(step % t), tiles(t) {}
  __device__ __forceinline__ void next() {
    it += step_it;
    tile += step_tile;
    if (tile >= tiles) {
      tile -= tiles;
      ++it;
    }
  }
};

// Chunks of tokens of many positions.
template <typename T, int V, int REP>
__device__ __forceinline__ void reduce_chunks(const T* __restrict__ dy, int64_t lddy, int64_t cols, float scale,
                                              const EmbedWs& w, T* __restrict__ dw, int64_t lddw, Units u) {
  typedef Tile<T, V, REP> TL;
  constexpr int NC = TL::NC;
  const int lane = threadIdx.x & 31;
  const int items = w.cursor[CUR_ITEM];
  for (; u.it < items; u.next()) {
    const Item me = w.item[u.it];
    const int* pos = w.pos + me.start;
    const int p0 = pos[min(lane, me.count - 1)], p1 = pos[min(lane + 32, me.count - 1)];
    TL tl;
    tl.cols = cols;
    tl.c0 = (int64_t)u.tile * TL::COLS + lane * V;
    Sums<T, V, REP> s;
    sum_rows<8>(s, tl, dy, lddy, me.count, [&](int j) { return __shfl_sync(0xffffffffu, j < 32 ? p0 : p1, j & 31); });
    if (me.part < 0 && s.fast) {
      float y[NC];
      s.values(scale, y);
      tl.store(dw + (int64_t)me.v * lddw, y);
      continue;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t col = tl.col(i);
      if (col >= cols) continue;
      int4 st = make_int4(s.I[i], s.digits(i, 0), s.digits(i, 1), s.digits(i, 2));
      if (!s.fast) st = slow_column<T>(dy, lddy, col, pos, me.count);
      if (me.part < 0) dw[(int64_t)me.v * lddw + col] = from_f32<T>(__fmul_rn(scale, state_value(st)));
      else w.part[(int64_t)me.part * cols + col] = st;
    }
  }
}

// Tokens of a few positions.  The next unit's entry is loaded while one is
// summed.
template <typename T, int V, int REP>
__device__ __forceinline__ void reduce_few(const T* __restrict__ dy, int64_t lddy, int64_t cols, float scale,
                                           const EmbedWs& w, T* __restrict__ dw, int64_t lddw, Units u) {
  typedef Tile<T, V, REP> TL;
  const int lane = threadIdx.x & 31;
  const int entries = w.cursor[CUR_FEW];
  auto entry = [&](int k) { return k < entries && lane < 16 ? ((const int*)(w.few + k))[lane] : 0; };
  int next = entry(u.it);
  while (u.it < entries) {
    const int e = next, me = u.it;
    TL tl;
    tl.cols = cols;
    tl.c0 = (int64_t)u.tile * TL::COLS + lane * V;
    u.next();
    next = entry(u.it);
    const int row = __shfl_sync(0xffffffffu, e, 0), count = __shfl_sync(0xffffffffu, e, 1);
    sum_to_row<4>(tl, dy, lddy, count, w.few[me].pos, scale, dw + (int64_t)row * lddw,
                  [&](int j) { return __shfl_sync(0xffffffffu, e, 2 + j); });
  }
}

// Zeros from p: 16-byte stores from the first aligned byte to the last,
// elements before and after.
template <typename T>
__device__ __forceinline__ void zero_span(T* p, int64_t count, int lane) {
  constexpr int N = Vec16<T>::N;
  const int64_t head = min(count, (int64_t)((16 - ((uintptr_t)p & 15u)) & 15u) / (int64_t)sizeof(T));
  const int64_t wide = (count - head) / N;
  if (lane < head) p[lane] = from_f32<T>(0.0f);
  for (int64_t i = lane; i < wide; i += 32) *(uint4*)(p + head + i * N) = make_uint4(0, 0, 0, 0);
  const int64_t tail = head + wide * N + lane;
  if (tail < count) p[tail] = from_f32<T>(0.0f);
}

// Zero rows, ZERO_ROWS tokens to a warp at a time.
constexpr int ZERO_ROWS = 4;
template <typename T>
__device__ __forceinline__ void zero_rows(int64_t cols, int vocab, const EmbedWs& w, T* __restrict__ dw, int64_t lddw,
                                          int64_t first, int64_t step) {
  const int lane = threadIdx.x & 31;
  for (int64_t v0 = first * ZERO_ROWS; v0 < vocab; v0 += step * ZERO_ROWS) {
    const int c = lane < ZERO_ROWS && v0 + lane < vocab ? w.count[v0 + lane] : 1;
    const unsigned none = __ballot_sync(0xffffffffu, c == 0);
#pragma unroll
    for (int j = 0; j < ZERO_ROWS; ++j) {
      if (!(none >> j & 1)) continue;
      zero_span(dw + (v0 + j) * lddw, cols, lane);
    }
  }
}

template <typename T, int V, int REP>
__global__ void __launch_bounds__(RED_T, RED_PER_SM)
    embed_reduce(const T* __restrict__ dy, int64_t lddy, int64_t cols, int vocab, float scale, EmbedWs w,
                 T* __restrict__ dw, int64_t lddw, int tiles) {
  chain_begin();
  // neighbouring units go to different blocks
  const int wid = (threadIdx.x >> 5) * gridDim.x + blockIdx.x, warps = gridDim.x * RED_W;
  reduce_chunks<T, V, REP>(dy, lddy, cols, scale, w, dw, lddw, Units(wid, warps, tiles));
  reduce_few<T, V, REP>(dy, lddy, cols, scale, w, dw, lddw, Units(wid, warps, tiles));
  zero_rows<T>(cols, vocab, w, dw, lddw, wid, warps);
}

// The chunks' states of a heavy token, a warp per eight columns: four lanes take
// every fourth state of a column, JOIN_U loads in flight each, and add up what
// they have.  All exact integers.  Bound by the chain of additions of the most
// common token (2000 positions, 32 states): 9 us beside the 59 above.
constexpr int JOIN_U = 8;
template <typename T>
__global__ void __launch_bounds__(128)
    embed_join(int64_t cols, float scale, EmbedWs w, T* __restrict__ dw, int64_t lddw, int groups) {
  chain_begin();
  const int lane = threadIdx.x & 31, strand = lane >> 3;
  const int heavy = w.cursor[CUR_HEAVY];
  for (Units u((threadIdx.x >> 5) * gridDim.x + blockIdx.x, 4 * gridDim.x, groups); u.it < heavy; u.next()) {
    const Heavy h = w.hv[u.it];
    const int64_t col = (int64_t)u.tile * 8 + (lane & 7);
    const int4* part = w.part + (int64_t)h.first * cols + col;
    Lanes<float, 3> a;
    a.init(3);
    if (col < cols)
      for (int j = strand; j < h.chunks; j += 4 * JOIN_U) {
        int4 st[JOIN_U];
#pragma unroll
        for (int i = 0; i < JOIN_U; ++i)
          if (j + 4 * i < h.chunks) st[i] = part[(int64_t)(j + 4 * i) * cols];
#pragma unroll
        for (int i = 0; i < JOIN_U; ++i)
          if (j + 4 * i < h.chunks) join_state(a, st[i]);
      }
#pragma unroll
    for (int d = 8; d <= 16; d <<= 1) {
      Lanes<float, 3> b;
      b.I = __shfl_xor_sync(0xffffffffu, a.I, d);
      b.flags = __shfl_xor_sync(0xffffffffu, a.flags, d);
#pragma unroll
      for (int i = 0; i < 3; ++i) b.L[i] = __shfl_xor_sync(0xffffffffu, a.L[i], d);
      if (b.I < a.I) a.raise_lanes(b.I);
      else b.raise_lanes(a.I);
      a.flags |= b.flags;
#pragma unroll
      for (int i = 0; i < 3; ++i) a.L[i] += b.L[i];
    }
    if (strand == 0 && col < cols) dw[(int64_t)h.v * lddw + col] = from_f32<T>(__fmul_rn(scale, lanes_value(a)));
  }
}

// -------------------------------------------------------- few positions
// At most SMALL_N positions: one launch and no workspace.  A block owns a range
// of table rows and some of their column tiles, finds its positions among all
// tokens, and lists them by row in shared memory (in any order).  509 x 769
// float32 over 10007 tokens: 12 us, the zeros (31 MB) among them; with
// the sorted path's six launches 21 us.  1024 positions: 15 and 28; 1024 x 2048
// over 50000 tokens 77 and 88.  (Where one token holds all 1024, the sorted path
// is the faster from 1024 columns on: 46 against 55 us.)
constexpr int SMALL_N = 1024, SMALL_ROWS = 512;
// A row of up to ALONE positions is summed by one warp per tile, a longer one
// by all eight, each an eighth of its positions.
constexpr int ALONE = 24;

template <typename T, int V, int REP>
__global__ void __launch_bounds__(RED_T, 2)
    embed_small(const T* __restrict__ dy, int64_t lddy, const int64_t* __restrict__ tok, int n, int64_t vocab,
                int64_t cols, float scale, T* __restrict__ dw, int64_t lddw, int64_t range, int tiles, int group) {
  typedef Tile<T, V, REP> TL;
  constexpr int NC = TL::NC, COLS = TL::COLS;
  __shared__ int count[SMALL_ROWS], start[SMALL_ROWS], fill[SMALL_ROWS], used[SMALL_ROWS];
  __shared__ int list[SMALL_N];
  __shared__ int total, rows_used, index[COLS], folds[3][COLS], special;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.y * group, t1 = min(tiles, t0 + group);
  const int64_t end = min(vocab, (int64_t)(blockIdx.x + 1) * range);
  for (int64_t v0 = (int64_t)blockIdx.x * range; v0 < end; v0 += SMALL_ROWS) {
    const int rows = (int)min((int64_t)SMALL_ROWS, end - v0);
    for (int i = threadIdx.x; i < rows; i += RED_T) count[i] = 0;
    if (threadIdx.x == 0) total = rows_used = 0;
    __syncthreads();
    int mine[SMALL_N / RED_T];   // this thread's tokens, as rows of the range
#pragma unroll
    for (int k = 0; k < SMALL_N / RED_T; ++k) {
      const int t = threadIdx.x + k * RED_T;
      const int64_t id = t < n ? tok[t] : -1;
      mine[k] = id >= v0 && id < v0 + rows ? (int)(id - v0) : -1;
      if (mine[k] >= 0) atomicAdd(&count[mine[k]], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows; i += RED_T)
      if (count[i]) {
        start[i] = atomicAdd(&total, count[i]);
        fill[i] = 0;
        used[atomicAdd(&rows_used, 1)] = i;
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < SMALL_N / RED_T; ++k)
      if (mine[k] >= 0) list[start[mine[k]] + atomicAdd(&fill[mine[k]], 1)] = threadIdx.x + k * RED_T;
    __syncthreads();
    // zero rows are dealt whole over the blocks of the range
    for (int i = warp * gridDim.y + blockIdx.y; i < rows; i += RED_W * gridDim.y)
      if (!count[i]) zero_span(dw + (v0 + i) * lddw, cols, lane);
    TL tl;
    tl.cols = cols;
    const int units = rows_used * (t1 - t0);
    for (int u = warp; u < units; u += RED_W) {
      const int i = used[u / (t1 - t0)], c = count[i];
      if (c > ALONE) continue;
      tl.c0 = (int64_t)(t0 + u % (t1 - t0)) * COLS + lane * V;
      const int* pos = list + start[i];
      sum_to_row<8>(tl, dy, lddy, c, pos, scale, dw + (v0 + i) * lddw);
    }
    for (int r = 0; r < rows_used; ++r) {
      const int i = used[r], c = count[i];
      if (c <= ALONE) continue;
      for (int tile = t0; tile < t1; ++tile) {
        for (int k = threadIdx.x; k < COLS; k += RED_T) {
          index[k] = 18;
          folds[0][k] = folds[1][k] = folds[2][k] = 0;
        }
        if (threadIdx.x == 0) special = 0;
        __syncthreads();
        tl.c0 = (int64_t)tile * COLS + lane * V;
        const int* pos = list + start[i] + warp;
        Sums<T, V, REP> s;
        sum_rows<8>(s, tl, dy, lddy, (c - warp + RED_W - 1) / RED_W, [&](int j) { return pos[j * RED_W]; });
        if (!s.fast) special = 1;
#pragma unroll
        for (int k = 0; k < NC; ++k) atomicMin(&index[tl.place(k, lane)], s.I[k]);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          const int at = tl.place(k, lane), d = s.I[k] - index[at];
#pragma unroll
          for (int f = 0; f < 3; ++f)
            if (f + d < 3) atomicAdd(&folds[f + d][at], s.digits(k, f));
        }
        __syncthreads();
        const int64_t col = (int64_t)tile * COLS + threadIdx.x;
        if (threadIdx.x < COLS && col < cols) {
          int4 st = make_int4(index[threadIdx.x], folds[0][threadIdx.x], folds[1][threadIdx.x], folds[2][threadIdx.x]);
          if (special) st = slow_column<T>(dy, lddy, col, list + start[i], c);
          dw[(v0 + i) * lddw + col] = from_f32<T>(__fmul_rn(scale, state_value(st)));
        }
        __syncthreads();
      }
    }
    __syncthreads();
  }
}

template <typename T, int V, int REP>
static cudaError_t embed_small_run(const T* dy, int64_t lddy, const int64_t* tok, int64_t n, int64_t vocab,
                                   int64_t cols, float scale, T* dw, int64_t lddw, int tiles, int sms, cudaStream_t s) {
  // Two blocks per SM, as ranges of rows by groups of tiles.  One token may hold many positions, and its block then
  // sums them alone: more groups bound that, and make every block look for its positions among more rows.  On the
  // device, over 10007 x 769, tokens by 1 / rank (a mean of ten draws), 4 groups and 8 in us:
  //               128            256            384            509            1024 positions
  //   float32      8.2 and 9.4    9.7 and 10.4  11.7 and 11.4  12.2 and 12.0  16.3 and 14.4
  //   bfloat16     6.7 and 7.3    8.3 and 8.2   10.2 and 9.3   10.8 and 9.9   14.9 and 12.4
  // One token for all: 256 positions 21 and 12, 1024 58 and 24; all tokens alike likely: 8.0 and 10.2, 11.6 and 15.6
  // (float32).  2 groups take 1 to 4 us more from 384 positions on; 16 are no faster before 2048 columns.
  const int most = n <= SMALL_N / 4 ? 4 : 8, groups = tiles < most ? tiles : most;
  const int group = (tiles + groups - 1) / groups, gy = (tiles + group - 1) / group;
  const int64_t want = (2 * (int64_t)sms + gy - 1) / gy, range = (vocab + want - 1) / want;
  const dim3 grid((unsigned)((vocab + range - 1) / range), (unsigned)gy);
  embed_small<T, V, REP><<<grid, RED_T, 0, s>>>(dy, lddy, tok, (int)n, vocab, cols, scale, dw, lddw, range, tiles,
                                                group);
  return cudaGetLastError();
}

template <typename T, int V, int REP>
static cudaError_t embed_reduce_run(Chain& chain, const EmbedWs& w, const T* dy, int64_t lddy, int64_t n,
                                    int64_t vocab, int64_t cols, float scale, T* dw, int64_t lddw, int tiles,
                                    int sms) {
  cudaError_t e = chain.launch(embed_reduce<T, V, REP>, (unsigned)(RED_PER_SM * sms), RED_T, 0, dy, lddy, cols,
                               (int)vocab, scale, w, dw, lddw, tiles);
  if (e != cudaSuccess) return e;
  const int64_t groups = (cols + 7) / 8, blocks = (n / (CHUNK + 1) * groups + 3) / 4;
  return chain.launch(embed_join<T>, (unsigned)(blocks < 16 * sms ? blocks : 16 * sms), 128, 0, cols, scale, w, dw,
                      lddw, (int)groups);
}

// Every warp tile is 128 columns: four adjacent ones per lane where rows are
// 16-byte aligned, else four runs of 32.
constexpr int64_t EMBED_TILE = 128;

template <typename T>
size_t embedding_grad_workspace_bytes(const T*, int64_t, int64_t n, int64_t vocab, int64_t cols, const T*, int64_t) {
  return n <= SMALL_N ? 0 : embed_ws(nullptr, n, vocab, cols).bytes;
}

template <typename T>
cudaError_t launch_embedding_grad(const T* dy, int64_t lddy, const int64_t* tok, int64_t n, int64_t vocab,
                                  int64_t cols, float scale, T* dw, int64_t lddw, unsigned char* ws, int sms,
                                  cudaStream_t s) {
  const int tiles = (int)((cols + EMBED_TILE - 1) / EMBED_TILE);
  const bool wide = rows_vec16(dy, lddy, cols, sizeof(T)) && rows_vec16(dw, lddw, cols, sizeof(T));
  if (n <= SMALL_N)
    return wide ? embed_small_run<T, 4, 1>(dy, lddy, tok, n, vocab, cols, scale, dw, lddw, tiles, sms, s)
                : embed_small_run<T, 1, 4>(dy, lddy, tok, n, vocab, cols, scale, dw, lddw, tiles, sms, s);
  const EmbedWs w = embed_ws(ws, n, vocab, cols);
  cudaError_t e = cudaMemsetAsync(w.cursor, 0, w.zero_bytes, s);
  if (e != cudaSuccess) return e;
  Chain chain(s);
  if ((e = chain.launch(embed_count, (unsigned)((n + 255) / 256), 256, 0, tok, (int)n, vocab, w.count, w.rank)) !=
          cudaSuccess ||
      (e = chain.launch(embed_plan, (unsigned)((vocab + 255) / 256), 256, 0, (int)vocab, w)) != cudaSuccess ||
      (e = chain.launch(embed_scatter, (unsigned)((n + 255) / 256), 256, 0, tok, (int)n, w)) != cudaSuccess)
    return e;
  return wide ? embed_reduce_run<T, 4, 1>(chain, w, dy, lddy, n, vocab, cols, scale, dw, lddw, tiles, sms)
              : embed_reduce_run<T, 1, 4>(chain, w, dy, lddy, n, vocab, cols, scale, dw, lddw, tiles, sms);
}

#define INSTANTIATE(T)                                                                                               \
  template size_t embedding_grad_workspace_bytes<T>(const T*, int64_t, int64_t, int64_t, int64_t, const T*, int64_t); \
  template cudaError_t launch_embedding_grad<T>(const T*, int64_t, const int64_t*, int64_t, int64_t, int64_t, float, \
                                                T*, int64_t, unsigned char*, int, cudaStream_t);
INSTANTIATE(float)
INSTANTIATE(__half)
INSTANTIATE(__nv_bfloat16)
#undef INSTANTIATE

}  // namespace repro
