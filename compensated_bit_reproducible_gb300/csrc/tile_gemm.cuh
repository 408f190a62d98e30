// Tiles of a 16-bit matrix product on the tensor cores, D = A B^T, with the
// accumulator handed to an epilogue: the core of the linear cross entropy.
//
// A pair of blocks (a cluster of two) works on tiles of 256 x tn (tn a multiple
// of 32, at most 256): each block stages 128 rows of A and tn / 2 rows of B per
// step of 64 along the inner dimension (TMA, 128-byte swizzle, TG_STAGES steps
// in flight), one thread of the pair issues the products (tcgen05.mma,
// cta_group::2), and each block's tensor memory holds its 128 rows of the
// accumulator, twice, so that the epilogue of one tile runs under the products
// of the next.  The pair halves what each SM takes from L2: 64 bytes a clock at
// full rate instead of the 96 of a block on its own with 128 x 256.
//
// The inner dimension can be cut into `splits` ranges, each a tile of its own:
// for products with few tiles and a long inner dimension.
//
// An operand is K-major (the inner dimension is contiguous) or MN-major (its
// own rows' index is contiguous); shapes need not be multiples of anything:
// TMA fills what lies outside with zeros.
//
// Warps: 0 copies, 1 multiplies, 2 allocates tensor memory, 4..11 epilogue
// (warps 4..7 the first half of a tile's columns, in runs of 32, 8..11 the
// rest).
//
// 8192 x 32768 x 2048 bfloat16: 592 us, 1.86 PFLOP/s, in 20 calls.  In 200
// calls back to back the loss (this kernel and the join) takes 629 to 636 us, a
// library's product alone, which writes the logits, 576 to 591; over 3 s, under
// the power limit, 656 and 633.  The epilogue's instructions draw on the same power.
// Bands of tiles (TileWalk) took half of a weight gradient from 331 to 305 us.
//
// Every wait is bounded: after about two seconds it sets both words of TileError and the block
// winds down (drops its tiles, leaves copies and products in flight a
// millisecond to end, frees its tensor memory, returns).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include "chain.cuh"
#include "elem.cuh"
#include "launch.h"
#include "mbarrier.cuh"
#include "tile_walk.h"

namespace repro {

constexpr int TG_STAGES = 6, TG_HALF = 128 * TG_K * 2;   // bytes of one block's half of an operand step
constexpr int TG_STAGE = 2 * TG_HALF;
constexpr int TG_THREADS = 384, TG_EPI_WARPS = 8;
// a warp's 32 x 32 outputs in 16 bits on their way to memory: rows of 80 bytes
// keep 16-byte accesses of both orders free of bank conflicts
constexpr int TG_ROW = 80, TG_OUT = 32 * TG_ROW;
constexpr int TG_SMEM = TG_STAGES * TG_STAGE + TG_EPI_WARPS * TG_OUT + 1024;   // 1024 for the swizzle's alignment

__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// Box at (x, y) of a tensor map into this block's shared memory, counted at a
// barrier of the pair.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(dst),
      "l"(map), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Arrives at the barrier of both blocks when the products issued so far are done.
__device__ __forceinline__ void mma_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 32 columns of this thread's accumulator row.  Load and wait are one asm
// statement: nothing that uses v can be scheduled between them.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}

// Shared-memory descriptor of a swizzled operand.  K-major: rows of 128 bytes,
// groups of eight rows 1024 bytes apart.  MN-major: blocks of 64 own indices,
// a row of 128 bytes per inner index, groups of eight inner indices 1024 bytes
// apart, blocks TG_K * 128 bytes apart.
template <bool MN>
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  constexpr uint64_t lead = MN ? (TG_K * 128) >> 4 : 1, stride = 1024 >> 4;
  return (uint64_t)((addr & 0x3ffff) >> 4) | lead << 16 | stride << 32 | 1ull << 46 | 2ull << 61;
}
// 16 further along the inner dimension, in 16-byte units of the descriptor.
template <bool MN> struct DescStep { static constexpr uint64_t V = MN ? 2048 >> 4 : 32 >> 4; };

// Instruction descriptor: float32 accumulator, 16-bit inputs (1: bfloat16),
// operand orders, N and M of the pair.
template <bool BF16, bool AMN, bool BMN>
__device__ __forceinline__ uint32_t instr_desc(int tn) {
  return 1u << 4 | (BF16 ? 1u << 7 | 1u << 10 : 0u) | (AMN ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u) |
         (uint32_t)(tn >> 3) << 17 | (uint32_t)(TG_M >> 4) << 24;
}

// 32 values of each lane's row, rounded to T and stored as rows of 32 columns
// from `col`: through `stage`, so that a store covers whole sectors of a row
// whatever its alignment.  The warp's rows are row0 .. row0 + 31; a lane whose
// `keep` is zero stores zeros.
template <typename T>
__device__ __forceinline__ void put_rows(const F2* v, unsigned char* stage, int lane, T* out, int64_t ld, int row0,
                                         int rows, int col, int cols, bool wide, unsigned keep = ~0u) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    Pack<T, 8> p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      set2(p, i, v[4 * j + i]);
      reinterpret_cast<unsigned*>(&p)[i] &= keep;
    }
    store_pack<T, 8>((T*)(stage + lane * TG_ROW) + 8 * j, p);
  }
  __syncwarp();
  if (wide && col + 32 <= cols) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 8 * j + lane / 4, c = lane % 4 * 8;
      if (row0 + r < rows)
        store_pack<T, 8>(out + (int64_t)(row0 + r) * ld + col + c, load_pack<T, 8>((T*)(stage + r * TG_ROW) + c));
    }
  } else {
    const bool in = col + lane < cols;
    T* o = out + (int64_t)row0 * ld + col + lane;
#pragma unroll 8
    for (int r = 0; r < 32; ++r)
      if (in && row0 + r < rows) o[(int64_t)r * ld] = *((T*)(stage + r * TG_ROW) + lane);
  }
}

// The epilogue E is a struct of plain values, passed by copy.  A thread sees one
// row of each of its block's tiles, and half of the tile's columns:
//   void row(int row, State&)                        before the first chunk
//   void chunk(int row, int col, F2* v, State&, const Place&)   32 columns, by pairs
//   void done(int row, State&, const Place&)         after the last
// with rows and columns counted in the product.  Every lane of a warp calls.
struct Place {
  int row0, lane;          // the warp's first row, the thread's lane
  int half, tile;          // of the tile: which half; its index along the columns
  int split;               // which range of the inner dimension
  unsigned char* stage;    // TG_OUT bytes of the warp's own
};
template <bool BF16, bool AMN, bool BMN, typename E>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(TG_THREADS, 1)
    tile_gemm(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, TileShape sh, E epi,
              TileError error) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[TG_STAGES], empty[TG_STAGES], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int stop;
  const uint32_t tiles0 = (smem_u32(raw) + 1023) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
  if (threadIdx.x == 0) {
    for (int i = 0; i < TG_STAGES; ++i) {
      mbar_init(smem_u32(&full[i]), 1 + error.never);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), 2 * TG_EPI_WARPS);
    }
    stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_slot;
  chain_begin();

  // false: gave up (here or in another warp of this block)
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const uint32_t b = smem_u32(bar);
    if (mbar_try(b, parity)) return true;
    const uint64_t t0 = now_ns();
    for (;;) {
      for (int i = 0; i < 64; ++i)
        if (mbar_try(b, parity)) return true;
      if (*(volatile int*)&stop) return false;
      if (now_ns() - t0 > error.limit_ns) {
        *(volatile int*)&stop = 1;
        *(volatile int*)error.device = 1;
        *(volatile int*)error.host = 1;
        __threadfence_system();
        return false;
      }
    }
  };

  const int kb = (sh.k + TG_K - 1) / TG_K, tn = sh.tn;
  // first step of a range of the inner dimension
  auto k_at = [&](int split) {
    return sh.splits == 1 ? split * kb : (int)((unsigned)kb * (unsigned)split / (unsigned)sh.splits);
  };
  TileWalk tile(sh, blockIdx.x >> 1, gridDim.x >> 1);

  if (warp == 0 && lane == 0) {
    // copies: this block's half of A and of B (MN-major: blocks of 64 rows)
    const uint32_t bytes = 2 * (TG_HALF + (BMN ? (tn > 128 ? TG_HALF : TG_HALF / 2) : tn / 2 * TG_K * 2));
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const uint32_t bar0 = mapa(smem_u32(&full[0]), 0);
    for (; tile.more() && ok; tile.next()) {
      const int m0 = tile.m * TG_M + (int)rank * 128;
      const int n0 = tile.n * tn + (int)rank * (tn / 2) + sh.bn0;
      for (int k = k_at(tile.split), k1 = k_at(tile.split + 1); k < k1; ++k) {
        if (!(ok = wait(&empty[s], ph ^ 1))) break;
        const uint32_t a = tiles0 + s * TG_STAGE, b = a + TG_HALF;
        const uint32_t bar = bar0 + 8 * s;
        if (rank == 0) mbar_expect(smem_u32(&full[s]), bytes);
        const int ka = k * TG_K, kbx = sh.bk0 + k * TG_K;
        if (AMN) {
          tma_load(a, &amap, m0, ka, bar);
          tma_load(a + TG_HALF / 2, &amap, m0 + 64, ka, bar);
        } else {
          tma_load(a, &amap, ka, m0, bar);
        }
        if (BMN) {
          tma_load(b, &bmap, n0, kbx, bar);
          if (tn > 128) tma_load(b + TG_HALF / 2, &bmap, n0 + 64, kbx, bar);
        } else {
          tma_load(b, &bmap, kbx, n0, bar);
        }
        if (++s == TG_STAGES) s = 0, ph ^= 1;
      }
    }
    // the last steps' release has arrived here before the block may end
    for (int i = 0; i < TG_STAGES && ok; ++i) {
      ok = wait(&empty[s], ph ^ 1);
      if (++s == TG_STAGES) s = 0, ph ^= 1;
    }
    if (!ok) pause_ns(WAIT_DRAIN_NS);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    const uint32_t idesc = instr_desc<BF16, AMN, BMN>(tn);
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (; tile.more() && ok; tile.next(), ++it) {
      const int buf = it & 1;
      if (!(ok = wait(&acc_empty[buf], ((it >> 1) & 1) ^ 1))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int k0 = k_at(tile.split), k1 = k_at(tile.split + 1);
      for (int k = k0; k < k1; ++k) {
        if (!(ok = wait(&full[s], ph))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint64_t a = smem_desc<AMN>(tiles0 + s * TG_STAGE);
        const uint64_t b = smem_desc<BMN>(tiles0 + s * TG_STAGE + TG_HALF);
#pragma unroll
        for (int j = 0; j < TG_K / 16; ++j)
          mma_f16(tmem + buf * TG_N, a + j * DescStep<AMN>::V, b + j * DescStep<BMN>::V, idesc, k > k0 || j > 0);
        mma_commit_both(smem_u32(&empty[s]));
        if (++s == TG_STAGES) s = 0, ph ^= 1;
      }
      if (ok) mma_commit_both(smem_u32(&acc_full[buf]));
    }
    if (!ok) pause_ns(WAIT_DRAIN_NS);
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2, runs = tn / 32;
    const int c0 = half ? (runs + 1) / 2 : 0, c1 = half ? runs : (runs + 1) / 2;
    Place at;
    at.lane = lane;
    at.half = half;
    at.stage = raw + (tiles0 - smem_u32(raw)) + TG_STAGES * TG_STAGE + (warp - 4) * TG_OUT;
    int it = 0;
    for (; tile.more(); tile.next(), ++it) {
      const int buf = it & 1;
      at.split = tile.split;
      at.row0 = tile.m * TG_M + (int)rank * 128 + q * 32;
      at.tile = tile.n;
      const int row = at.row0 + lane;
      typename E::State st;
      epi.row(row, st);
      if (!__all_sync(0xffffffffu, wait(&acc_full[buf], (it >> 1) & 1))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * TG_N;
      // the accumulator is free once every warp of both blocks has read its part
      auto release = [&] {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&acc_empty[buf]), 0));
      };
      if (c0 == c1) release();
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        float f[32];
        tmem_load32(acc + c * 32, f);
        if (c + 1 == c1) release();
        F2 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = pk2(f[2 * i], f[2 * i + 1]);
        epi.chunk(row, at.tile * tn + c * 32, v, st, at);
      }
      epi.done(row, st, at);
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace repro
