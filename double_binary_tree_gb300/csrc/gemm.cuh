// Matrix products on the fifth-generation tensor cores (tcgen05) with a
// fused epilogue: the base of the training operators.
//
//   D[z][m][n] = sum_k A[z][m][k] B[z][n][k],  16-bit operands, fp32 sums
//
// Persistent CTAs, one per SM, 128 x BN tiles, or pairs of CTAs (PAIR) that
// work on one 256 x BN tile: each CTA holds its 128 rows of A and of the
// accumulator and half of B, so a slice of the tile costs an SM a third less
// shared memory traffic (what bounds 128-wide tiles) and L2 traffic.  Warp 0 moves 64-deep slices of
// A and B into a ring of shared-memory stages with tensor copies (TMA), warp
// 1 issues the products on them, warps 4 on (Epi::kWarps of them, 8 or 16) read
// finished accumulators from tensor memory and run the epilogue.  Two accumulators take turns, so the
// epilogue of one tile overlaps the products of the next.
//
// PARTS = 2: each operand is the sum of a high and a low 16-bit plane
// (22 bits) and three products are summed -- high x high, high x low, low x
// high; low x low is below what the planes resolve.
//
// An operand is K-major (its rows are contiguous along k) or MN-major (its
// rows are k, contiguous along m or n); both are read as they lie in memory,
// so no operand is ever transposed by a pass of its own.  Elements outside
// the operand's extents are read as zero by the copy, which makes every
// ragged edge correct without a second path.
//
// SPLIT: too few tiles for the SMs.  A cluster of several CTAs (pairs) takes
// one tile, each a share of k; the partial sums meet in shared memory and
// every CTA of the cluster adds up and finishes some of the columns, in the
// order of the shares.
//
// Measured on GB300, 4864 x 4864 x 4096 fp16 with an epilogue that stores
// nothing: pairs 256 x 256 1950 TFLOP/s (1.01 of a cuBLAS bf16 product of
// 8192^3; either operand K- or MN-major), summed in chunks of 512 1910,
// 256 x 128 1800, single CTAs 128 x 256 1850, 128 x 128 1490 (shared memory
// bandwidth); two planes, sums handed over every 128, 1660 over their three
// products.  One tile of 64 k takes 2.7 us, 4.2 us on a pair.  What bounds a
// call is the products, where k is long; the epilogue, where it is short
// (a 256 x 256 tile's products take 0.31 us per 64 k).
//
// Every wait is bounded.  A CTA that gives up records VR_ERR_TIMEOUT, waits
// (bounded) for its copies and products in flight, frees its tensor memory
// and returns.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "gemm_host.h"
#include "staged.cuh"

namespace vr {

constexpr int kTileM = 128;
constexpr int kTileK = 64;  // 16-bit elements: one 128-byte swizzled row
constexpr int kGemmSmem = 220 * 1024;  // barriers included

struct GemmArgs {
  CUtensorMap a[2], b[2];  // high and low planes
  int M, N, K, batch;
  const int* dynM;  // extents known on the device only (at most M, K), or null
  const int* dynK;
  int triangle;     // 128-blocks on or below the diagonal only
  unsigned* status;
  unsigned long long timeoutNs;
};

// A tile's place.
struct Tile {
  int z, m0, n0;
};

// PAIR: `bar` may be in the other CTA of the pair (peer_addr).
template <bool PAIR>
__device__ __forceinline__ void tensor_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  if constexpr (PAIR) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  }
}
// True in one lane of a converged warp (known to be one to the compiler,
// which keeps what that lane computes in uniform registers).
__device__ __forceinline__ bool elected() {
  unsigned is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of the same place in another CTA of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float peer_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// Relaxed: what is handed over is tensor memory, ordered by tmem_fence_before.
// (A release at cluster scope waits for the thread's global stores too: a third
// of the time of a kernel whose epilogue stores.)
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
// Shared-memory operand descriptor of a 128-byte swizzled tile.  K-major:
// rows of 64 elements, eight rows to a 1024-byte group (strideBytes).
// MN-major: slabs 64 elements wide, leadBytes apart, whose k rows are 128
// bytes each, eight to a 1024-byte group.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, unsigned leadBytes,
                                                 unsigned strideBytes) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(leadBytes >> 4) << 16 |
         (uint64_t)(strideBytes >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t acc, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(acc),
        "l"(a), "l"(b), "r"(idesc), "r"((unsigned)accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(acc),
        "l"(a), "l"(b), "r"(idesc), "r"((unsigned)accumulate)
        : "memory");
  }
}
// Arrives on `bar` (in both CTAs of a pair) when the products issued so far
// are done.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar, uint16_t pairMask) {
  if constexpr (PAIR) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"(pairMask)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
  }
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
// 32 columns of the warp's 32 accumulator rows: lane = row.  The values are
// there after tmem_wait, through which they are passed so that nothing uses
// them earlier.
__device__ __forceinline__ void tmem_issue32(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
// The same for 16 columns, in one go.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  tmem_issue32(addr, v);
  tmem_wait(v);
}
__device__ __forceinline__ float tmem_load1(uint32_t addr) {
  uint32_t r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r)
      : "r"(addr)
      : "memory");
  return __uint_as_float(r);
}
// A warp's rows of a finished accumulator in tensor memory; called by whole
// warps.  Without a product (K = 0) the sums are zero and it is not read.
struct TmemAcc {
  static constexpr int kStep = 32;  // columns best fetched at a time
  uint32_t addr;
  bool summed;
  __device__ __forceinline__ void operator()(int c, float (&v)[32]) const {
    __syncwarp();
    if (summed) {
      tmem_load32(addr + (unsigned)c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.0f;
    }
  }
  // every lane names a column of its own row (or a negative number: none)
  // and f(value) is called by the lanes that named one
  template <class F>
  __device__ __forceinline__ void pick(int c, F f) const {
    unsigned left = __ballot_sync(0xffffffffu, c >= 0);
    const unsigned lane = threadIdx.x % 32;
    while (left) {
      const int src = __ffs(left) - 1;
      left &= left - 1;
      const int at = __shfl_sync(0xffffffffu, c, src);
      const float x = summed ? tmem_load1(addr + (unsigned)at) : 0.0f;
      if (lane == (unsigned)src) f(x);
      __syncwarp();
    }
  }
};

// The same rows already in registers (N columns from `first`); the columns
// asked for are constants once the epilogue's loops are unrolled.
template <int N>
struct RegAcc {
  static constexpr int kStep = 16;
  const float (&sum)[N];
  int first;
  template <int K>
  __device__ __forceinline__ void operator()(int c, float (&v)[K]) const {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = sum[c - first + i];  // a constant once unrolled
  }
  template <class F>
  __device__ __forceinline__ void pick(int c, F f) const {
    if (c < 0) return;
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)  // a select each: no indexed registers
      asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, %2;\n\t@p mov.f32 %0, %3;\n\t}"
          : "+f"(x)
          : "r"(c - first), "r"(i), "f"(sum[i]));
    f(x);
  }
};

// Instruction descriptor of kind::f16 with fp32 accumulators.
template <typename T>
__host__ __device__ constexpr uint32_t mma_idesc(int m, int n, bool aMn, bool bMn) {
  const uint32_t format = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return 1u << 4 | format << 7 | format << 10 | (uint32_t)aMn << 15 | (uint32_t)bMn << 16 |
         (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

template <int BN, int PARTS, bool PAIR, int AUX = 0>
struct GemmShape {
  static constexpr int kABytes = kTileM * kTileK * 2;
  static constexpr int kBRows = PAIR ? BN / 2 : BN;
  static constexpr int kBBytes = kBRows * kTileK * 2;
  static constexpr int kStageBytes = PARTS * (kABytes + kBBytes);
  static constexpr int kTileRows = PAIR ? 2 * kTileM : kTileM;
  // Two accumulators.  With two planes three, since they change hands every
  // few slices (three cover the way there and back: 0.47 us a slice instead of
  // 0.57), and one more for the products of a low plane, which are summed
  // apart over the whole tile (their size would not survive being added one
  // by one).
  static constexpr int kAccs = PARTS == 2 ? 3 : 2;
  static constexpr int kTmem = 2 * PARTS * BN;
  static constexpr int kStages = (kGemmSmem - 2048 - AUX) / kStageBytes;
  // alignment, the stages, the epilogue's tiles
  static constexpr int kSmem = 2048 + kStages * kStageBytes + AUX;
  static_assert(kStages >= 2 && kTmem <= 512, "too large");
  static_assert(kStages * kStageBytes >= kTileM * BN * 4, "a share's sums do not fit");
};

// An epilogue that reads and writes 16-bit tiles (Epi::kAux) works on units of
// 32 columns: one of warps 2 and 3 loads a unit's tiles into shared memory,
// the four warps of its half of the accumulator change them in place, and the
// same helper warp stores them.  Two buffers take turns, so a unit's copies
// overlap the work on the other.  (Read and written by each thread straight
// from memory, row by row, these tiles took more time than the products: 32
// rows are 32 lines an access.)
constexpr int kAuxCols = 32;
constexpr int kAuxTile = kTileM * kAuxCols * 2;  // 128 rows of 64 bytes, 64-byte swizzled
constexpr int kAuxHalf = 2 * 2 * kAuxTile;       // two buffers of two planes
struct AuxArgs {
  CUtensorMap in[2], out[2];  // the planes as 32 x 128 tiles
  int nIn, nOut;              // planes loaded and stored
};
struct AuxTile {
  uint32_t smem;
  // 16 bytes (8 columns) of a row
  __device__ __forceinline__ uint32_t piece(int plane, int row, int i) const {
    return smem + (unsigned)(plane * kAuxTile + row * 64 + ((i ^ (row >> 1 & 3)) << 4));
  }
};

// Blocks of 2048 rows are walked column by column, so that the rows' and
// columns' operands of the tiles in flight stay in L2.
// Tiles of a triangle's block row i: those whose first column is not above
// its last row.
__host__ __device__ __forceinline__ int triangle_row(int i, int rows, int cols) {
  return ((i + 1) * rows + cols - 1) / cols;
}
template <int ROWS, int BN>
__device__ __forceinline__ Tile tile_of(int t, int tilesM, int tilesN, bool triangle) {
  Tile o;
  if (triangle) {
    int per = 0;
    for (int i = 0; i < tilesM; ++i) per += min(triangle_row(i, ROWS, BN), tilesN);
    o.z = t / per;
    t -= o.z * per;
    int i = 0;
    for (int n; t >= (n = min(triangle_row(i, ROWS, BN), tilesN)); ++i) t -= n;
    o.m0 = i * ROWS;
    o.n0 = t * BN;
    return o;
  }
  const int per = tilesM * tilesN;
  o.z = t / per;
  t -= o.z * per;
  constexpr int kGroup = 2048 / ROWS;
  const int group = t / (kGroup * tilesN);
  const int rows = min(kGroup, tilesM - group * kGroup);
  t -= group * kGroup * tilesN;
  o.n0 = t / rows * BN;
  o.m0 = (group * kGroup + t % rows) * ROWS;
  return o;
}

// Epi: struct with `Args` (kernel parameter) and
//   static __device__ void run(const Args&, const GemmArgs&, const Tile&, int row, int col0,
//                              int M, const Acc& acc)
// (templates: int COLS, class Acc) called by every thread of the epilogue warps for its accumulator row `row`
// (of the tile) and its columns [col0, col0 + COLS) of the tile; acc(c, v)
// fetches the 32 accumulator columns from c.  Epi::kAux (without SPLIT):
// unit(e, g, o, row, n, c, M, acc, tile) in place of run, for the 32 columns n
// of the product, c of the tile, unless skip(g, o, n, M), which then holds for
// the rest of the tile too; e.aux names the planes.
//
// CHUNK > 0: the tensor cores truncate where they add a product to the
// accumulator (one addition per 16 k), an error that grows with the length of
// the sum.  Every CHUNK slices of 64 the accumulator is handed to the
// epilogue warps, which add the partial sums in registers with rounding; the
// next chunk is summed meanwhile in the other accumulator.
template <typename T, int BN, int PARTS, bool AMN, bool BMN, int CHUNK, bool PAIR, bool SPLIT,
          class Epi>
__global__ void __launch_bounds__(128 + 32 * Epi::kWarps, 1)
    gemm_kernel(const __grid_constant__ GemmArgs g, const __grid_constant__ typename Epi::Args e) {
  constexpr bool kAux = Epi::kAux && !SPLIT;
  using Shape = GemmShape<BN, PARTS, PAIR, kAux ? 2 * kAuxHalf : 0>;
  static_assert(PARTS == 1 || CHUNK > 0, "two planes are summed in the epilogue warps");
  constexpr int kStages = Shape::kStages;
  constexpr int kCtas = PAIR ? 2 : 1;  // that share a tile's products
  extern __shared__ unsigned char smemRaw[];
  constexpr int kAccs = Shape::kAccs, kEpilogueWarps = Epi::kWarps;
  constexpr int kGroups = kEpilogueWarps / 4;  // of four warps: the rows of the accumulator
  constexpr int kPart = BN / kGroups;          // columns of a group
  static_assert(!kAux || kGroups == 2, "one helper warp per group");
  __shared__ alignas(8) uint64_t bars[2 * kStages + 2 * kAccs + 2 + (kAux ? 8 : 0)];
  __shared__ uint32_t tmemBase;
  __shared__ volatile int abortFlag;

  // (a shuffle, so that the role is known to be the warp's)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t rank = PAIR || SPLIT ? cluster_rank() : 0u;
  const uint32_t inPair = PAIR ? rank & 1u : 0u;
  const bool leader = inPair == 0;
  const uint16_t pairMask = (uint16_t)(3u << (rank & ~1u));
  const uint32_t stage0 = (smem_addr(smemRaw) + 1023) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto accFull = [&](int i) { return bar0 + 8u * (2 * kStages + i); };
  auto accEmpty = [&](int i) { return bar0 + 8u * (2 * kStages + kAccs + i); };
  const uint32_t drained = bar0 + 8u * (2 * kStages + 2 * kAccs), lowEmpty = drained + 8u;
  auto auxFull = [&](int half, int i) { return lowEmpty + 8u * (1 + 2 * half + i); };
  auto auxDone = [&](int half, int i) { return lowEmpty + 8u * (5 + 2 * half + i); };
  const uint32_t aux0 = stage0 + (unsigned)(kStages * Shape::kStageBytes);
  auto wait = [&](uint32_t bar, unsigned parity, bool honorAbort = true) {
    return wait_phase(bar, parity, &abortFlag, honorAbort, g.timeoutNs);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(accFull(i), 1);
      mbar_init(accEmpty(i), kEpilogueWarps * kCtas);
    }
    mbar_init(drained, 1);
    mbar_init(lowEmpty, kEpilogueWarps * kCtas);
    for (int i = 0; kAux && i < 4; ++i) {
      mbar_init(auxFull(i / 2, i % 2), 1);
      mbar_init(auxDone(i / 2, i % 2), 4);
    }
    abortFlag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async;" ::: "memory");
  }
  if (warp == 1 && elected()) {  // the copies' descriptors, before the data is there
    for (int p = 0; p < PARTS; ++p) {
      prefetch_map(&g.a[p]);
      prefetch_map(&g.b[p]);
    }
    if constexpr (kAux)
      for (int p = 0; p < 2; ++p) {
        if (p < e.aux.nIn) prefetch_map(&e.aux.in[p]);
        if (p < e.aux.nOut) prefetch_map(&e.aux.out[p]);
      }
  }
  if (warp == 2) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&tmemBase)),
                   "r"(Shape::kTmem)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&tmemBase)),
                   "r"(Shape::kTmem)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  tmem_fence_before();
  __syncthreads();
  if constexpr (PAIR || SPLIT) cluster_sync();  // the peers' barriers are set up
  tmem_fence_after();
  const uint32_t tmem = tmemBase;
  pdl_launch();
  pdl_wait();

  const int M = g.dynM ? min(*g.dynM, g.M) : g.M;
  const int K = g.dynK ? min(*g.dynK, g.K) : g.K;
  const int tilesM = (M + Shape::kTileRows - 1) / Shape::kTileRows, tilesN = (g.N + BN - 1) / BN;
  const int slices = (K + kTileK - 1) / kTileK;
  int tiles = tilesM * tilesN;
  if (g.triangle) {
    tiles = 0;
    for (int i = 0; i < tilesM; ++i) tiles += min(triangle_row(i, Shape::kTileRows, BN), tilesN);
  }
  tiles *= g.batch;
  // This CTA's tiles and its share [kb0, kb1) of their slices of k.
  const int shares = SPLIT ? (int)cluster_size() / kCtas : 1;
  const int share = SPLIT ? (int)rank / kCtas : 0;
  const int kb0 = SPLIT ? (int)((long long)slices * share / shares) : 0;
  const int kb1 = SPLIT ? (int)((long long)slices * (share + 1) / shares) : slices;
  const int blocks = kb1 - kb0;
  const int chunk = CHUNK ? CHUNK : max(blocks, 1);
  const int firstTile = (int)blockIdx.x / (kCtas * shares);
  const int tileStep = SPLIT ? tiles + 1 : (int)gridDim.x / kCtas;  // SPLIT: one tile

  if (warp == 0) {
    int s = 0, turn = 0;
    bool ok = true;
    long long issued = 0;
    // a pair's copies are counted on the barriers of its first CTA
    const uint32_t landed0 = PAIR ? peer_addr(full(0), rank & ~1u) : full(0);
    for (int t = firstTile; ok && t < tiles; t += tileStep) {
      const Tile o = tile_of<Shape::kTileRows, BN>(t, tilesM, tilesN, g.triangle);
      const int m0 = o.m0 + (int)inPair * kTileM, n0 = o.n0 + (int)inPair * Shape::kBRows;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(0xffffffffu, wait(empty(s), turn ^ 1)) != 0;
        if (!ok) break;
        if (elected()) {
          if (leader) mbar_arrive_expect_tx(full(s), kCtas * Shape::kStageBytes);
          uint32_t dst = stage0 + (unsigned)s * Shape::kStageBytes;
          const int k0 = kb * kTileK;
          const uint32_t landed = landed0 + 8u * s;
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            if (AMN) {
#pragma unroll
              for (int i = 0; i < kTileM / 64; ++i)
                tensor_load<PAIR>(dst + i * (64 * kTileK * 2), &g.a[p], m0 + i * 64, k0, o.z,
                                  landed);
            } else {
              tensor_load<PAIR>(dst, &g.a[p], k0, m0, o.z, landed);
            }
            dst += Shape::kABytes;
          }
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            if (BMN) {
#pragma unroll
              for (int i = 0; i < Shape::kBRows / 64; ++i)
                tensor_load<PAIR>(dst + i * (64 * kTileK * 2), &g.b[p], n0 + i * 64, k0, o.z,
                                  landed);
            } else {
              tensor_load<PAIR>(dst, &g.b[p], k0, n0, o.z, landed);
            }
            dst += Shape::kBBytes;
          }
        }
        __syncwarp();
        ++issued;
        if (++s == kStages) s = 0, turn ^= 1;
      }
    }
    // The last slices' stages are handed back before the CTA leaves: in a pair
    // that arrival comes from the other CTA's products and would otherwise
    // land in whatever runs on this SM next.
    for (long long i = issued > kStages ? issued - kStages : 0; ok && i < issued; ++i)
      ok = __all_sync(0xffffffffu, wait(empty((int)(i % kStages)), (int)(i / kStages & 1))) != 0;
    if (!ok) {
      raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
      // copies in flight land before the CTA's shared memory is given up (in a
      // pair they are counted on the first CTA's barriers, which waits for both)
      if (leader)
        for (long long i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
          wait(full((int)(i % kStages)), (int)(i / kStages & 1), false);
    }
  } else if (warp == 1 && leader) {
    // the whole warp walks the slices and waits, one lane issues
    constexpr uint32_t idesc = mma_idesc<T>(Shape::kTileRows, BN, AMN, BMN);
    constexpr unsigned kSlab = 64 * kTileK * 2;  // MN-major: bytes of a 64-wide slab
    // one product takes 16 k: 32 bytes along a K-major row, 16 rows of 128
    // bytes of an MN-major slab
    constexpr unsigned aStep = (AMN ? 16 * 128 : 32) >> 4, bStep = (BMN ? 16 * 128 : 32) >> 4;
    const uint64_t aDesc0 = operand_desc(stage0, AMN ? kSlab : 16, 1024);
    const uint64_t bDesc0 = operand_desc(stage0 + PARTS * Shape::kABytes, BMN ? kSlab : 16, 1024);
    int s = 0, turn = 0, buf = 0, bufTurn = 0, lowTurn = 0;
    bool ok = true;
    auto ready = [&](uint32_t bar, unsigned parity) {
      const bool mine = wait(bar, parity);
      return __all_sync(0xffffffffu, mine) != 0;
    };
    for (int t = firstTile; ok && t < tiles; t += tileStep) {
      if (PARTS == 2 && blocks) {
        ok = ready(lowEmpty, lowTurn ^ 1);
        lowTurn ^= 1;
      }
      for (int c0 = 0; ok && c0 < blocks; c0 += chunk) {
        ok = ready(accEmpty(buf), bufTurn ^ 1);
        if (!ok) break;
        tmem_fence_after();
        const uint32_t acc = tmem + (unsigned)(buf * BN), low = tmem + (unsigned)(kAccs * BN);
        const int c1 = min(c0 + chunk, blocks);
        for (int kb = c0; kb < c1; ++kb) {
          ok = ready(full(s), turn);
          if (!ok) break;
          tmem_fence_after();
          if (elected()) {
            const uint64_t at = (uint64_t)((unsigned)s * (Shape::kStageBytes >> 4));
#pragma unroll
            for (int p = 0; p < (PARTS == 2 ? 3 : 1); ++p) {
              const uint64_t aDesc = aDesc0 + at + (p == 2 ? Shape::kABytes >> 4 : 0);
              const uint64_t bDesc = bDesc0 + at + (p == 1 ? Shape::kBBytes >> 4 : 0);
#pragma unroll
              for (int k = 0; k < kTileK / 16; ++k)
                mma_f16<PAIR>(p ? low : acc, aDesc + k * aStep, bDesc + k * bStep, idesc,
                              p ? kb | (p == 2) | k : (kb - c0) | k);
            }
            mma_commit<PAIR>(empty(s), pairMask);
            if (kb + 1 == c1) mma_commit<PAIR>(accFull(buf), pairMask);
          }
          __syncwarp();
          if (++s == kStages) s = 0, turn ^= 1;
        }
        if (!ok) break;
        if (++buf == kAccs) buf = 0, bufTurn ^= 1;
      }
    }
    if (!ok) {
      raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
      if (elected()) {
        mma_commit<PAIR>(drained, pairMask);
        wait(drained, 0, false);
      }
    }
  } else if (warp >= 4) {
    const int quad = warp % 4, half = (warp - 4) / 4;
    const int row = quad * 32 + lane;
    const uint32_t quadBase = tmem + ((uint32_t)(quad * 32) << 16);
    int buf = 0, bufTurn = 0;
    // the next accumulator, or false when the warp has to leave, as a whole
    auto next = [&]() {
      const bool ready = wait(accFull(buf), bufTurn);
      if (!__all_sync(0xffffffffu, ready)) {
        raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
        return false;
      }
      tmem_fence_after();
      return true;
    };
    auto hand_back = [&](uint32_t bar) {
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) {
          peer_arrive(peer_addr(bar, rank & ~1u));
        } else {
          mbar_arrive(bar);
        }
      }
    };
    auto release = [&]() {
      hand_back(accEmpty(buf));
      if (++buf == kAccs) buf = 0, bufTurn ^= 1;
    };
    int unit = 0;  // of the Aux tiles
    auto units = [&](const Tile& o, const auto& acc) {
      if constexpr (kAux) {
#pragma unroll
        for (int c = 0; c < kPart; c += kAuxCols) {
          const int n = o.n0 + half * kPart + c, b = unit & 1;
          if (Epi::skip(g, o, n, M)) break;
          const bool there = wait(auxFull(half, b), (unsigned)(unit >> 1 & 1));
          if (!__all_sync(0xffffffffu, there)) {
            raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
            return false;
          }
          Epi::unit(e, g, o, row, n, half * kPart + c, M, acc,
                    AuxTile{aux0 + (unsigned)(half * kAuxHalf + b * (2 * kAuxTile))});
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(auxDone(half, b));
          ++unit;
        }
      }
      return true;
    };
    for (int t = firstTile; t < tiles; t += tileStep) {
      Tile o = tile_of<Shape::kTileRows, BN>(t, tilesM, tilesN, g.triangle);
      o.m0 += (int)inPair * kTileM;
      bool left = false;
      // a share's sums: [column][row] in the stages' memory, free by now
      auto put = [&](int c, const float(&v)[32]) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage0 + 4u * ((c + i) * kTileM + row)),
                       "f"(v[i])
                       : "memory");
      };
      if constexpr (CHUNK > 0) {
        float sum[kPart];
#pragma unroll
        for (int i = 0; i < kPart; ++i) sum[i] = 0.0f;
        for (int c0 = 0; c0 < blocks; c0 += chunk) {
          left = !next();
          if (left) break;
          auto add = [&](uint32_t at) {
            if constexpr (kEpilogueWarps == 8) {  // two loads in flight
#pragma unroll
              for (int c = 0; c < kPart; c += 64) {
                float v[32], w[32];
                tmem_issue32(at + (unsigned)c, v);
                tmem_issue32(at + (unsigned)c + 32, w);
                tmem_wait(v);
                tmem_wait(w);
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[c + i] += v[i], sum[c + 32 + i] += w[i];
              }
            } else {
#pragma unroll
              for (int c = 0; c < kPart; c += 16) {
                float v[16];
                tmem_load16(at + (unsigned)c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[c + i] += v[i];
              }
            }
          };
          add(quadBase + (unsigned)(buf * BN + half * kPart));
          release();
          if (PARTS == 2 && c0 + chunk >= blocks) {  // done with the last slice's
            add(quadBase + (unsigned)(kAccs * BN + half * kPart));
            hand_back(lowEmpty);
          }
        }
        if (left) break;
        const RegAcc<kPart> acc{sum, half * kPart};
        if constexpr (SPLIT) {
#pragma unroll
          for (int c = 0; c < kPart; c += 32) {
            float v[32];
            acc(half * kPart + c, v);
            put(half * kPart + c, v);
          }
        } else if constexpr (kAux) {
          if (!units(o, acc)) break;
        } else {
          Epi::template run<kPart>(e, g, o, row, half * kPart, M, acc);
        }
      } else {
        if (blocks && !next()) break;
        const TmemAcc acc{quadBase + (unsigned)(buf * BN), blocks != 0};
        if constexpr (SPLIT) {
#pragma unroll
          for (int c = 0; c < kPart; c += 32) {
            float v[32];
            acc(half * kPart + c, v);
            put(half * kPart + c, v);
          }
        } else if constexpr (kAux) {
          if (!units(o, acc)) break;
        } else {
          Epi::template run<kPart>(e, g, o, row, half * kPart, M, acc);
        }
        if (blocks) release();
      }
    }
  } else if (kAux && warp >= 2) {
    if constexpr (kAux) {
      const int half = warp - 2;
      int unit = 0, atX[2] = {0, 0}, atY[2] = {0, 0}, atZ[2] = {0, 0};
      bool ok = true;
      auto tile_at = [&](int b, int p) {
        return aux0 + (unsigned)(half * kAuxHalf + b * (2 * kAuxTile) + p * kAuxTile);
      };
      // unit v has been worked on: stores its tiles, and waits until they
      // are read when its buffer is wanted again
      auto finish = [&](int v) {
        const int b = v & 1;
        ok = __all_sync(0xffffffffu, wait(auxDone(half, b), (unsigned)(v >> 1 & 1))) != 0;
        if (ok && e.aux.nOut && elected()) {
          for (int p = 0; p < e.aux.nOut; ++p)
            asm volatile(
                "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], "
                "[%4];" ::"l"(&e.aux.out[p]),
                "r"(atX[b]), "r"(atY[b]), "r"(atZ[b]), "r"(tile_at(b, p))
                : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncwarp();
      };
      for (int t = firstTile; ok && t < tiles; t += tileStep) {
        Tile o = tile_of<Shape::kTileRows, BN>(t, tilesM, tilesN, g.triangle);
        o.m0 += (int)inPair * kTileM;
        for (int c = 0; ok && c < kPart; c += kAuxCols) {
          const int n = o.n0 + half * kPart + c, b = unit & 1;
          if (Epi::skip(g, o, n, M)) break;
          if (unit >= 2) finish(unit - 2);
          if (!ok) break;
          if (elected()) {
            if (e.aux.nIn) {
              mbar_arrive_expect_tx(auxFull(half, b), (unsigned)(e.aux.nIn * kAuxTile));
              for (int p = 0; p < e.aux.nIn; ++p)
                tensor_load<false>(tile_at(b, p), &e.aux.in[p], n, o.m0, o.z, auxFull(half, b));
            } else {
              mbar_arrive(auxFull(half, b));
            }
          }
          __syncwarp();
          atX[b] = n, atY[b] = o.m0, atZ[b] = o.z;
          ++unit;
        }
      }
      for (int v = max(0, unit - 2); ok && v < unit; ++v) finish(v);
      if (!ok) {
        raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
        // loads in flight land before the CTA's shared memory is given up
        for (int v = max(0, unit - 2); v < unit; ++v)
          wait(auxFull(half, v & 1), (unsigned)(v >> 1 & 1), false);
      }
      if (elected()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      __syncwarp();
    }
  }
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync();  // all shares' sums are in place
    constexpr int kPieces = BN / 32;  // of 32 columns; four warps (row quadrants) each
    if (warp >= 4 && firstTile < tiles) {
      const int quad = warp % 4, row = quad * 32 + lane;
      Tile o = tile_of<Shape::kTileRows, BN>(firstTile, tilesM, tilesN, g.triangle);
      o.m0 += (int)inPair * kTileM;
      for (int group = share * kGroups + (warp - 4) / 4; group < kPieces;
           group += kGroups * shares) {
        float sum[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[i] = 0.0f;
        for (int from = 0; from < shares; ++from) {
          const uint32_t at = peer_addr(stage0, (uint32_t)(from * kCtas) + inPair) +
                              4u * (unsigned)(group * 32 * kTileM + row);
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[i] += peer_load(at + 4u * (unsigned)(i * kTileM));
        }
        Epi::template run<32>(e, g, o, row, group * 32, M, RegAcc<32>{sum, group * 32});
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  // no CTA leaves while a peer still reads its memory or arrives on its barriers
  if constexpr (PAIR || SPLIT) cluster_sync();
  if (warp == 2) {
    tmem_fence_after();
    if constexpr (PAIR) {
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(Shape::kTmem));
    } else {
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(Shape::kTmem));
    }
  }
}

// One product D = A B^T per batch entry: operands as they lie in memory.
struct Operand {
  const void *hi, *lo;  // lo: second plane (PARTS = 2)
  size_t ld;            // elements between rows
};
struct GemmSize {
  size_t M, N, K, batch;
  bool triangle;
};

template <int BN, bool PAIR>
size_t gemm_tiles(const GemmSize& z) {
  const size_t rows = PAIR ? 2 * kTileM : kTileM;
  const size_t tm = (z.M + rows - 1) / rows, tn = (z.N + BN - 1) / BN;
  size_t tiles = tm * tn;
  if (z.triangle) {
    tiles = 0;
    for (size_t i = 0; i < tm; ++i)
      tiles += std::min<size_t>(triangle_row((int)i, (int)rows, BN), tn);
  }
  return tiles * z.batch;
}

template <typename T, int BN, int PARTS, bool AMN, bool BMN, int CHUNK, bool PAIR, bool SPLIT,
          class Epi>
vr_result_t gemm_launch(const OpDevice& dev, const Operand& a, const Operand& b, const GemmSize& z,
                        const int* dynM, const int* dynK, typename Epi::Args& epi, int shares,
                        void* stream) {
  using Shape = GemmShape<BN, PARTS, PAIR, Epi::kAux && !SPLIT ? 2 * kAuxHalf : 0>;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const void* fn = (const void*)gemm_kernel<T, BN, PARTS, AMN, BMN, CHUNK, PAIR, SPLIT, Epi>;
  GemmArgs g = {};
  for (int i = 0; i < PARTS; ++i) {
    vr_result_t e = gemm_operand(&g.a[i], i ? a.lo : a.hi, bf16, AMN ? z.M : z.K,
                                 AMN ? z.K : z.M, z.batch, a.ld * 2, a.ld * 2 * (AMN ? z.K : z.M),
                                 AMN ? kTileK : kTileM);
    if (e != VR_SUCCESS) return e;
    e = gemm_operand(&g.b[i], i ? b.lo : b.hi, bf16, BMN ? z.N : z.K, BMN ? z.K : z.N, z.batch,
                     b.ld * 2, b.ld * 2 * (BMN ? z.K : z.N), BMN ? kTileK : Shape::kBRows);
    if (e != VR_SUCCESS) return e;
  }
  const vr_result_t e = gemm_prepare(fn, dev.device, Shape::kSmem);
  if (e != VR_SUCCESS) return e;
  g.M = (int)z.M;
  g.N = (int)z.N;
  g.K = (int)z.K;
  g.batch = (int)z.batch;
  g.dynM = dynM;
  g.dynK = dynK;
  g.triangle = z.triangle;
  g.status = dev.status;
  g.timeoutNs = dev.timeoutNs;
  constexpr size_t kCtas = PAIR ? 2 : 1;
  const size_t tiles = gemm_tiles<BN, PAIR>(z);
  const size_t groups = SPLIT ? tiles : std::min<size_t>(tiles, dev.sms / kCtas);
  const size_t cluster = kCtas * (SPLIT ? (size_t)shares : 1);
  void* args[] = {&g, &epi};
  return op_launch(fn, dim3((unsigned)(groups * cluster)), dim3(128 + 32 * Epi::kWarps), args, Shape::kSmem,
                   stream, (int)cluster);
}

}  // namespace vr
