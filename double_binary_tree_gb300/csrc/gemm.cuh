// Matrix products on the fifth-generation tensor cores (tcgen05) with a
// fused epilogue: the base of the training operators.
//
//   D[z][m][n] = sum_k A[z][m][k] B[z][n][k],  16-bit operands, fp32 sums
//
// One persistent CTA per SM, 128 x BN tiles.  Warp 0 moves 64-deep slices of
// A and B into a ring of shared-memory stages with tensor copies (TMA), warp
// 1 issues the products on them, warps 4-11 read finished accumulators from
// tensor memory and run the epilogue.  Two accumulators take turns, so the
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
// Every wait is bounded.  A CTA that gives up records VR_ERR_TIMEOUT, waits
// (bounded) for its copies and products in flight, frees its tensor memory
// and returns.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "staged.cuh"

namespace vr {

constexpr int kTileM = 128;
constexpr int kTileK = 64;  // 16-bit elements: one 128-byte swizzled row
constexpr int kGemmThreads = 384;
constexpr int kEpilogueWarps = 8;
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

__device__ __forceinline__ void tensor_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
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
__device__ __forceinline__ void mma_f16(uint32_t acc, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(acc),
      "l"(a), "l"(b), "r"(idesc), "r"((unsigned)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
// 32 columns of the warp's 32 accumulator rows: lane = row.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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
  const float (&sum)[N];
  int first;
  __device__ __forceinline__ void operator()(int c, float (&v)[32]) const {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = sum[c - first + i];
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

template <int BN, int PARTS>
struct GemmShape {
  static constexpr int kABytes = kTileM * kTileK * 2;
  static constexpr int kBBytes = BN * kTileK * 2;
  static constexpr int kStageBytes = PARTS * (kABytes + kBBytes);
  // columns of an accumulator: with two planes the products of a low plane
  // are summed apart (their size would not survive being added one by one)
  static constexpr int kAcc = PARTS * BN;
  static constexpr int kStages = (kGemmSmem - 2048) / kStageBytes;
  static constexpr int kSmem = 2048 + kStages * kStageBytes;  // header, alignment
  static_assert(kStages >= 2 && 2 * kAcc <= 512, "too large");
};

// Blocks of 16 tile rows are walked column by column, so that the rows' and
// columns' operands of the tiles in flight stay in L2.
__device__ __forceinline__ Tile tile_of(int t, int tilesM, int tilesN, int BN, bool triangle) {
  Tile o;
  int per;
  if (triangle) {
    // row i holds the tiles whose first column is not above its last row
    const int ratio = BN / kTileM;
    per = 0;
    for (int i = 0; i < tilesM; ++i) per += i / ratio + 1;
    o.z = t / per;
    t -= o.z * per;
    int i = 0;
    while (t >= i / ratio + 1) t -= i / ratio + 1, ++i;
    o.m0 = i * kTileM;
    o.n0 = t * BN;
    return o;
  }
  per = tilesM * tilesN;
  o.z = t / per;
  t -= o.z * per;
  constexpr int kGroup = 16;
  const int group = t / (kGroup * tilesN);
  const int rows = min(kGroup, tilesM - group * kGroup);
  t -= group * kGroup * tilesN;
  o.n0 = t / rows * BN;
  o.m0 = (group * kGroup + t % rows) * kTileM;
  return o;
}

// Epi: struct with `Args` (kernel parameter) and
//   static __device__ void run(const Args&, const GemmArgs&, const Tile&, int row, int col0,
//                              int M, const Acc& acc)
// (templates: int COLS, class Acc) called by every thread of the epilogue warps for its accumulator row `row`
// (of the tile) and its columns [col0, col0 + COLS) of the tile; acc(c, v)
// fetches the 32 accumulator columns from c.
//
// CHUNK > 0: the tensor cores truncate where they add a product to the
// accumulator (one addition per 16 k), an error that grows with the length of
// the sum.  Every CHUNK slices of 64 the accumulator is handed to the
// epilogue warps, which add the partial sums in registers with rounding; the
// next chunk is summed meanwhile in the other accumulator.
template <typename T, int BN, int PARTS, bool AMN, bool BMN, int CHUNK, class Epi>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ GemmArgs g, const __grid_constant__ typename Epi::Args e) {
  using Shape = GemmShape<BN, PARTS>;
  static_assert(PARTS == 1 || CHUNK > 0, "two planes are summed in the epilogue warps");
  extern __shared__ unsigned char smemRaw[];
  __shared__ alignas(8) uint64_t bars[2 * Shape::kStages + 5];
  __shared__ uint32_t tmemBase;
  __shared__ volatile int abortFlag;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t stage0 = (smem_addr(smemRaw) + 1023) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (Shape::kStages + s); };
  auto accFull = [&](int i) { return bar0 + 8u * (2 * Shape::kStages + i); };
  auto accEmpty = [&](int i) { return bar0 + 8u * (2 * Shape::kStages + 2 + i); };
  const uint32_t drained = bar0 + 8u * (2 * Shape::kStages + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < Shape::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(accFull(i), 1);
      mbar_init(accEmpty(i), kEpilogueWarps);
    }
    mbar_init(drained, 1);
    abortFlag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmemBase)),
                 "r"(2 * Shape::kAcc)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmemBase;
  pdl_launch();
  pdl_wait();

  const int M = g.dynM ? min(*g.dynM, g.M) : g.M;
  const int K = g.dynK ? min(*g.dynK, g.K) : g.K;
  const int tilesM = (M + kTileM - 1) / kTileM, tilesN = (g.N + BN - 1) / BN;
  const int blocks = (K + kTileK - 1) / kTileK;
  const int chunk = CHUNK ? CHUNK : max(blocks, 1);
  constexpr int kHalf = BN / 2;  // columns of an epilogue warp
  int tiles = tilesM * tilesN;
  if (g.triangle) {
    tiles = 0;
    for (int i = 0; i < tilesM; ++i) tiles += i / (BN / kTileM) + 1;
  }
  tiles *= g.batch;

  if (warp == 0 && lane == 0) {
    int s = 0, turn = 0;
    bool ok = true;
    long long issued = 0;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const Tile o = tile_of(t, tilesM, tilesN, BN, g.triangle);
      for (int kb = 0; kb < blocks; ++kb) {
        ok = wait_phase(empty(s), turn ^ 1, &abortFlag, true, g.timeoutNs);
        if (!ok) break;
        mbar_arrive_expect_tx(full(s), Shape::kStageBytes);
        uint32_t dst = stage0 + (unsigned)s * Shape::kStageBytes;
        const int k0 = kb * kTileK;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
          if (AMN) {
#pragma unroll
            for (int i = 0; i < kTileM / 64; ++i)
              tensor_load(dst + i * (64 * kTileK * 2), &g.a[p], o.m0 + i * 64, k0, o.z, full(s));
          } else {
            tensor_load(dst, &g.a[p], k0, o.m0, o.z, full(s));
          }
          dst += Shape::kABytes;
        }
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
          if (BMN) {
#pragma unroll
            for (int i = 0; i < BN / 64; ++i)
              tensor_load(dst + i * (64 * kTileK * 2), &g.b[p], o.n0 + i * 64, k0, o.z, full(s));
          } else {
            tensor_load(dst, &g.b[p], k0, o.n0, o.z, full(s));
          }
          dst += Shape::kBBytes;
        }
        ++issued;
        if (++s == Shape::kStages) s = 0, turn ^= 1;
      }
    }
    if (!ok) {
      raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
      // copies in flight land before the CTA's shared memory is given up
      for (long long i = issued > Shape::kStages ? issued - Shape::kStages : 0; i < issued; ++i)
        wait_phase(full((int)(i % Shape::kStages)), (int)(i / Shape::kStages & 1), &abortFlag,
                   false, g.timeoutNs);
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = mma_idesc<T>(kTileM, BN, AMN, BMN);
    constexpr unsigned kSlab = 64 * kTileK * 2;  // MN-major: bytes of a 64-wide slab
    // one product takes 16 k: 32 bytes along a K-major row, 16 rows of 128
    // bytes of an MN-major slab
    constexpr unsigned aStep = (AMN ? 16 * 128 : 32) >> 4, bStep = (BMN ? 16 * 128 : 32) >> 4;
    int s = 0, turn = 0, buf = 0, bufTurn = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      for (int kb0 = 0; ok && kb0 < blocks; kb0 += chunk) {
        ok = wait_phase(accEmpty(buf), bufTurn ^ 1, &abortFlag, true, g.timeoutNs);
        if (!ok) break;
        tmem_fence_after();
        const uint32_t acc = tmem + (unsigned)buf * Shape::kAcc;
        const int kb1 = min(kb0 + chunk, blocks);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait_phase(full(s), turn, &abortFlag, true, g.timeoutNs);
          if (!ok) break;
          tmem_fence_after();
          const uint32_t base = stage0 + (unsigned)s * Shape::kStageBytes;
#pragma unroll
          for (int p = 0; p < (PARTS == 2 ? 3 : 1); ++p) {
            const uint32_t aAt = base + (p == 2 ? Shape::kABytes : 0);
            const uint32_t bAt = base + PARTS * Shape::kABytes + (p == 1 ? Shape::kBBytes : 0);
            const uint64_t aDesc = operand_desc(aAt, AMN ? kSlab : 16, 1024);
            const uint64_t bDesc = operand_desc(bAt, BMN ? kSlab : 16, 1024);
#pragma unroll
            for (int k = 0; k < kTileK / 16; ++k)
              mma_f16(p ? acc + BN : acc, aDesc + k * aStep, bDesc + k * bStep, idesc,
                      (kb - kb0) | (p == 2) | k);
          }
          mma_commit(empty(s));
          if (++s == Shape::kStages) s = 0, turn ^= 1;
        }
        if (!ok) break;
        mma_commit(accFull(buf));
        if (++buf == 2) buf = 0, bufTurn ^= 1;
      }
    }
    if (!ok) {
      raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
      mma_commit(drained);
      wait_phase(drained, 0, &abortFlag, false, g.timeoutNs);
    }
  } else if (warp >= 4) {
    const int quad = warp % 4, half = (warp - 4) / 4;
    int buf = 0, bufTurn = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const Tile o = tile_of(t, tilesM, tilesN, BN, g.triangle);
      const uint32_t quadBase = tmem + ((uint32_t)(quad * 32) << 16);
      const int row = quad * 32 + lane;
      // the next accumulator, or false when the warp has to leave
      auto next = [&]() {
        const bool ready = wait_phase(accFull(buf), bufTurn, &abortFlag, true, g.timeoutNs);
        if (!__all_sync(0xffffffffu, ready)) {  // as a whole
          raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
          return false;
        }
        tmem_fence_after();
        return true;
      };
      auto release = [&]() {
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(accEmpty(buf));
        if (++buf == 2) buf = 0, bufTurn ^= 1;
      };
      if (CHUNK) {
        float sum[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) sum[i] = 0.0f;
        bool left = false;
        for (int kb0 = 0; kb0 < blocks; kb0 += chunk) {
          left = !next();
          if (left) break;
#pragma unroll
          for (int c = 0; c < kHalf; c += 32) {
            float v[32];
            const uint32_t at = quadBase + (unsigned)(buf * Shape::kAcc + half * kHalf + c);
            tmem_load32(at, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c + i] += v[i];
            if (PARTS == 2) {
              tmem_load32(at + BN, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) sum[c + i] += v[i];
            }
          }
          release();
        }
        if (left) break;
        Epi::template run<kHalf>(e, g, o, row, half * kHalf, M,
                                 RegAcc<kHalf>{sum, half * kHalf});
      } else {
        if (blocks && !next()) break;
        Epi::template run<kHalf>(e, g, o, row, half * kHalf, M,
                                 TmemAcc{quadBase + (unsigned)(buf * Shape::kAcc), blocks != 0});
        if (blocks) release();
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 2) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(2 * Shape::kAcc));
  }
}

}  // namespace vr
