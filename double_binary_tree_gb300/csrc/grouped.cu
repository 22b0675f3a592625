// Matrix products grouped by expert (vr_grouped_linear) and their gradients
// (vr_grouped_linear_grad).
//
//   y_r = W_e(r) x_r;   dx_r = W_e(r)^T dy_r;   dW_e = sum_{r: e(r) = e} dy_r x_r^T
//
// Rows are sorted by group; how many each group has is known on the device
// only.  One launch takes the tiles of all groups: every CTA adds the counts up
// for itself (a microsecond or two, less than a launch that writes a table) and
// walks the tiles with the grid's stride, the roles of its warps those of the
// products of gemm.cuh: tensor copies, tcgen05 products, epilogue.
//
//   rows    (out, dX)  The weight's rows fill the 128 or 256 rows of a tile and a
//           group's rows are its columns, since an instruction takes any
//           multiple of 16 (pairs of CTAs: 32) of those: a group's last tile costs what it
//           holds.  (The other way round 64 groups of 512 rows on average pay
//           for 640: 2048 x 4096 in 400 us instead of the 286 of the peak.)  A group's
//           rows are cut into tiles of about the same size.  The accumulator then
//           holds the results transposed; they are turned on their way through
//           shared memory (stmatrix), so that a store covers 64 bytes of eight rows.
//   few     The same for few rows a group: up to 32 columns, so that nearly all
//           of shared memory holds weights on their way.
//   weight  (dW)  A sum over the group's rows.  The last slice of 64 reads on
//           into the next group; the rows behind the end, up to the next
//           multiple of the 16 that a product takes, are zeroed in shared memory
//           (in both operands: they may hold NaN).
//   both    dW's tiles and then dX's in one launch, where they are few.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "rows.cuh"

namespace vr {
namespace {

constexpr int kMostGroups = 1024;
constexpr int kGroupedSmem = 212 * 1024;  // the stages; the tables of the groups are beside them

enum Kind : int { kLinear, kGradRows, kGradWeight, kGradBoth };
struct Product {
  CUtensorMap a, b, c;  // c: dW, where its rows are 16-byte units
  int M, N, K;          // N (rows) or K (weight) is counted on the device
  int align;
  void* out;
  long long ld;         // elements between its rows
};
struct GroupedArgs {
  Product rows, weight;  // those that the kind has
  const int* counts;
  int groups, most;      // most: rows that the buffers have
  unsigned* status;
  unsigned long long timeoutNs;
};

// Results are stored through shared memory.  dW: a warp's 32 rows of 32 columns at a
// time, by a tensor copy, or, rows that are no 16-byte units, an element a lane.
// (Straight from registers a store covers 16 or 32 bytes of 32 rows, as many lines
// as there are rows, which took a third of the time where groups have a few hundred
// rows.)  Rows: 16 rows of 32 columns, 64 bytes of eight rows to a store.
constexpr int kStaged = 32 * 64;  // bytes of a warp's 32 rows

template <int BN, bool PAIR, bool WEIGHT>
struct GroupedShape {
  static constexpr int kABytes = kTileM * kTileK * 2;
  static constexpr int kBRows = PAIR ? BN / 2 : BN;
  static constexpr int kBBytes = kBRows * kTileK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kTileRows = PAIR ? 2 * kTileM : kTileM;
  static constexpr int kWarps = BN >= 128 ? 16 : 4;  // of the epilogue
  static constexpr int kStagedBytes = kWarps * (WEIGHT ? kStaged : kStaged / 2);
  static constexpr int kStages = (kGroupedSmem - kStagedBytes) / kStageBytes;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kStagedBytes;
  static constexpr int kTmem = 2 * BN;
  static constexpr int kGrain = PAIR ? 32 : 16;      // columns of an instruction
  static constexpr int kBox = BN < 128 ? 16 : 32;    // rows that a copy of a group's rows fetches
};

// t / d of small numbers, exactly: the quotient of t + 1/2 is at least 1 / 2d away
// from a whole number, its error (2.5 ulp, 2.5 2^-23 of it) is less for t < 2^20.
// (Integer divisions take a third of a microsecond of each tile.)
__device__ __forceinline__ int quotient(int t, int d) {
  return t < 1 << 20 ? (int)__fdividef((float)t + 0.5f, (float)d) : t / d;
}

// A tile: its group, its place in the product and its columns, a multiple of
// what an instruction takes; the group's rows [lo, hi).
struct GroupTile {
  int g, m0, n0, width, lo, hi;
  bool weight;  // of dW
};

// The same arrive and wait as mbar_arrive and mbar_test for what another CTA of
// the cluster wrote.
__device__ __forceinline__ void peer_arrive_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// Rows [from, to) of the MN-major slabs of a stage made zero by a warp, for
// products that are issued after this.  (A row is 128 bytes; the swizzle moves
// 16-byte pieces within it.)
template <int SLABS>
__device__ __forceinline__ void zero_rows(uint32_t stage, int from, int to, int lane) {
  constexpr unsigned kSlab = 64 * kTileK * 2;
#pragma unroll
  for (int slab = 0; slab < SLABS; ++slab)
    for (int i = from * 8 + lane; i < to * 8; i += 32)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(stage + slab * kSlab +
                                                                    (unsigned)(i * 16)),
                   "r"(0)
                   : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// 32 columns of a warp's 32 rows in its part of shared memory, as a 64-byte
// swizzled tile (no bank twice in a phase, neither by rows nor along them).
__device__ __forceinline__ uint32_t staged_piece(uint32_t staged, int row, int i) {
  return staged + (unsigned)(row * 64 + ((i ^ (row >> 1 & 3)) << 4));
}
template <typename T>
__device__ __forceinline__ void stage_rows(uint32_t staged, const float (&v)[32]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(staged_piece(staged, lane, i)),
                 "r"(pack2<T>(v[8 * i], v[8 * i + 1])), "r"(pack2<T>(v[8 * i + 2], v[8 * i + 3])),
                 "r"(pack2<T>(v[8 * i + 4], v[8 * i + 5])), "r"(pack2<T>(v[8 * i + 6], v[8 * i + 7]))
                 : "memory");
}
// From there to memory: the tile's place is x, y, z of the map (what is outside is
// cut off).  The part may be written again after staged_free.
__device__ __forceinline__ void store_staged(uint32_t staged, const CUtensorMap* map, int x, int y,
                                             int z) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (threadIdx.x % 32 == 0) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
        "r"(x), "r"(y), "r"(z), "r"(staged)
        : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
__device__ __forceinline__ void staged_free() {
  if (threadIdx.x % 32 == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
// The same for rows that are no 16-byte units: `rows` and `cols` of them are there.
template <typename T>
__device__ __forceinline__ void store_staged(uint32_t staged, T* out, long long ld, int rows,
                                             int cols) {
  const int lane = threadIdx.x % 32;
  __syncwarp();
#pragma unroll 8
  for (int row = 0; row < min(rows, 32); ++row) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];"
                 : "=h"(x)
                 : "r"(staged_piece(staged, row, lane / 8) + lane % 8 * 2)
                 : "memory");
    if (lane < cols) reinterpret_cast<uint16_t*>(out + row * ld)[lane] = x;
  }
}

// 16 rows of the accumulator by 32 columns, as products hand them out: lane l has of
// each eight columns 2 (l % 4) and the next, of row l / 4, then of row l / 4 + 8.
__device__ __forceinline__ void tmem_issue_fragment(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_fragment(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
// A warp's 32 rows of the accumulator by 32 columns, turned: its columns are `rows`
// rows of the result, its rows `cols` columns (at most 32 of each).
template <typename T>
__device__ __forceinline__ void store_turned(uint32_t acc, uint32_t staged, T* out, long long ld,
                                             int rows, int cols, int align) {
  const int lane = threadIdx.x % 32;
  float a[16], b[16];  // rows 0 to 15 and 16 to 31
  tmem_issue_fragment(acc, a);
  tmem_issue_fragment(acc + (16u << 16), b);
  tmem_wait_fragment(a);
  tmem_wait_fragment(b);
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // 16 rows of the result
    __syncwarp();                // (what was there has been read)
#pragma unroll
    for (int i = 8 * h; i < 8 * h + 8; i += 4)  // eight rows: four 8 x 8 matrices, transposed
      asm volatile(
          "stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
              staged_piece(staged, i % 8 * 2 + lane % 8, lane / 8)),
          "r"(pack2<T>(a[i], a[i + 1])), "r"(pack2<T>(a[i + 2], a[i + 3])),
          "r"(pack2<T>(b[i], b[i + 1])), "r"(pack2<T>(b[i + 2], b[i + 3]))
          : "memory");
    __syncwarp();
    T* to = out + 16 * h * ld;
    const int n = rows - 16 * h;
    if (align >= 16 && cols >= 32) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = k * 8 + lane / 4;
        uint4 q;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "r"(staged_piece(staged, row, lane % 4))
                     : "memory");
        if (row < n) *reinterpret_cast<uint4*>(to + row * ld + lane % 4 * 8) = q;
      }
    } else {
#pragma unroll 8
      for (int row = 0; row < min(n, 16); ++row) {
        uint16_t x;
        asm volatile("ld.shared.u16 %0, [%1];"
                     : "=h"(x)
                     : "r"(staged_piece(staged, row, lane / 8) + lane % 8 * 2)
                     : "memory");
        if (lane < cols) reinterpret_cast<uint16_t*>(to + row * ld)[lane] = x;
      }
    }
  }
}

// A warp's 32 columns m of `rows` (at most 32) rows, 32 values a lane, one of
// each row.  align >= 4: two columns of a row in one store, which a pair of
// lanes make of each two rows.
template <typename T>
__device__ __forceinline__ void store_columns(T* out, long long ld, const float (&v)[32], int rows,
                                              int m, int M, int align) {
  if (align >= 4 && M % 2 == 0) {
    const bool odd = m & 1;
    uint32_t* p = reinterpret_cast<uint32_t*>(out + (odd ? ld : 0) + (m & ~1));
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint32_t mine = pack2<T>(v[i], v[i + 1]);
      const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
      const uint32_t both = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
      if (m < M && i + (int)odd < rows) p[i * (ld / 2)] = both;
    }
  } else {
    typename Ty<T>::Bits* p = reinterpret_cast<typename Ty<T>::Bits*>(out) + m;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (m < M && i < rows) p[i * ld] = Ty<T>::narrow(v[i]);
  }
}

template <typename T, int BN, int KIND, bool PAIR, int CHUNK>
__global__ void __launch_bounds__(128 + 32 * GroupedShape<BN, PAIR, (KIND >= kGradWeight)>::kWarps, 1)
    grouped_kernel(const __grid_constant__ GroupedArgs g) {
  constexpr bool kWeight = KIND >= kGradWeight, kRowsToo = KIND != kGradWeight;  // the tiles it has
  using Shape = GroupedShape<BN, PAIR, kWeight>;
  static_assert(!(kWeight && kRowsToo) || (PAIR && CHUNK == 0), "both: pairs, sums of one piece");
  constexpr bool kTurned = KIND != kLinear;  // rows: the weight's rows are the summed dimension
  constexpr int kStages = Shape::kStages, kCtas = PAIR ? 2 : 1, kRows = Shape::kTileRows;
  constexpr int kEpilogueWarps = Shape::kWarps, kGroups = kEpilogueWarps / 4;
  constexpr int kUnits = BN / 32 / kGroups;  // of 32 columns, for each group of four warps
  constexpr bool kTails = PAIR && kWeight;
  constexpr unsigned kSlab = 64 * kTileK * 2;  // MN-major: bytes of a 64-wide slab
  extern __shared__ unsigned char smemRaw[];
  __shared__ alignas(8) uint64_t bars[2 * kStages + 5 + (kTails ? 2 * kStages : 0)];
  __shared__ uint32_t tmemBase;
  __shared__ volatile int abortFlag;
  __shared__ int rowStart[kMostGroups + 1], tileStart[kMostGroups + 1], chosenCap;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const uint16_t pairMask = 3;
  const uint32_t stage0 = (smem_addr(smemRaw) + 1023) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto accFull = [&](int i) { return bar0 + 8u * (2 * kStages + i); };
  auto accEmpty = [&](int i) { return bar0 + 8u * (2 * kStages + 2 + i); };
  const uint32_t drained = bar0 + 8u * (2 * kStages + 4);
  // the end of a group on a pair: the CTA's own copies have landed in stage s; the
  // other CTA has zeroed its rows of it
  auto tailFull = [&](int s) { return bar0 + 8u * (2 * kStages + 5 + s); };
  auto tailPeer = [&](int s) { return bar0 + 8u * (3 * kStages + 5 + s); };
  auto wait = [&](uint32_t bar, unsigned parity, bool honorAbort = true) {
    return wait_phase(bar, parity, &abortFlag, honorAbort, g.timeoutNs);
  };
  auto all_wait = [&](uint32_t bar, unsigned parity) {
    const bool mine = wait(bar, parity);
    return __all_sync(0xffffffffu, mine) != 0;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
      if (kTails) {
        mbar_init(tailFull(s), 1);
        mbar_init(tailPeer(s), 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(accFull(i), 1);
      mbar_init(accEmpty(i), kEpilogueWarps * kCtas);
    }
    mbar_init(drained, 1);
    abortFlag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async;" ::: "memory");
  }
  if (warp == 1 && elected()) {
    if (kRowsToo) {
      prefetch_map(&g.rows.a);
      prefetch_map(&g.rows.b);
    }
    if (kWeight) {
      prefetch_map(&g.weight.a);
      prefetch_map(&g.weight.b);
      if (g.weight.align >= 16) prefetch_map(&g.weight.c);
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
  pdl_launch();
  pdl_wait();
  // tiles along the products' M, and along dW's N; dW's come first
  const int rowsM = (g.rows.M + kRows - 1) / kRows, weightM = (g.weight.M + kRows - 1) / kRows;
  const int weightN = (g.weight.N + BN - 1) / BN;
  const int weightTiles = kWeight ? g.groups * weightM * weightN : 0;
  if (warp == 3) {  // the groups' rows and tiles
    // Caps of a tile's columns, and the tiles of all groups with each.
    constexpr int kCaps = kWeight || BN < 128 ? 1 : 4;  // (both: dW has tiles enough)
    auto cap_of = [](int i) { return i == 0 ? BN : i == 1 ? 192 : i == 2 ? 128 : 64; };
    int rows = 0, sums[kCaps] = {};
#pragma unroll 4
    for (int e0 = 0; e0 < g.groups; e0 += 32) {
      const int e = e0 + lane;
      const int given = e < g.groups ? g.counts[e] : 0;
      // sums of what is given, held to the buffers' rows: what a bad count
      // reaches is reported, not read or written
      long long end = max(given, 0);
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const long long up = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += up;
      }
      end += rows;
      if (given < 0 || end > g.most) atomicCAS(g.status, 0u, (unsigned)VR_ERR_INVALID_ARGUMENT);
      const int hi = (int)min(end, (long long)g.most);
      const int up = __shfl_up_sync(0xffffffffu, hi, 1), lo = lane ? up : rows;
      if (e < g.groups) rowStart[e + 1] = hi;
      if constexpr (kCaps > 1) {
#pragma unroll
        for (int i = 0; i < kCaps; ++i) sums[i] += (hi - lo + cap_of(i) - 1) / cap_of(i);
      }
      rows = __shfl_sync(0xffffffffu, hi, 31);
    }
    if (lane == 0) rowStart[0] = tileStart[0] = 0;
    __syncwarp();
    // Fewer than three rounds of tiles: the cap whose rounds take the least time.  (A
    // slice takes about 0.13 us for the weight's copies and 0.0007 us a column; by the
    // mean width.)
    int cap = BN;
    if constexpr (kCaps > 1) {
      const float workers = (float)((int)gridDim.x / kCtas);
      float best = 0.0f;
#pragma unroll
      for (int i = 0; i < kCaps; ++i) {
        const float across = (float)__reduce_add_sync(0xffffffffu, sums[i]);
        const float rounds = ceilf(across * (float)rowsM / workers);
        const float time = rounds * (0.13f + 0.0007f * (float)rows / fmaxf(across, 1.0f));
        if (i == 0 || time < best) best = time, cap = cap_of(i);
        if (i == 0 && rounds >= 3.0f) break;
      }
    }
    int tiles = 0;
    for (int e0 = 0; kRowsToo && e0 < g.groups; e0 += 32) {
      const int e = e0 + lane;
      int sum = 0;
      if (e < g.groups) sum = (rowStart[e + 1] - rowStart[e] + cap - 1) / cap * rowsM;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      if (e < g.groups) tileStart[e + 1] = tiles + sum;
      tiles += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) chosenCap = cap;
  }
  tmem_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the peer's barriers are set up
  tmem_fence_after();
  const uint32_t tmem = tmemBase;
  const int tiles = weightTiles + (kRowsToo ? tileStart[g.groups] : 0), cap = chosenCap;
  const int firstTile = (int)blockIdx.x / kCtas, tileStep = (int)gridDim.x / kCtas;
  // Tiles are walked upwards: `e` is the group of the last one of rows.
  auto tile_at = [&](int t, int& e) {
    constexpr int kHigh = 2048 / kRows, G = Shape::kGrain;
    const bool weight = kWeight && (!kRowsToo || t < weightTiles);
    int of, high;
    if (weight) {
      of = quotient(t, weightM * weightN);
      t -= of * weightM * weightN;
      high = weightM;
    } else {
      t -= weightTiles;
      while (t >= tileStart[e + 1]) ++e;
      t -= tileStart[e];
      of = e;
      high = rowsM;
    }
    GroupTile o = {of, 0, 0, BN, rowStart[of], rowStart[of + 1], weight};
    // the tiles of a block of 2048 rows of the product column by column, so that
    // the operands of the tiles in flight stay in L2
    const int n = o.hi - o.lo, across = weight ? weightN : quotient(n + cap - 1, cap);
    const int block = quotient(t, kHigh * across);
    high = min(kHigh, high - block * kHigh);
    t -= block * kHigh * across;
    const int column = quotient(t, high);
    o.m0 = (block * kHigh + t - column * high) * kRows;
    if (weight) {
      o.n0 = column * BN;
    } else {  // columns in shares of about one size, none of them empty
      const int share = quotient((n + G - 1) / G + across - 1, across) * G, from = column * share;
      o.n0 = o.lo + from;
      o.width = min(share, (n - from + G - 1) / G * G);
    }
    return o;
  };
  // (known where a kind has tiles of one sort only)
  auto of_weight = [](const GroupTile& o) { return kWeight && (!kRowsToo || o.weight); };
  auto slices_of = [&](const GroupTile& o) {
    return ((of_weight(o) ? o.hi - o.lo : g.rows.K) + kTileK - 1) / kTileK;
  };

  if (warp == 0) {
    int s = 0, turn = 0, e = 0;
    unsigned tailTurn = 0, tailed = 0;  // a bit for each stage
    bool ok = true;
    long long issued = 0;
    const uint32_t landed0 = PAIR ? peer_addr(full(0), 0) : full(0);
    for (int t = firstTile; ok && t < tiles; t += tileStep) {
      const GroupTile o = tile_at(t, e);
      const int slices = slices_of(o);
      const bool weight = of_weight(o);
      const int mine = PAIR ? o.width / 2 : o.width;  // columns that this CTA holds
      const int m0 = o.m0 + (int)rank * kTileM, n0 = o.n0 + (int)rank * mine;
      const int boxes = (mine + Shape::kBox - 1) / Shape::kBox;
      const unsigned bytes =
          Shape::kABytes + (weight ? Shape::kBBytes : boxes * (Shape::kBox * 128));
      for (int kb = 0; kb < slices; ++kb) {
        ok = all_wait(empty(s), turn ^ 1);
        if (!ok) break;
        const bool tail = kTails && weight && o.hi - o.lo < (kb + 1) * kTileK;
        if (elected()) {
          uint32_t landed = landed0 + 8u * s;
          if (tail) {
            mbar_arrive_expect_tx(tailFull(s), bytes);
            landed = peer_addr(tailFull(s), rank);
          } else if (leader) {
            mbar_arrive_expect_tx(full(s), kCtas * bytes);
          }
          const uint32_t a = stage0 + (unsigned)s * Shape::kStageBytes, b = a + Shape::kABytes;
          const int k0 = kb * kTileK;
          if (weight) {
#pragma unroll
            for (int i = 0; i < kTileM / 64; ++i)
              tensor_load<PAIR>(a + i * kSlab, &g.weight.a, m0 + i * 64, o.lo + k0, 0, landed);
#pragma unroll
            for (int i = 0; i < Shape::kBRows / 64; ++i)
              tensor_load<PAIR>(b + i * kSlab, &g.weight.b, n0 + i * 64, o.lo + k0, 0, landed);
          } else {
            if constexpr (kTurned) {
#pragma unroll
              for (int i = 0; i < kTileM / 64; ++i)
                tensor_load<PAIR>(a + i * kSlab, &g.rows.a, m0 + i * 64, k0, o.g, landed);
            } else {
              tensor_load<PAIR>(a, &g.rows.a, k0, m0, o.g, landed);
            }
            for (int i = 0; i < boxes; ++i)
              tensor_load<PAIR>(b + i * (Shape::kBox * 128), &g.rows.b, k0, n0 + i * Shape::kBox, 0,
                                landed);
          }
        }
        __syncwarp();
        if (tail) tailTurn ^= 1u << s, tailed |= 1u << s;
        else tailed &= ~(1u << s);
        ++issued;
        if (++s == kStages) s = 0, turn ^= 1;
      }
    }
    // as in gemm_kernel: no arrival of the other CTA's products after this one
    // has left, no copy into memory that is no longer its own
    for (long long i = issued > kStages ? issued - kStages : 0; ok && i < issued; ++i)
      ok = all_wait(empty((int)(i % kStages)), (unsigned)(i / kStages & 1));
    if (!ok) {
      raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
      for (long long i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
        const int at = (int)(i % kStages);
        if (tailed >> at & 1) wait(tailFull(at), (tailTurn >> at & 1) ^ 1, false);
        else if (leader) wait(full(at), (unsigned)(i / kStages & 1), false);
      }
    }
  } else if (warp == 1 && leader) {
    // MN-major operands: slabs of 64 columns, 16 rows of 128 bytes to a product;
    // K-major ones: 32 bytes along a row
    const uint64_t aMn = operand_desc(stage0, kSlab, 1024), aK = operand_desc(stage0, 16, 1024);
    const uint64_t bMn = operand_desc(stage0 + Shape::kABytes, kSlab, 1024);
    const uint64_t bK = operand_desc(stage0 + Shape::kABytes, 16, 1024);
    constexpr unsigned kStepMn = 16 * 128 >> 4, kStepK = 32 >> 4;
    int s = 0, turn = 0, buf = 0, bufTurn = 0, e = 0;
    bool ok = true;
    for (int t = firstTile; ok && t < tiles; t += tileStep) {
      const GroupTile o = tile_at(t, e);
      const int slices = slices_of(o), chunk = CHUNK ? CHUNK : max(slices, 1);
      const bool weight = of_weight(o);
      const uint32_t idesc = (weight ? mma_idesc<T>(kRows, 0, true, true)
                                     : mma_idesc<T>(kRows, 0, kTurned, false)) |
                             (uint32_t)(o.width >> 3) << 17;
      const uint64_t aDesc0 = weight || kTurned ? aMn : aK, bDesc0 = weight ? bMn : bK;
      const unsigned aStep = weight || kTurned ? kStepMn : kStepK;
      const unsigned bStep = weight ? kStepMn : kStepK;
      for (int c0 = 0; ok && c0 < slices; c0 += chunk) {
        ok = all_wait(accEmpty(buf), bufTurn ^ 1);
        if (!ok) break;
        tmem_fence_after();
        const uint32_t acc = tmem + (unsigned)(buf * BN);
        const int c1 = min(c0 + chunk, slices);
        for (int kb = c0; kb < c1; ++kb) {
          ok = all_wait(full(s), turn);
          if (!ok) break;
          int steps = kTileK / 16;
          if (weight) {
            const int left = o.hi - o.lo - kb * kTileK;  // rows of the group in this slice
            if (left < kTileK) {
              steps = (left + 15) / 16;
              if (!kTails)
                zero_rows<Shape::kStageBytes / (int)kSlab>(
                    stage0 + (unsigned)s * Shape::kStageBytes, left, steps * 16, lane);
            }
          }
          tmem_fence_after();
          if (elected()) {
            const uint64_t at = (uint64_t)((unsigned)s * (Shape::kStageBytes >> 4));
#pragma unroll
            for (int k = 0; k < kTileK / 16; ++k)
              if (!kWeight || k < steps)
                mma_f16<PAIR>(acc, aDesc0 + at + k * aStep, bDesc0 + at + k * bStep, idesc,
                              (kb - c0) | k);
            mma_commit<PAIR>(empty(s), pairMask);
            if (kb + 1 == c1) mma_commit<PAIR>(accFull(buf), pairMask);
          }
          __syncwarp();
          if (++s == kStages) s = 0, turn ^= 1;
        }
        if (!ok) break;
        if (++buf == 2) buf = 0, bufTurn ^= 1;
      }
    }
    if (!ok) {
      raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
      if (elected()) {
        mma_commit<PAIR>(drained, pairMask);
        wait(drained, 0, false);
      }
    }
  } else if (kTails && warp == 3) {
    // The ends of the groups on a pair: each CTA zeroes its rows behind the end
    // once its copies have landed, the first one hands the stage on when both
    // have.
    int e = 0;
    long long done = 0;  // slices before the tile
    unsigned tailTurn = 0;
    bool ok = true;
    for (int t = firstTile; ok && t < tiles; t += tileStep) {
      const GroupTile o = tile_at(t, e);
      const int slices = slices_of(o), left = (o.hi - o.lo) % kTileK;
      done += slices;
      if (!of_weight(o) || !left) continue;
      const int s = (int)((done - 1) % kStages);
      const unsigned parity = tailTurn >> s & 1;
      tailTurn ^= 1u << s;
      // (the whole tile before it: one limit for each 65536 slices)
      for (int i = 0; !(ok = all_wait(tailFull(s), parity)) && i < slices >> 16 && !abortFlag; ++i) {
      }
      if (!ok) break;
      zero_rows<Shape::kStageBytes / (int)kSlab>(stage0 + (unsigned)s * Shape::kStageBytes, left,
                                                 (left + 15) / 16 * 16, lane);
      if (leader) {
        ok = all_wait(tailPeer(s), parity);
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        if (ok && lane == 0) mbar_arrive(full(s));
      } else if (lane == 0) {
        peer_arrive_release(peer_addr(tailPeer(s), 0));
      }
      __syncwarp();
    }
    if (!ok) raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
  } else if (warp >= 4) {
    const int quad = warp % 4, part = (warp - 4) / 4;
    const uint32_t quadBase = tmem + ((uint32_t)(quad * 32) << 16);
    int buf = 0, bufTurn = 0, e = 0;
    auto next = [&]() {
      if (!all_wait(accFull(buf), bufTurn)) {
        raise_error(g.status, &abortFlag, VR_ERR_TIMEOUT);
        return false;
      }
      tmem_fence_after();
      return true;
    };
    auto release = [&]() {
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) peer_arrive(peer_addr(accEmpty(buf), 0));
        else mbar_arrive(accEmpty(buf));
      }
      if (++buf == 2) buf = 0, bufTurn ^= 1;
    };
    const uint32_t staged = stage0 + (unsigned)(kStages * Shape::kStageBytes +
                                                (warp - 4) * (kWeight ? kStaged : kStaged / 2));
    const int m = (int)rank * kTileM + quad * 32;  // the warp's first row of a tile
    // 32 columns from c of a tile of dW
    auto store_weight = [&](const GroupTile& o, int c, const float(&v)[32]) {
      const Product& p = g.weight;
      const int first = o.m0 + m, n = o.n0 + c;
      staged_free();
      stage_rows<T>(staged, v);
      if (first >= p.M) return;
      if (p.align >= 16)
        store_staged(staged, &p.c, n, first, o.g);
      else
        store_staged(staged, static_cast<T*>(p.out) + ((long long)o.g * p.M + first) * p.ld + n,
                     p.ld, p.M - first, p.N - n);
    };
    // and of one of rows: the first row's place
    auto row_of = [&](const GroupTile& o, int c) {
      return static_cast<T*>(g.rows.out) + (o.n0 + c) * g.rows.ld;
    };
    // rows that the tile has from its column c on
    auto rows_of = [&](const GroupTile& o, int c) { return min(o.hi - o.n0, o.width) - c; };
    // whether the 32 columns from c are in the product
    auto there = [&](const GroupTile& o, int c) {
      return of_weight(o) ? o.n0 + c < g.weight.N : rows_of(o, c) > 0;
    };
    for (int t = firstTile; t < tiles; t += tileStep) {
      const GroupTile o = tile_at(t, e);
      const int slices = slices_of(o);
      if constexpr (CHUNK > 0) {
        float sum[kUnits * 32];
#pragma unroll
        for (int i = 0; i < kUnits * 32; ++i) sum[i] = 0.0f;
        bool left = false;
        for (int c0 = 0; c0 < slices; c0 += CHUNK) {
          left = !next();
          if (left) break;
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            const int c = (part + i * kGroups) * 32;
            if (!there(o, c)) break;
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              float v[16];
              tmem_load16(quadBase + (unsigned)(buf * BN + c + h), v);
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[i * 32 + h + j] += v[j];
            }
          }
          release();
        }
        if (left) break;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          const int c = (part + i * kGroups) * 32;
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = sum[i * 32 + j];
          if (!there(o, c)) break;
          if constexpr (kWeight)
            store_weight(o, c, v);
          else
            store_columns(row_of(o, c), g.rows.ld, v, rows_of(o, c), o.m0 + m + lane, g.rows.M,
                          g.rows.align);
        }
      } else {
        if (slices && !next()) break;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          const int c = (part + i * kGroups) * 32;
          if (!there(o, c)) break;
          __syncwarp();
          if (of_weight(o)) {
            float v[32];
            if (slices) {
              tmem_load32(quadBase + (unsigned)(buf * BN + c), v);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.0f;
            }
            store_weight(o, c, v);
          } else {
            if (kWeight) staged_free();
            store_turned(quadBase + (unsigned)(buf * BN + c), staged, row_of(o, c) + o.m0 + m,
                         g.rows.ld, rows_of(o, c), g.rows.M - o.m0 - m, g.rows.align);
          }
        }
        if (slices) release();
      }
    }
    if (kWeight && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
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

// ------------------------------------------------------------- host side
constexpr size_t kMostRows = (size_t)1 << 30, kMostDim = (size_t)1 << 24,
                 kMostStride = (size_t)1 << 31;

// A matrix of 16-bit elements as it is given, or its copy in whole sectors.
struct Matrix {
  const void* p;
  size_t rows, cols, stride;  // batch * rows of them
  size_t batch;
  size_t copy;                // place of the copy in the workspace, where it needs one
  bool pad;
};
struct GroupedPlan {
  Matrix x, w, dy;
  size_t bytes;
};

void plan_matrix(const void* p, size_t rows, size_t cols, size_t stride, size_t batch, Matrix* m,
                 size_t* at) {
  *m = {p, rows, cols, stride, batch, 0, !packed_rows(p, stride)};
  if (m->pad) {
    m->copy = *at;
    *at += op_round(batch * rows * up(cols, 16) * 2);
  }
}

bool sizes_ok(size_t rows, size_t dim, size_t outDim, int groups, int dtype) {
  return (dtype == VR_FLOAT16 || dtype == VR_BFLOAT16) && rows <= kMostRows && dim >= 1 &&
         dim <= kMostDim && outDim >= 1 && outDim <= kMostDim && groups >= 1 &&
         groups <= kMostGroups;
}
bool stride_ok(size_t stride, size_t cols) { return stride >= cols && stride <= kMostStride; }

bool plan_linear(const void* x, size_t xStride, const void* w, size_t rows, size_t dim,
                 size_t outDim, int groups, int dtype, GroupedPlan* p) {
  if (!sizes_ok(rows, dim, outDim, groups, dtype) || !stride_ok(xStride, dim)) return false;
  size_t at = 0;
  *p = GroupedPlan{};
  plan_matrix(x, rows, dim, xStride, 1, &p->x, &at);
  plan_matrix(w, outDim, dim, dim, (size_t)groups, &p->w, &at);
  p->bytes = at + kOpSlack;
  return true;
}
bool plan_grad(const void* dy, size_t dyStride, const void* x, size_t xStride, const void* w,
               size_t rows, size_t dim, size_t outDim, int groups, int dtype, GroupedPlan* p) {
  if (!sizes_ok(rows, dim, outDim, groups, dtype) || !stride_ok(xStride, dim) ||
      !stride_ok(dyStride, outDim))
    return false;
  size_t at = 0;
  *p = GroupedPlan{};
  plan_matrix(dy, rows, outDim, dyStride, 1, &p->dy, &at);
  plan_matrix(x, rows, dim, xStride, 1, &p->x, &at);
  plan_matrix(w, outDim, dim, dim, (size_t)groups, &p->w, &at);
  p->bytes = at + kOpSlack;
  return true;
}

// `counts`: of the groups whose matrices m holds; the others are not read.
vr_result_t pad_matrix(Matrix* m, char* w, const OpDevice& dev, void* stream,
                       const int* counts = nullptr) {
  if (!m->pad || !m->rows) return VR_SUCCESS;
  const size_t ld = up(m->cols, 16), rows = m->batch * m->rows;
  PadArgs a = {static_cast<const uint16_t*>(m->p), (long long)m->stride, (long long)rows,
               (int)m->cols, (int)ld, reinterpret_cast<uint16_t*>(w + m->copy), counts,
               (long long)m->rows};
  void* args[] = {&a};
  m->p = w + m->copy;
  m->stride = ld;
  return op_launch((const void*)pad_kernel,
                   dim3((unsigned)std::min<size_t>((rows + 7) / 8, (size_t)dev.sms * 32)),
                   dim3(256), args, 0, stream);
}

// What a call multiplies: K summed; rows and dW's sums are counted on the device.
struct GroupedSize {
  size_t M, N, K, rows;
  int groups;
};

// The operands of a product and where its result goes.
vr_result_t fill(Product* p, bool bf16, const Matrix& a, int aBox, const Matrix& b, int bBox,
                 const GroupedSize& z, void* out, size_t ld, bool weight) {
  auto map = [&](CUtensorMap* to, const Matrix& m, int boxRows) {
    return gemm_operand(to, m.p, bf16, m.cols, m.rows, m.batch, m.stride * 2,
                        m.stride * 2 * m.rows, boxRows);
  };
  vr_result_t e = map(&p->a, a, aBox);
  if (e != VR_SUCCESS || (e = map(&p->b, b, bBox)) != VR_SUCCESS) return e;
  p->M = (int)z.M;
  p->N = (int)z.N;
  p->K = (int)z.K;
  p->out = out;
  p->ld = (long long)ld;
  const uintptr_t bits = (uintptr_t)out | (uintptr_t)(2 * ld);
  p->align = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
  if (!weight || p->align < 16) return VR_SUCCESS;
  return gemm_operand(&p->c, out, bf16, z.N, z.M, (size_t)z.groups, ld * 2, ld * 2 * z.M, 32,
                      kAuxCols);
}
template <int BN, bool PAIR, int KIND>
vr_result_t fill_rows(GroupedArgs* g, bool bf16, const Matrix& w, const Matrix& x,
                      const GroupedSize& z, void* out, size_t ld) {
  return fill(&g->rows, bf16, w, KIND == kLinear ? kTileM : kTileK, x,
              GroupedShape<BN, PAIR, false>::kBox, z, out, ld, false);
}
vr_result_t fill_weight(GroupedArgs* g, bool bf16, const Matrix& dy, const Matrix& x,
                        const GroupedSize& z, void* out, size_t ld) {
  return fill(&g->weight, bf16, dy, kTileK, x, kTileK, z, out, ld, true);
}

template <typename T, int BN, int KIND, bool PAIR, int CHUNK>
vr_result_t launch(const OpDevice& dev, GroupedArgs& g, size_t rows, int groups, const int* counts,
                   void* stream) {
  using Shape = GroupedShape<BN, PAIR, (KIND >= kGradWeight)>;
  const void* fn = (const void*)grouped_kernel<T, BN, KIND, PAIR, CHUNK>;
  const vr_result_t e = gemm_prepare(fn, dev.device, Shape::kSmem);
  if (e != VR_SUCCESS) return e;
  g.counts = counts;
  g.groups = groups;
  g.most = (int)rows;
  g.status = dev.status;
  g.timeoutNs = dev.timeoutNs;
  // at most so many tiles: every group's last one may be cut; with the smallest cap
  constexpr size_t kCap = BN < 128 ? BN : 64;
  auto along = [](int n, int tile) { return (size_t)((n + tile - 1) / tile); };
  size_t tiles = 0;
  if (KIND != kGradWeight)
    tiles += (rows / kCap + std::min<size_t>((size_t)groups, rows)) *
             along(g.rows.M, Shape::kTileRows);
  if (KIND >= kGradWeight)
    tiles += (size_t)groups * along(g.weight.M, Shape::kTileRows) * along(g.weight.N, BN);
  constexpr size_t kCtas = PAIR ? 2 : 1;
  const size_t grid = std::min<size_t>(tiles, dev.sms / kCtas) * kCtas;
  void* args[] = {&g};
  return op_launch(fn, dim3((unsigned)grid), dim3(128 + 32 * Shape::kWarps), args, Shape::kSmem,
                   stream, (int)kCtas);
}

// Sums longer than these are taken in chunks of 2048: the tensor cores truncate
// where a product is added, 1.6e-8 of the sum per 16 k (xent.cu).  So the longest sum
// of one piece is off by about 3.3e-5 (fp16) or 2.6e-4 (bf16) of the running sum, a
// fifteenth of the result's rounding.  For dW the host knows the rows of all groups together
// only: fp16 in a buffer of 32769 rows, 12 groups, instead of 32768 takes 91 us
// instead of 79 for dW of 1024 x 1536, both gradients 143.5 instead of 143, those of
// 512 x 512, which share a launch otherwise, 57 instead of 48.
constexpr int kLongChunk = 32;
template <typename T>
constexpr size_t kLongSum = std::is_same<T, __half>::value ? 32768 : 262144;

// A group on average: the counts are not known here.  Tiles of 32 / of up to 256
// columns, 64 groups of 2048 x 4096 in bf16 (us):
//   every group has 8, 16, 24, 32 rows      183/183, 184/185, 187/185, 189/185
//   8 groups have 8, 32, 64, 120, 240 rows  38/40, 38/42, 42/42, 54/42, 91/46
//   16 groups have 8, 32, 64, 120 rows      62/66, 63/66, 64/66, 95/68
// Few columns are quicker where few groups have few rows each, a step that decodes
// some tokens, and cost up to twice the time where few have many.
constexpr size_t kFewRows = 32;
constexpr size_t kBothMost = 4;  // tiles for each SM: eight rounds of pairs

bool few_rows(size_t rows, int groups) { return rows <= kFewRows * (size_t)groups; }

// out or dX: w's rows by a group's rows.
template <typename T, int KIND>
vr_result_t rows_product(const OpDevice& dev, const Matrix& w, const Matrix& x,
                         const GroupedSize& z, const int* counts, void* out, size_t ld,
                         void* stream) {
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  GroupedArgs g = {};
  auto go = [&](auto bn, auto pair) {
    constexpr int BN = decltype(bn)::value;
    constexpr bool PAIR = decltype(pair)::value;
    const vr_result_t e = fill_rows<BN, PAIR, KIND>(&g, bf16, w, x, z, out, ld);
    if (e != VR_SUCCESS) return e;
    if (z.K > kLongSum<T>)
      return launch<T, BN, KIND, PAIR, kLongChunk>(dev, g, z.rows, z.groups, counts, stream);
    return launch<T, BN, KIND, PAIR, 0>(dev, g, z.rows, z.groups, counts, stream);
  };
  using std::integral_constant;
  if (few_rows(z.rows, z.groups)) return go(integral_constant<int, 32>(), std::false_type());
  if (z.M <= kTileM) return go(integral_constant<int, 256>(), std::false_type());
  return go(integral_constant<int, 256>(), std::true_type());
}
template <typename T>
vr_result_t linear(const GroupedPlan& p, const OpDevice& dev, size_t rows, size_t dim,
                   size_t outDim, int groups, const int* counts, void* out, size_t ld,
                   void* stream) {
  return rows_product<T, kLinear>(dev, p.w, p.x, {outDim, rows, dim, rows, groups}, counts, out,
                                  ld, stream);
}
template <typename T>
vr_result_t weight_product(const OpDevice& dev, const Matrix& dy, const Matrix& x,
                           const GroupedSize& z, const int* counts, void* out, void* stream) {
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  GroupedArgs g = {};
  const vr_result_t e = fill_weight(&g, bf16, dy, x, z, out, z.N);
  if (e != VR_SUCCESS) return e;
#define VR_GO(PAIR, CHUNK) \
  launch<T, 256, kGradWeight, PAIR, CHUNK>(dev, g, z.rows, z.groups, counts, stream)
  if (z.K > kLongSum<T>) return z.M <= kTileM ? VR_GO(false, kLongChunk) : VR_GO(true, kLongChunk);
  return z.M <= kTileM ? VR_GO(false, 0) : VR_GO(true, 0);
#undef VR_GO
}
template <typename T>
vr_result_t grad(const GroupedPlan& p, const OpDevice& dev, size_t rows, size_t dim, size_t outDim,
                 int groups, const int* counts, void* dx, void* dw, void* stream) {
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const GroupedSize zx = {dim, rows, outDim, rows, groups}, zw = {outDim, dim, rows, rows, groups};
  vr_result_t e = VR_SUCCESS;
  // One launch where both take pairs and sums of one piece, and few tiles.  It saves
  // the second one's start and a round that is not full (12 groups of 250 rows, 1000 x
  // 1512: 37 us instead of 46); with many tiles the epilogues of dW beside dX's
  // cost more (64 groups of 128 rows, 2048 x 4096: 450 us instead of 438; 32 of 2048
  // rows 1302 instead of 1285).
  const size_t tiles = (rows / 256 + std::min<size_t>((size_t)groups, rows)) * (up(dim, 256) / 256) +
                       (size_t)groups * (up(dim, 256) / 256) * (up(outDim, 256) / 256);
  if (dx && dw && !few_rows(rows, groups) && dim > kTileM && outDim > kTileM &&
      rows <= kLongSum<T> && outDim <= kLongSum<T> && tiles <= kBothMost * (size_t)dev.sms) {
    GroupedArgs g = {};
    if ((e = fill_rows<256, true, kGradRows>(&g, bf16, p.w, p.dy, zx, dx, dim)) != VR_SUCCESS ||
        (e = fill_weight(&g, bf16, p.dy, p.x, zw, dw, dim)) != VR_SUCCESS)
      return e;
    return launch<T, 256, kGradBoth, true, 0>(dev, g, rows, groups, counts, stream);
  }
  if (dx && (e = rows_product<T, kGradRows>(dev, p.w, p.dy, zx, counts, dx, dim, stream)) !=
                VR_SUCCESS)
    return e;
  return dw ? weight_product<T>(dev, p.dy, p.x, zw, counts, dw, stream) : VR_SUCCESS;
}

}  // namespace
}  // namespace vr

using namespace vr;

extern "C" {

vr_result_t vr_grouped_linear_workspace_bytes(const void* x, size_t xStride, const void* weight,
                                              size_t rows, size_t dim, size_t outDim, int groups,
                                              vr_dtype_t dtype, size_t* bytes) {
  GroupedPlan p;
  if (!bytes || !plan_linear(x, xStride, weight, rows, dim, outDim, groups, dtype, &p))
    return VR_ERR_INVALID_ARGUMENT;
  *bytes = p.bytes;
  return VR_SUCCESS;
}

vr_result_t vr_grouped_linear(const void* x, size_t xStride, const void* weight, const int* counts,
                              size_t rows, size_t dim, size_t outDim, int groups, vr_dtype_t dtype,
                              void* out, size_t outStride, void* workspace, size_t workspaceBytes,
                              void* stream) {
  GroupedPlan p;
  if (!plan_linear(x, xStride, weight, rows, dim, outDim, groups, dtype, &p) ||
      !stride_ok(outStride, outDim) || !weight || !counts || !workspace ||
      (rows && (!x || !out)) || ((uintptr_t)workspace & 15) || workspaceBytes < p.bytes ||
      ((uintptr_t)counts & 3) || (((uintptr_t)x | (uintptr_t)weight | (uintptr_t)out) & 1))
    return VR_ERR_INVALID_ARGUMENT;
  const size_t nw = (size_t)groups * outDim * dim * 2;
  // (an output listed before the inputs may be none of them)
  const OpBuffer buf[5] = {{workspace, 1, workspaceBytes, workspaceBytes, true},
                           {out, rows, outDim * 2, outStride * 2, true},
                           {x, rows, dim * 2, xStride * 2, false},
                           {weight, 1, nw, nw, false},
                           {counts, 1, (size_t)groups * 4, (size_t)groups * 4, false}};
  if (!op_buffers_ok(buf, 5)) return VR_ERR_INVALID_ARGUMENT;
  OpDevice dev;
  vr_result_t e = op_device(&dev);
  if (e != VR_SUCCESS || (e = op_reachable(buf, 5, dev.device)) != VR_SUCCESS) return e;
  if (!rows) return VR_SUCCESS;
  char* w = op_workspace(workspace);
  if ((e = pad_matrix(&p.x, w, dev, stream)) != VR_SUCCESS ||
      (e = pad_matrix(&p.w, w, dev, stream, counts)) != VR_SUCCESS)
    return e;
  return dtype == VR_BFLOAT16 ? linear<__nv_bfloat16>(p, dev, rows, dim, outDim, groups, counts,
                                                      out, outStride, stream)
                              : linear<__half>(p, dev, rows, dim, outDim, groups, counts, out,
                                               outStride, stream);
}

vr_result_t vr_grouped_linear_grad_workspace_bytes(const void* dOut, size_t dOutStride,
                                                   const void* x, size_t xStride,
                                                   const void* weight, size_t rows, size_t dim,
                                                   size_t outDim, int groups, vr_dtype_t dtype,
                                                   size_t* bytes) {
  GroupedPlan p;
  if (!bytes ||
      !plan_grad(dOut, dOutStride, x, xStride, weight, rows, dim, outDim, groups, dtype, &p))
    return VR_ERR_INVALID_ARGUMENT;
  *bytes = p.bytes;
  return VR_SUCCESS;
}

vr_result_t vr_grouped_linear_grad(const void* dOut, size_t dOutStride, const void* x,
                                   size_t xStride, const void* weight, const int* counts,
                                   size_t rows, size_t dim, size_t outDim, int groups,
                                   vr_dtype_t dtype, void* dX, void* dWeight, void* workspace,
                                   size_t workspaceBytes, void* stream) {
  GroupedPlan p;
  if (!plan_grad(dOut, dOutStride, x, xStride, weight, rows, dim, outDim, groups, dtype, &p) ||
      !counts || !workspace || (!dX && !dWeight) || (dX && !weight) ||
      (rows && (!dOut || (dWeight && !x))) || ((uintptr_t)workspace & 15) ||
      workspaceBytes < p.bytes || ((uintptr_t)counts & 3) ||
      (((uintptr_t)dOut | (uintptr_t)x | (uintptr_t)weight | (uintptr_t)dX | (uintptr_t)dWeight) &
       1))
    return VR_ERR_INVALID_ARGUMENT;
  const size_t nw = (size_t)groups * outDim * dim * 2, nx = rows * dim * 2;
  OpBuffer buf[7] = {{workspace, 1, workspaceBytes, workspaceBytes, true}};
  int n = 1;
  if (dX) buf[n++] = {dX, 1, nx, nx, true};
  if (dWeight) buf[n++] = {dWeight, 1, nw, nw, true};
  buf[n++] = {dOut, rows, outDim * 2, dOutStride * 2, false};
  if (dWeight) buf[n++] = {x, rows, dim * 2, xStride * 2, false};
  if (dX) buf[n++] = {weight, 1, nw, nw, false};
  buf[n++] = {counts, 1, (size_t)groups * 4, (size_t)groups * 4, false};
  if (!op_buffers_ok(buf, n)) return VR_ERR_INVALID_ARGUMENT;
  OpDevice dev;
  vr_result_t e = op_device(&dev);
  if (e != VR_SUCCESS || (e = op_reachable(buf, n, dev.device)) != VR_SUCCESS) return e;
  if (!rows) {
    if (dWeight && cudaMemsetAsync(dWeight, 0, nw, (cudaStream_t)stream) != cudaSuccess)
      return VR_ERR_CUDA;
    return VR_SUCCESS;
  }
  char* w = op_workspace(workspace);
  if ((e = pad_matrix(&p.dy, w, dev, stream)) != VR_SUCCESS ||
      (dWeight && (e = pad_matrix(&p.x, w, dev, stream)) != VR_SUCCESS) ||
      (dX && (e = pad_matrix(&p.w, w, dev, stream, counts)) != VR_SUCCESS))
    return e;
  return dtype == VR_BFLOAT16
             ? grad<__nv_bfloat16>(p, dev, rows, dim, outDim, groups, counts, dX, dWeight, stream)
             : grad<__half>(p, dev, rows, dim, outDim, groups, counts, dX, dWeight, stream);
}

}  // extern "C"
