// Newton-Schulz orthogonalisation of matrices of one shape (vr_orthogonalize).
//
//   X = M / (|M|_F + eps)          (transposed when M has more rows than columns)
//   steps times:  A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// Every step is three products on the tensor cores (gemm.cuh), with the
// polynomial's sums in their epilogues.  A and B are symmetric: only the
// 128-blocks on and below the diagonal are computed, the others are stored
// as their mirror images.
//
// Operands are fp16 planes of the values times 2^12 (the entries of X, A and
// B stay below 16, which the entry point checks, and typical ones, of size
// 1 / sqrt(m n) to 1, stay in fp16's normal range).  X itself is kept as a
// high and a low plane, 22 bits: a rounding of X would be amplified by a with
// every later step in the directions of small singular values, where a
// rounding of an operand of B X is not (it enters between a small and a large
// direction, which the next steps damp).  So bf16 results take one product of
// high planes, fp16 and fp32 results three products of both planes, summed in
// chunks.  The operands' roundings of 2^-12, a few per step, average out over
// many directions: 1.2e-3 before the result's own rounding (1.7e-3) at 128 x
// 1024, 3.4e-3 at most over 200 matrices of 32 x 500, but up to 1.6e-2 at 2 x 3.
// Up to 16 rows (of X) bf16 results take both planes, too (8 matrices of 16 x
// 128: 25 -> 38 us; as exact as fp32's).
// (Holding X in fp32 beside the planes measured 4 % slower at 4096 x 1024
// and no more exact, but where all but a few singular values are below 1e-3:
// 1.2e-5 against 1.5e-5, fp32 arithmetic throughout 2.2e-5.)
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "gemm.cuh"

namespace vr {
namespace {

constexpr int kMost = 64;          // matrices per launch
constexpr float kScale = 4096.0f;  // of the planes
constexpr int kNormCtas = 256;     // partial sums of squares per matrix, at most
constexpr int kSplitChunk = 2;     // slices of 64 summed before rounding (two planes)
constexpr size_t kFewRows = 16;    // of X: bf16 results take both planes, too

struct Planes {
  __half *hi, *lo;
};

// v as a high plane and what the rounding left.
__device__ __forceinline__ void split(float v, __half& hi, __half& lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn(v - __half2float(hi));
}

// 32 consecutive values of a row of a plane whose rows are whole groups of
// 32; 32 bytes an access, since a warp's rows are 32 lines apart.
__device__ __forceinline__ void store_plane(__half* out, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __half2 h = __floats2half2_rn(v[16 * i + 2 * j], v[16 * i + 2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + 16 * i),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                 "r"(w[7])
                 : "memory");
  }
}
__device__ __forceinline__ void add_plane(const __half* in, float by, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[8];
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(in + 16 * i)
                 : "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[16 * i + 2 * j] = fmaf(by, f.x, v[16 * i + 2 * j]);
      v[16 * i + 2 * j + 1] = fmaf(by, f.y, v[16 * i + 2 * j + 1]);
    }
  }
}
// The low plane of v: what its high plane's rounding left.
__device__ __forceinline__ void residue(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] -= __half2float(__float2half_rn(v[i]));
}

// What an epilogue of a step does with the sum of products v of an element:
//   v <- byAcc v + byFrom (from_hi + from_lo) [- diagonal]
// into the planes `to`: on tiles in shared memory (unit; aux.nIn and aux.nOut
// planes read and written), or row by row where k is shared out over a
// cluster (run).
struct PlaneArgs {
  Planes from, to;
  long long ld, size;         // elements of a row, of a matrix
  float byFrom, byAcc, diagonal;
};

// A thread's row of a tile.
__device__ __forceinline__ void add_tile(const AuxTile& tile, int plane, int row, float by,
                                         float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "r"(tile.piece(plane, row, i))
                 : "memory");
    const __half2* h = reinterpret_cast<const __half2*>(&q);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(h[j]);
      v[8 * i + 2 * j] = fmaf(by, f.x, v[8 * i + 2 * j]);
      v[8 * i + 2 * j + 1] = fmaf(by, f.y, v[8 * i + 2 * j + 1]);
    }
  }
}
__device__ __forceinline__ void store_tile(const AuxTile& tile, int plane, int row,
                                           const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 q;
    __half2* h = reinterpret_cast<__half2*>(&q);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile.piece(plane, row, i)),
                 "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w)
                 : "memory");
  }
}

// A = X X^T (no `from`) or B = b A + c A A - d I: the block and, below the
// diagonal, its mirror image.
// (Its planes are m x m: not worth the stages that Aux tiles take from the
// products, 22 against 26 us at 4 x 1024 x 4096.)
struct SymmetricEpilogue {
  static constexpr bool kAux = false;
  static constexpr int kWarps = 16;
  struct Args {
    PlaneArgs p;
    int nIn, nOut;  // planes read and written
  };
  static __device__ __forceinline__ void mirror(const Args& a, const GemmArgs& g, const Tile& o,
                                                __half* plane, int r, int n, const float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i)  // the lanes' rows are consecutive columns here
      if (n + i < g.N) plane[o.z * a.p.size + (n + i) * a.p.ld + r] = __float2half_rn(v[i]);
  }
  template <int COLS, class Acc>
  static __device__ __forceinline__ void run(const Args& a, const GemmArgs& g, const Tile& o,
                                             int row, int col0, int M, const Acc& acc) {
    const int r = o.m0 + row, blockR = o.m0 / kTileM, blockC = (o.n0 + col0) / kTileM;
    const bool live = r < M && blockC <= blockR;
    const long long base = o.z * a.p.size;
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      const int n = o.n0 + col0 + c;
      if (n >= g.N) break;
      float v[32];
      acc(col0 + c, v);
      if (!live) continue;
      const long long at = base + r * a.p.ld + n;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= a.p.byAcc;
      if (a.nIn) add_plane(a.p.from.hi + at, a.p.byFrom, v);
      if (a.nIn > 1) add_plane(a.p.from.lo + at, a.p.byFrom, v);
      if (blockC == blockR) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (n + i == r) v[i] -= a.p.diagonal;
      }
      store_plane(a.p.to.hi + at, v);
      if (blockC < blockR) mirror(a, g, o, a.p.to.hi, r, n, v);
      if (a.nOut > 1) {
        residue(v);
        store_plane(a.p.to.lo + at, v);
        if (blockC < blockR) mirror(a, g, o, a.p.to.lo, r, n, v);
      }
    }
  }
};

// X <- a X + B X into the other pair of planes, or, after the last step,
// into the result.
template <typename T>
struct ApplyEpilogue {
  static constexpr bool kAux = true;
  static constexpr int kWarps = 8;
  struct Args {
    AuxArgs aux;
    PlaneArgs p;
    int last, tall, vec;
    float byOut;
    int cols;         // of X
    T* out[kMost];
  };
  static __device__ __forceinline__ void finish(const Args& a, const GemmArgs& g, int z, int r,
                                                int n, int M, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= a.byOut;
    typename Ty<T>::Bits* out = reinterpret_cast<typename Ty<T>::Bits*>(a.out[z]);
    if (a.tall) {  // the lanes' rows are consecutive columns of the result
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (n + i < g.N) out[(long long)(n + i) * M + r] = Ty<T>::narrow(v[i]);
    } else if (a.vec && n + 32 <= g.N) {
      constexpr int U = Ty<T>::U;
      uint4* p = reinterpret_cast<uint4*>(out + (long long)r * a.cols + n);
#pragma unroll
      for (int i = 0; i < 32 / U; ++i) {
        uint4 q;
        typename Ty<T>::Bits* b = reinterpret_cast<typename Ty<T>::Bits*>(&q);
#pragma unroll
        for (int j = 0; j < U; ++j) b[j] = Ty<T>::narrow(v[i * U + j]);
        p[i] = q;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (n + i < g.N) out[(long long)r * a.cols + n + i] = Ty<T>::narrow(v[i]);
    }
  }
  static __device__ __forceinline__ bool skip(const GemmArgs& g, const Tile& o, int n, int M) {
    return n >= g.N || o.m0 >= M;
  }
  template <class Acc>
  static __device__ __forceinline__ void unit(const Args& a, const GemmArgs& g, const Tile& o,
                                              int row, int n, int c, int M, const Acc& acc,
                                              const AuxTile& tile) {
    const int r = o.m0 + row;
    float v[32];
    acc(c, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= a.p.byAcc;
    add_tile(tile, 0, row, a.p.byFrom, v);
    add_tile(tile, 1, row, a.p.byFrom, v);
    if (a.last) {
      if (r < M) finish(a, g, o.z, r, n, M, v);
    } else {
      store_tile(tile, 0, row, v);
      residue(v);
      store_tile(tile, 1, row, v);
    }
  }
  template <int COLS, class Acc>
  static __device__ __forceinline__ void run(const Args& a, const GemmArgs& g, const Tile& o,
                                             int row, int col0, int M, const Acc& acc) {
    const int r = o.m0 + row;
    const bool live = r < M;
    const long long base = o.z * a.p.size;
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      const int n = o.n0 + col0 + c;
      if (n >= g.N) break;
      float v[32];
      acc(col0 + c, v);
      if (!live) continue;
      const long long at = base + r * a.p.ld + n;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= a.p.byAcc;
      add_plane(a.p.from.hi + at, a.p.byFrom, v);
      add_plane(a.p.from.lo + at, a.p.byFrom, v);
      if (a.last) {
        finish(a, g, o.z, r, n, M, v);
      } else {
        store_plane(a.p.to.hi + at, v);
        residue(v);
        store_plane(a.p.to.lo + at, v);
      }
    }
  }
};

struct LoadArgs {
  const void* src[kMost];
  long long rows, cols;
  float* part;     // [matrix][kNormCtas]
  int ctas;        // partial sums per matrix
  float eps;
  int tall;
  Planes x;
  long long ld, size;
};

// Partial sums of squares, fp32: a run of elements per thread, then a tree.
template <typename T>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const __grid_constant__ LoadArgs a) {
  __shared__ float s[8];
  pdl_launch();
  pdl_wait();
  const typename Ty<T>::Bits* p = static_cast<const typename Ty<T>::Bits*>(a.src[blockIdx.y]);
  const long long n = a.rows * a.cols;
  constexpr int U = Ty<T>::U;
  float sum = 0.0f;
  const long long step = (long long)gridDim.x * 256;
  const long long first = (long long)blockIdx.x * 256 + threadIdx.x;
  if (((uintptr_t)p & 15) == 0) {
    const long long units = n / U;
    for (long long i = first; i < units; i += step) {
      const uint4 q = reinterpret_cast<const uint4*>(p)[i];
      const typename Ty<T>::Bits* b = reinterpret_cast<const typename Ty<T>::Bits*>(&q);
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float x = Ty<T>::widen(b[j]);
        t = fmaf(x, x, t);
      }
      sum += t;
    }
    for (long long i = units * U + first; i < n; i += step) {
      const float x = Ty<T>::widen(p[i]);
      sum = fmaf(x, x, sum);
    }
  } else {
    for (long long i = first; i < n; i += step) {
      const float x = Ty<T>::widen(p[i]);
      sum = fmaf(x, x, sum);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += s[w];
    a.part[blockIdx.y * kNormCtas + blockIdx.x] = sum;
  }
}

// The normalised matrix into the planes of X: eight elements a thread, or
// through shared memory, 64 x 32 blocks at a time, when it is transposed.
template <typename T>
__global__ void __launch_bounds__(256) ortho_load_kernel(const __grid_constant__ LoadArgs a) {
  using Bits = typename Ty<T>::Bits;
  __shared__ float tile[64][33];
  pdl_launch();
  pdl_wait();
  const int z = blockIdx.y;
  float sum = 0.0f;
  for (int i = 0; i < a.ctas; ++i) sum += a.part[z * kNormCtas + i];
  const float by = kScale / (sqrtf(sum) + a.eps);
  const Bits* p = static_cast<const Bits*>(a.src[z]);
  __half *hi = a.x.hi + z * a.size, *lo = a.x.lo + z * a.size;
  if (!a.tall) {
    const bool vec = a.cols % 8 == 0 && ((uintptr_t)p & 15) == 0;
    const long long perRow = (a.cols + 7) / 8, units = a.rows * perRow;
    for (long long u = (long long)blockIdx.x * 256 + threadIdx.x; u < units;
         u += (long long)gridDim.x * 256) {
      const long long r = u / perRow, c = u % perRow * 8;
      alignas(16) Bits in[8];
      if (vec) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(in) / 16; ++i)
          reinterpret_cast<uint4*>(in)[i] =
              reinterpret_cast<const uint4*>(p + r * a.cols + c)[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) in[i] = c + i < a.cols ? p[r * a.cols + c + i] : (Bits)0;
      }
      alignas(16) __half h[8], l[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) split(Ty<T>::widen(in[i]) * by, h[i], l[i]);
      // rows are padded to whole groups of 32
      *reinterpret_cast<uint4*>(hi + r * a.ld + c) = *reinterpret_cast<const uint4*>(h);
      *reinterpret_cast<uint4*>(lo + r * a.ld + c) = *reinterpret_cast<const uint4*>(l);
    }
    return;
  }
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const long long blocksC = (a.cols + 31) / 32, blocks = blocksC * ((a.rows + 63) / 64);
  for (long long b = blockIdx.x; b < blocks; b += gridDim.x) {
    const long long r0 = b / blocksC * 64, c0 = b % blocksC * 32;
#pragma unroll
    for (int i = 0; i < 64; i += 8) {
      const long long r = r0 + ty + i, c = c0 + tx;
      tile[ty + i][tx] = r < a.rows && c < a.cols ? Ty<T>::widen(p[r * a.cols + c]) * by : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      const long long r = c0 + ty + i, c = r0 + 2 * tx;  // of X
      if (r < a.cols && c < a.rows) {
        __half2 h, l;
        split(tile[2 * tx][ty + i], h.x, l.x);
        split(tile[2 * tx + 1][ty + i], h.y, l.y);
        *reinterpret_cast<__half2*>(hi + r * a.ld + c) = h;
        *reinterpret_cast<__half2*>(lo + r * a.ld + c) = l;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------- small matrices
// Up to 128 rows (of X) and 2048 columns: one launch, a cluster of up to eight
// CTAs per matrix, each holding its 256 columns of X in shared memory for all
// steps.  (A launch per product costs 5 to 7 us whatever its size, 17 of them
// 85 us at 8 x 128 x 128.)  A slab of 128 rows of 64 columns, 128 bytes a
// row, is the K-major operand of X X^T and the MN-major one of B X at once,
// so nothing is laid out twice.  In a cluster every CTA sums X X^T over its
// own columns; each adds up a share of A's columns from all of them in rank
// order and gives the planes of its share to all.
constexpr int kSmallRows = 128, kSmallCols = 256, kSmallCtas = 8;
constexpr int kSlab = kSmallRows * 128;                       // bytes of 64 columns
constexpr int kSmallX = kSmallCols / 64 * kSlab;              // a plane of X
constexpr int kSmallA = 2 * kSlab;                            // a plane of A or B
constexpr int kSmallSmem = 1024 + 2 * kSmallX + 2 * kSmallA;
static_assert(2 * kSmallA == kSmallRows * kSmallRows * 4, "partial sums of A use A's planes");

struct SmallArgs {
  const void* src[kMost];
  void* dst[kMost];
  int m, n, w;      // X: rows, columns, columns of a CTA (whole slabs)
  int tall, steps;
  float eps, byOut;
  float coefs[32][4];  // factor of X, b, c, what is subtracted from B's diagonal
  unsigned* status;
  unsigned long long timeoutNs;
};

__device__ __forceinline__ uint32_t slab_at(uint32_t plane, int r, int c) {
  return plane + (unsigned)((c >> 6) * kSlab + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) +
                            (c & 7) * 2);
}
__device__ __forceinline__ void shared_store16(uint32_t at, const __half (&h)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(h);
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(q.x), "r"(q.y), "r"(q.z),
               "r"(q.w)
               : "memory");
}
// 32 columns from c of row r of a plane: added to v, or written from it.
__device__ __forceinline__ void slab_add(uint32_t plane, int r, int c, float by, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "r"(slab_at(plane, r, c + 8 * i))
                 : "memory");
    const __half2* h = reinterpret_cast<const __half2*>(&q);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(h[j]);
      v[8 * i + 2 * j] = fmaf(by, f.x, v[8 * i + 2 * j]);
      v[8 * i + 2 * j + 1] = fmaf(by, f.y, v[8 * i + 2 * j + 1]);
    }
  }
}
__device__ __forceinline__ void slab_put(uint32_t plane, int r, int c, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    alignas(16) __half h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __float2half_rn(v[8 * i + j]);
    shared_store16(slab_at(plane, r, c + 8 * i), h);
  }
}

template <typename T, int PARTS>
__global__ void __launch_bounds__(256, 1) ortho_small_kernel(const __grid_constant__ SmallArgs a) {
  using Bits = typename Ty<T>::Bits;
  extern __shared__ unsigned char smemRaw[];
  __shared__ alignas(8) uint64_t bar;
  __shared__ uint32_t tmemBase;
  __shared__ float sSquares[9];  // of the warps, and their sum
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int shares = (int)cluster_size(), rank = (int)cluster_rank();
  const int z = (int)blockIdx.x / shares;
  const uint32_t base = (smem_addr(smemRaw) + 1023) & ~1023u;
  const uint32_t xHi = base, xLo = base + kSmallX, aHi = base + 2 * kSmallX, aLo = aHi + kSmallA;
  const uint32_t done = smem_addr(&bar);
  if (threadIdx.x == 0) {
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmemBase)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmemBase;
  pdl_launch();
  pdl_wait();

  // this CTA's columns [c0, c0 + width) of X
  const int c0 = rank * a.w, width = max(0, min(a.n - c0, a.w));
  const Bits* src = static_cast<const Bits*>(a.src[z]);
  // Pieces of eight consecutive elements of src: of a row of X, or, tall (X is
  // the transpose of src), of a column.
  const int length = a.tall ? a.m : a.n;  // of a row of src
  const int perRow = ((a.tall ? a.m : width) + 7) / 8;
  const int pieces = perRow * (a.tall ? width : a.m);
  const bool vec = length % 8 == 0 && ((uintptr_t)src & 15) == 0;
  auto load8 = [&](int i, float(&x)[8], int& line, int& at) {
    line = i / perRow;  // row of X, or its column from c0
    at = i % perRow * 8;
    const Bits* p = src + (a.tall ? (long long)(c0 + line) * length + at
                                  : (long long)line * length + c0 + at);
    const int left = (a.tall ? a.m : width) - at;
    if (vec && left >= 8) {
      alignas(16) Bits in[8];
#pragma unroll
      for (int j = 0; j < (int)sizeof(in) / 16; ++j)
        reinterpret_cast<uint4*>(in)[j] = reinterpret_cast<const uint4*>(p)[j];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = Ty<T>::widen(in[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = j < left ? Ty<T>::widen(p[j]) : 0.0f;
    }
  };

  // the norm: fp32 squares per thread, then trees, then the ranks in order
  float squares = 0.0f;
#pragma unroll 4
  for (int i = threadIdx.x; i < pieces; i += 256) {
    float x[8], t = 0.0f;
    int line, at;
    load8(i, x, line, at);
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaf(x[j], x[j], t);
    squares += t;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) squares += __shfl_xor_sync(0xffffffffu, squares, o);
  if (lane == 0) sSquares[warp] = squares;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int i = 0; i < 8; ++i) s += sSquares[i];
    sSquares[8] = s;
  }
  __syncthreads();
  if (shares > 1) cluster_sync();
  float sum = 0.0f;
  for (int from = 0; from < shares; ++from)
    sum += peer_load(peer_addr(smem_addr(&sSquares[8]), (uint32_t)from));
  const float by = kScale / (sqrtf(sum) + a.eps);

  // X into its planes, zeros around it
  for (int i = threadIdx.x; i < kSmallRows * (a.w / 8); i += 256) {
    const int r = i % kSmallRows, c = i / kSmallRows * 8;
    if (!a.tall && r < a.m && c < width) continue;
    alignas(16) const __half zero[8] = {};
    shared_store16(slab_at(xHi, r, c), zero);
    shared_store16(slab_at(xLo, r, c), zero);
  }
  if (a.tall) __syncthreads();
#pragma unroll 2
  for (int i = threadIdx.x; i < pieces; i += 256) {
    float x[8];
    int line, at;
    load8(i, x, line, at);
    alignas(16) __half h[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) split(x[j] * by, h[j], l[j]);
    if (a.tall) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < a.m) {
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(slab_at(xHi, at + j, line)),
                       "h"(__half_as_ushort(h[j]))
                       : "memory");
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(slab_at(xLo, at + j, line)),
                       "h"(__half_as_ushort(l[j]))
                       : "memory");
        }
    } else {
      shared_store16(slab_at(xHi, line, at), h);
      shared_store16(slab_at(xLo, line, at), l);
    }
  }

  const int quad = warp % 4, half = warp / 4, row = quad * 32 + lane;
  const uint32_t rows = tmem + ((uint32_t)(quad * 32) << 16);
  unsigned turn = 0;
  bool ok = true;
  // Everything written to shared memory is there for the products, which
  // `issue` starts; returns when they are done.  A wait that runs out is
  // reported, and the kernel goes on without waiting (its peers count on it).
  auto products = [&](auto issue) {
    asm volatile("fence.proxy.async;" ::: "memory");
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 0 && elected()) {
      issue();
      mma_commit<false>(done, 0);
    }
    __syncwarp();
    if (ok) ok = wait_phase(done, turn, nullptr, false, a.timeoutNs);
    ok = __syncthreads_and(ok) != 0;
    if (!ok && threadIdx.x == 0) atomicCAS(a.status, 0u, (unsigned)VR_ERR_TIMEOUT);
    turn ^= 1;
    tmem_fence_after();
  };
  // 32 columns of the sums at `main` (and of the low planes' at 256)
  auto sums = [&](int column, bool second, float(&v)[32]) {
    tmem_load32(rows + (unsigned)column, v);
    float u[32];
    if (second) {
      tmem_load32(rows + (unsigned)(128 + column), u);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += u[i];
    }
    if (PARTS == 2) {
      tmem_load32(rows + (unsigned)(256 + column), u);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += u[i];
    }
  };
  auto put_a = [&](int c, float(&v)[32]) {
    slab_put(aHi, row, c, v);
    if (PARTS == 2) {
      residue(v);
      slab_put(aLo, row, c, v);
    }
  };
  constexpr uint32_t kSquare = mma_idesc<__half>(128, 128, false, false);
  const uint32_t wide = mma_idesc<__half>(128, a.w, false, true);
  const int slabs = a.w / 64;

  for (int k = 0; k < a.steps; ++k) {
    // A = X X^T over this CTA's columns: two sums of two slabs each (they are
    // truncated where they are added), the low planes' apart
    products([&]() {
      for (int s = 0; s < slabs; ++s)
#pragma unroll
        for (int p = 0; p < (PARTS == 2 ? 3 : 1); ++p) {
          const uint64_t da = operand_desc((p == 2 ? xLo : xHi) + s * kSlab, 16, 1024);
          const uint64_t db = operand_desc((p == 1 ? xLo : xHi) + s * kSlab, 16, 1024);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f16<false>(tmem + (p ? 256u : s < 2 ? 0u : 128u), da + 2 * j, db + 2 * j, kSquare,
                           p ? s | (p == 2) | j : (s & 1) | j);
        }
    });
    if (shares == 1) {
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        float v[32];
        sums(half * 64 + c, slabs > 2, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= 1.0f / kScale;
        put_a(half * 64 + c, v);
      }
    } else {
      // fp32 where A's planes will be, four columns of a row together
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        float v[32];
        sums(half * 64 + c, slabs > 2, v);
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                           aHi + 16u * (unsigned)((half * 64 + c + i) / 4 * kSmallRows + row)),
                       "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3])
                       : "memory");
      }
      cluster_sync();
      // pieces of eight columns: 16 / shares of them are this CTA's, half of
      // those this thread's; with the ranks they come from, eight loads
      const int own = 16 / shares / 2, r = threadIdx.x % 128;
      const int piece0 = rank * (16 / shares) + (int)(threadIdx.x / 128) * own;
      float4 got[8][2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int piece = piece0 + i / shares;
        const uint32_t at = peer_addr(aHi, (uint32_t)(i % shares)) +
                            16u * (unsigned)(piece * 2 * kSmallRows + r);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(got[i][j].x), "=f"(got[i][j].y), "=f"(got[i][j].z), "=f"(got[i][j].w)
                       : "r"(at + 16u * (unsigned)(j * kSmallRows))
                       : "memory");
      }
      alignas(16) __half h[4][8], l[4][8];
      float v[8] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* x = reinterpret_cast<const float*>(got[i]);
        if (i % shares == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += x[j];
        if ((i + 1) % shares == 0) {
          // (i / shares is 0 .. 3 for two shares, 0 .. 1 for four, 0 for eight)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q == i / shares) {
#pragma unroll
              for (int j = 0; j < 8; ++j) split(v[j] * (1.0f / kScale), h[q][j], l[q][j]);
            }
        }
      }
      cluster_sync();  // every partial sum has been read
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q >= own) break;
        for (int to = 0; to < shares; ++to)
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            const uint4 x = *reinterpret_cast<const uint4*>(p ? l[q] : h[q]);
            asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             peer_addr(slab_at(p ? aLo : aHi, r, (piece0 + q) * 8), (uint32_t)to)),
                         "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                         : "memory");
          }
      }
      asm volatile("fence.proxy.async;" ::: "memory");
      cluster_sync();
    }
    // B = b A + c A A - d I in A's place
    products([&]() {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < (PARTS == 2 ? 3 : 1); ++p) {
          const uint64_t da = operand_desc((p == 2 ? aLo : aHi) + s * kSlab, 16, 1024);
          const uint64_t db = operand_desc((p == 1 ? aLo : aHi) + s * kSlab, 16, 1024);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f16<false>(tmem + (p ? 256u : 0u), da + 2 * j, db + 2 * j, kSquare, s | (p == 2) | j);
        }
    });
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
      float v[32];
      const int at = half * 64 + c;
      sums(at, false, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= a.coefs[k][2] * (1.0f / kScale);
      slab_add(aHi, row, at, a.coefs[k][1], v);
      if (PARTS == 2) slab_add(aLo, row, at, a.coefs[k][1], v);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (at + i == row) v[i] -= a.coefs[k][3] * kScale;
      put_a(at, v);
    }
    // X <- a X + B X
    products([&]() {
#pragma unroll
      for (int p = 0; p < (PARTS == 2 ? 3 : 1); ++p) {
        const uint64_t da = operand_desc(p == 2 ? aLo : aHi, 16, 1024);
        const uint64_t db = operand_desc(p == 1 ? xLo : xHi, kSlab, 1024);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          mma_f16<false>(tmem + (p ? 256u : 0u), da + (j / 4) * (kSlab >> 4) + 2 * (j % 4),
                         db + j * (2048 >> 4), wide, (p == 2) | j);
      }
    });
#pragma unroll 1
    for (int c = 0; c < a.w / 2; c += 32) {
      float v[32];
      const int at = half * (a.w / 2) + c;
      sums(at, false, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= 1.0f / kScale;
      slab_add(xHi, row, at, a.coefs[k][0], v);
      slab_add(xLo, row, at, a.coefs[k][0], v);
      if (k + 1 < a.steps) {
        slab_put(xHi, row, at, v);
        residue(v);
        slab_put(xLo, row, at, v);
      } else if (a.tall) {
        if (row < a.m) {  // the lanes' rows are consecutive columns of the result
          Bits* out = static_cast<Bits*>(a.dst[z]);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (at + i < width) out[(long long)(c0 + at + i) * a.m + row] = Ty<T>::narrow(v[i] * a.byOut);
        }
      } else {
        // through the warp's corner of A's place, so that a store is a row's
        // 32 columns, not 32 rows' one
        const uint32_t corner = aHi + (unsigned)(warp * (32 * 33 * 4));
#pragma unroll
        for (int i = 0; i < 32; ++i)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(corner + 4u * (unsigned)(lane * 33 + i)),
                       "f"(v[i] * a.byOut)
                       : "memory");
        __syncwarp();
        Bits* out = static_cast<Bits*>(a.dst[z]) + (long long)(quad * 32) * a.n + c0 + at + lane;
        const int rowsLeft = min(32, a.m - quad * 32);
#pragma unroll 8
        for (int i = 0; i < rowsLeft; ++i) {
          float x;
          asm volatile("ld.shared.f32 %0, [%1];"
                       : "=f"(x)
                       : "r"(corner + 4u * (unsigned)(i * 33 + lane))
                       : "memory");
          if (at + lane < width) out[(long long)i * a.n] = Ty<T>::narrow(x);
        }
        __syncwarp();
      }
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (shares > 1) cluster_sync();  // no peer reads this CTA's memory any more
  if (warp == 0) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

size_t up(size_t n, size_t to) { return (n + to - 1) / to * to; }

struct OrthoPlan {
  int parts;         // planes of the operands
  size_t m, n;       // X: m <= n
  size_t ldX, ldA, group;  // matrices per launch
  size_t part, x[2][2], a[2], b[2], bytes;
};

bool make_plan(int count, size_t rows, size_t cols, int dtype, OrthoPlan* p) {
  if (!op_elem_size(dtype) || count < 1 || rows < 1 || cols < 1 || rows > (1u << 24) ||
      cols > (1u << 24))
    return false;
  p->m = std::min(rows, cols);
  p->parts = dtype == VR_BFLOAT16 && p->m > kFewRows ? 1 : 2;
  p->n = std::max(rows, cols);
  p->ldX = up(p->n, 32);
  p->ldA = up(p->m, 32);
  p->group = std::min<size_t>(count, kMost);
  size_t at = 0;
  auto take = [&at](size_t n) {
    const size_t here = at;
    at += op_round(n);
    return here;
  };
  p->part = take(p->group * kNormCtas * 4);
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      // one plane: the low plane is no operand, every element of it is read and
      // written by one thread, so it is updated in place
      p->x[i][j] = i && j && p->parts == 1 ? p->x[0][1] : take(p->group * p->m * p->ldX * 2);
  for (int j = 0; j < p->parts; ++j) p->a[j] = take(p->group * p->m * p->ldA * 2);
  for (int j = 0; j < p->parts; ++j) p->b[j] = take(p->group * p->m * p->ldA * 2);
  p->bytes = at + kOpSlack;
  return true;
}

// What moves from B's diagonal to the factor of X: X <- (a + d) X + (B - d I) X.
// Near convergence A is near I and B near (b + c) I, so B - d I is small, and
// with it what the roundings of B's and X's operands contribute (bf16 results
// of decaying spectra: 1.7e-3 to 1.2e-3 before the last rounding, simulated
// and measured).  Early steps keep d = 0: it would add roundings of X in the
// small directions, which later steps amplify.
float shift_of(const float* coefs, int steps, int k) {
  const float at1 = coefs[3 * k + 1] + coefs[3 * k + 2];
  return k + 1 == steps ? at1 : k + 2 == steps ? 0.5f * at1 : 0.0f;
}

// Whether every intermediate stays below what the planes hold (16) for any
// matrix: the singular values start in [0, 1], and a step maps s to
// a s + b s^3 + c s^5.
bool in_range(const float* coefs, int steps) {
  double top = 1.0;
  for (int k = 0; k < steps; ++k) {
    const double a = coefs[3 * k], b = coefs[3 * k + 1], c = coefs[3 * k + 2];
    const double reach = top * 1.01;  // roundings
    double next = 0.0;
    if (reach * reach > 15.0) return false;
    for (int i = 0; i <= 512; ++i) {
      const double s = reach * i / 512.0, q = s * s;
      const double poly = b * q + c * q * q;
      if (std::fabs(poly) > 15.0 || std::fabs(poly - shift_of(coefs, steps, k)) > 15.0)
        return false;
      next = std::max(next, std::fabs(s * (a + b * q + c * q * q)));
    }
    top = next;
  }
  return top <= 15.0;
}

constexpr float kCoefs[3] = {3.4445f, -4.7750f, 2.0315f};

// One product of a step, on the tile shape that a model of the measured
// times puts first.  A slice of 64 k takes 0.205 us on a 128 x 128 tile of one
// CTA, 0.167 us on a 256 x 128 tile of a pair (half the operand traffic per
// SM), 0.31 us on a 256 x 256 one (two planes: 0.56 and 0.47 us, no 256-wide
// tile, tensor memory holds 128 columns), the epilogue of the last round 3 us
// per 128 columns, and joining s shares of k s + 2 us.  Wide tiles win when there
// are many, single CTAs when they fill the SMs once, shares when few tiles
// leave SMs idle.
template <int PARTS, bool BMN, class Epi>
vr_result_t product(const OpDevice& dev, const Planes& a, size_t aLd, const Planes& b, size_t bLd,
                    const GemmSize& z, typename Epi::Args& epi, void* stream) {
  const Operand oa = {a.hi, a.lo, aLd}, ob = {b.hi, b.lo, bLd};
  constexpr int CHUNK = PARTS == 2 ? kSplitChunk : 0;
  const double slices = (double)((z.K + kTileK - 1) / kTileK);
  double best = 0;
  int shape = -1, shares = 1;  // shape: 0 single, 1 pair, 2 wide pair
  auto offer = [&](int which, size_t tiles, double slice, int s) {
    // clusters of four and eight CTAs do not fill the GPU (36 and 15 of them are
    // resident at a time), and are only worth while in one round
    const size_t ctas = (which ? 2 : 1) * (size_t)s;
    const size_t room = ctas > 4 ? 15 : ctas > 2 ? 36 : (size_t)dev.sms / ctas;
    const double rounds = (double)((tiles + room - 1) / room);
    if (s > 1 && rounds > 1) return;
    const double t = rounds * std::ceil(slices / s) * slice + (which == 2 ? 6 : 3) + (s > 1 ? s + 2 : 0);
    if (shape < 0 || t < best) best = t, shape = which, shares = s;
  };
  const size_t singles = gemm_tiles<128, false>(z), pairs = gemm_tiles<128, true>(z);
  for (int s = 1; s <= 8 && s <= slices; s *= 2) {
    offer(0, singles, PARTS == 2 ? 0.56 : 0.205, s);
    if (s <= 4 && z.M > kTileM) offer(1, pairs, PARTS == 2 ? 0.47 : 0.167, s);
  }
  if (PARTS == 1 && z.M > kTileM) offer(2, gemm_tiles<256, true>(z), 0.31, 1);
#define VR_PRODUCT(BN, PAIR, SPLIT)                                                      \
  return gemm_launch<__half, BN, PARTS, false, BMN, CHUNK, PAIR, SPLIT, Epi>(            \
      dev, oa, ob, z, nullptr, nullptr, epi, shares, stream)
  if constexpr (PARTS == 1) {
    if (shape == 2) VR_PRODUCT(256, true, false);
  }
  if (shape == 1) {
    if (shares > 1) VR_PRODUCT(128, true, true);
    VR_PRODUCT(128, true, false);
  }
  if (shares > 1) VR_PRODUCT(128, false, true);
  VR_PRODUCT(128, false, false);
#undef VR_PRODUCT
}

template <typename T, int PARTS>
vr_result_t run(const OrthoPlan& p, const OpDevice& dev, const void* const* src, void* const* dst,
                int count, size_t rows, size_t cols, int steps, const float* coefs, float eps,
                float scale, char* w, void* stream) {
  const bool tall = rows > cols;
  if (p.m <= kSmallRows && p.n <= (size_t)kSmallCols * kSmallCtas) {
    SmallArgs a = {};
    int shares = 1;
    // 128 columns a CTA where the SMs allow, at most 256
    while ((size_t)shares * kSmallCols < p.n ||
           (shares < kSmallCtas && (size_t)shares * 128 < p.n && 2 * shares * count <= dev.sms))
      shares *= 2;
    a.m = (int)p.m;
    a.n = (int)p.n;
    a.w = (int)up((p.n + shares - 1) / shares, 64);
    a.tall = tall;
    a.steps = steps;
    a.eps = eps;
    a.byOut = scale / kScale;
    a.status = dev.status;
    a.timeoutNs = dev.timeoutNs;
    for (int k = 0; k < steps; ++k) {
      const float d = shift_of(coefs, steps, k);
      a.coefs[k][0] = coefs[3 * k] + d;
      a.coefs[k][1] = coefs[3 * k + 1];
      a.coefs[k][2] = coefs[3 * k + 2];
      a.coefs[k][3] = d;
    }
    for (int i = 0; i < count; ++i) a.src[i] = src[i], a.dst[i] = dst[i];
    const void* fn = (const void*)ortho_small_kernel<T, PARTS>;
    const vr_result_t e = gemm_prepare(fn, dev.device, kSmallSmem);
    if (e != VR_SUCCESS) return e;
    void* args[] = {&a};
    return op_launch(fn, dim3((unsigned)(count * shares)), dim3(256), args, kSmallSmem, stream,
                     shares);
  }
  auto plane = [w](size_t at) { return reinterpret_cast<__half*>(w + at); };
  const Planes x[2] = {{plane(p.x[0][0]), plane(p.x[0][1])}, {plane(p.x[1][0]), plane(p.x[1][1])}};
  const Planes A = {plane(p.a[0]), PARTS == 2 ? plane(p.a[1]) : nullptr};
  const Planes B = {plane(p.b[0]), PARTS == 2 ? plane(p.b[1]) : nullptr};
  const long long sizeX = (long long)(p.m * p.ldX), sizeA = (long long)(p.m * p.ldA);
  LoadArgs la = {};
  la.rows = (long long)rows;
  la.cols = (long long)cols;
  la.part = reinterpret_cast<float*>(w + p.part);
  la.eps = eps;
  la.tall = tall;
  la.x = x[0];
  la.ld = (long long)p.ldX;
  la.size = sizeX;
  typename ApplyEpilogue<T>::Args ap = {};
  ap.vec = cols % Ty<T>::U == 0;
  for (int i = 0; i < count; ++i) {
    la.src[i] = src[i];
    ap.out[i] = static_cast<T*>(dst[i]);
    if ((uintptr_t)dst[i] & 15) ap.vec = 0;
  }
  // about two CTAs per SM over all matrices, 8192 elements each at least
  la.ctas = (int)std::max<size_t>(
      1, std::min({(size_t)kNormCtas, rows * cols / 8192, (size_t)(2 * dev.sms / count + 1)}));
  void* args[] = {&la};
  vr_result_t e = op_launch((const void*)ortho_norm_kernel<T>, dim3(la.ctas, count), dim3(256),
                            args, 0, stream);
  if (e != VR_SUCCESS) return e;
  const size_t blocks =
      tall ? (rows + 63) / 64 * ((cols + 31) / 32) : (rows * ((cols + 7) / 8) + 255) / 256;
  e = op_launch((const void*)ortho_load_kernel<T>,
                dim3((unsigned)std::min<size_t>(blocks, (size_t)dev.sms * 8), count), dim3(256),
                args, 0, stream);
  if (e != VR_SUCCESS) return e;
  const size_t n = (size_t)count;
  for (int k = 0; k < steps; ++k) {
    const float a = coefs[3 * k], b = coefs[3 * k + 1], c = coefs[3 * k + 2];
    const Planes &from = x[k % 2], &to = x[1 - k % 2];
    const float shift = shift_of(coefs, steps, k);
    SymmetricEpilogue::Args sym = {};
    sym.p.to = A;
    sym.p.ld = (long long)p.ldA;
    sym.p.size = sizeA;
    sym.p.byAcc = 1.0f / kScale;
    sym.nOut = PARTS;
    if ((e = product<PARTS, false, SymmetricEpilogue>(dev, from, p.ldX, from, p.ldX,
                                                      {p.m, p.m, p.n, n, true}, sym, stream)) !=
        VR_SUCCESS)
      return e;
    sym.p.from = A;
    sym.p.to = B;
    sym.p.byFrom = b;
    sym.p.byAcc = c / kScale;
    sym.p.diagonal = shift * kScale;
    sym.nIn = PARTS;
    if ((e = product<PARTS, false, SymmetricEpilogue>(
             dev, A, p.ldA, A, p.ldA, {p.m, p.m, p.m, n, true}, sym, stream)) != VR_SUCCESS)
      return e;
    ap.last = k + 1 == steps;
    ap.aux.nIn = 2;
    ap.aux.nOut = ap.last ? 0 : 2;
    for (int i = 0; i < 2; ++i) {
      auto tiles = [&](CUtensorMap* map, const __half* plane) {
        return gemm_operand(map, plane, false, p.n, p.m, n, p.ldX * 2, (size_t)sizeX * 2, kTileM,
                            kAuxCols);
      };
      if ((e = tiles(&ap.aux.in[i], i ? from.lo : from.hi)) != VR_SUCCESS ||
          (e = tiles(&ap.aux.out[i], i ? to.lo : to.hi)) != VR_SUCCESS)
        return e;
    }
    ap.p.from = from;
    ap.p.to = to;
    ap.p.ld = (long long)p.ldX;
    ap.p.size = sizeX;
    ap.p.byFrom = a + shift;
    ap.p.byAcc = 1.0f / kScale;
    ap.tall = tall;
    ap.byOut = scale / kScale;
    ap.cols = (int)p.n;
    if ((e = product<PARTS, true, ApplyEpilogue<T>>(
             dev, B, p.ldA, from, p.ldX, {p.m, p.n, p.m, n, false}, ap, stream)) != VR_SUCCESS)
      return e;
  }
  return VR_SUCCESS;
}

}  // namespace
}  // namespace vr

using namespace vr;

extern "C" {

vr_result_t vr_orthogonalize_workspace_bytes(int count, size_t rows, size_t cols, vr_dtype_t dtype,
                                             size_t* bytes) {
  OrthoPlan p = {};
  if (!bytes || !make_plan(count, rows, cols, dtype, &p)) return VR_ERR_INVALID_ARGUMENT;
  *bytes = p.bytes;
  return VR_SUCCESS;
}

vr_result_t vr_orthogonalize(const void* const* src, void* const* dst, int count, size_t rows,
                             size_t cols, vr_dtype_t dtype, int steps, const float* coefs,
                             float eps, float scale, void* workspace, size_t workspaceBytes,
                             void* stream) {
  OrthoPlan p = {};
  if (!make_plan(count, rows, cols, dtype, &p) || !src || !dst || steps < 1 || steps > 32 ||
      !(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(scale) || !workspace ||
      workspaceBytes < p.bytes || ((uintptr_t)workspace & 15))
    return VR_ERR_INVALID_ARGUMENT;
  const size_t E = op_elem_size(dtype), bytes = rows * cols * E;
  float use[3 * 32];
  for (int k = 0; k < 3 * steps; ++k) {
    use[k] = coefs ? coefs[k] : kCoefs[k % 3];
    if (!std::isfinite(use[k])) return VR_ERR_INVALID_ARGUMENT;
  }
  for (int i = 0; i < count; ++i)
    if (!src[i] || !dst[i] || ((uintptr_t)src[i] | (uintptr_t)dst[i]) % E)
      return VR_ERR_INVALID_ARGUMENT;
  if (!op_lists_ok(src, dst, count, bytes, workspace, workspaceBytes))
    return VR_ERR_INVALID_ARGUMENT;
  if (!in_range(use, steps)) return VR_ERR_UNSUPPORTED;
  OpDevice dev;
  vr_result_t e = op_device(&dev);
  const void* const work = workspace;
  if (e != VR_SUCCESS || (e = op_reachable(src, count, dev.device)) != VR_SUCCESS ||
      (e = op_reachable(dst, count, dev.device)) != VR_SUCCESS ||
      (e = op_reachable(&work, 1, dev.device)) != VR_SUCCESS)
    return e;
  char* w = op_workspace(workspace);
  for (int at = 0; at < count && e == VR_SUCCESS; at += kMost) {
    const int n = std::min(kMost, count - at);
    e = dtype == VR_FLOAT32 ? run<float, 2>(p, dev, src + at, dst + at, n, rows, cols, steps, use,
                                            eps, scale, w, stream)
        : dtype == VR_FLOAT16
            ? run<__half, 2>(p, dev, src + at, dst + at, n, rows, cols, steps, use, eps, scale, w,
                             stream)
        : p.parts == 2
            ? run<__nv_bfloat16, 2>(p, dev, src + at, dst + at, n, rows, cols, steps, use, eps,
                                    scale, w, stream)
            : run<__nv_bfloat16, 1>(p, dev, src + at, dst + at, n, rows, cols, steps, use, eps,
                                    scale, w, stream);
  }
  return e;
}

}  // extern "C"
