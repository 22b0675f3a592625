// Softmax cross entropy of a linear layer over a large vocabulary
// (vr_linear_xent).
//
//   l_tv = h_t . w_v;  lse_t = log sum_v exp l_tv;  loss_t = lse_t - l_t,y(t)
//   g_tv = s (exp(l_tv - lse_t) - [v = y(t)]);  dH = G W;  dW = G^T H
//
// The logits are never stored.  The first product (gemm.cuh) turns every 64
// (few rows: 32) columns of a row of them into one maximum and one sum of
// exp(l - maximum) in its epilogue; joining these pairs gives the row's, and
// lse.  For the gradients there are two ways:
//   kept     the same epilogue also writes exp(l - the tile's maximum) in 16
//            bits; once lse is known a pass over them makes the gradient
//            factors p - [v = y] of them in place.  6 T D V operations.  Taken
//            while T x V 16-bit values are no more memory than the weight has
//            (T <= D), or 256 MB, and the workspace has room for them.
//   pieces   the vocabulary is taken piece by piece: the product runs again,
//            its epilogue now writing the factors.  8 T D V operations; of the
//            workspace only the pairs grow with T x V, an eighth of a byte each.
// Two more products multiply the factors with the weight and with the hidden
// states.  (4096 tokens x 4096 x 131072, bf16: 8.4-8.6 ms kept, 10.4 ms in pieces.)
//
// Only tokens that count take part in the gradients: the hidden states are
// packed first, tokens that count before ignored ones, which leaves out the
// products of ignored tokens and whatever such tokens hold (NaN times zero
// is NaN).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "rows.cuh"

namespace vr {
namespace {

constexpr int kBN = 256;
// Columns of one pair of statistics: a quarter of a tile of 256, or of 128
// where few rows and few tiles would leave SMs idle.
constexpr int kPartCols = kBN / 4;
// The losses are fp32 results: their logits are summed in chunks of 512.
// The gradients are rounded to 16 bits; the truncation takes 1.6e-8 off them
// per 16 k (1.3e-4 of a dH summed over 131072 in one go: with fp16's rounding of
// 2.08e-4 on average 2.58e-4 in all, 2.09e-4 in chunks; with bf16's 1.663e-3
// 1.671e-3).  Sums that it would cost more than a sixth of the rounding go in
// chunks of 2048, which takes no longer.
// Up to 128 rows the weight's traffic bounds the product, whose sums then
// change hands every 128.
constexpr int kStatsChunk = 8, kFewRowsChunk = 2, kLongChunk = 32;
template <typename T>
constexpr size_t kLongSum = std::is_same<T, __half>::value ? 32768 : 262144;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Device-side results of the preparation.
struct XentState {
  int valid;        // tokens that count
  int rows;         // packed rows: those, zeros up to whole slices, the others
  float lossScale;  // 1 / valid or 1
  float gradScale;  // of the 16-bit gradient factors
};

// The gradient factors p - [v = y] lie in [-1, 1]; small p are common.  fp16
// holds them times 2^14 (down to 2^-28 normal), bf16 as they are.
template <typename T>
constexpr int kShift = std::is_same<T, __half>::value ? 14 : 0;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The target of a row, -1 where there is none: prepared with the packed
// tokens, or, for the loss alone, the caller's own.
struct Targets {
  const int* of;
  const long long* raw;  // used where `of` is null
  long long ignore;
  int V;
  __device__ __forceinline__ bool bad(long long y) const {
    return y != ignore && (y < 0 || y >= V);
  }
  __device__ __forceinline__ int at(int row) const {
    if (of) return of[row];
    const long long y = raw[row];
    return y == ignore || bad(y) ? -1 : (int)y;
  }
};

// Row statistics of a tile of logits: the maximum and the sum of exp(l -
// maximum) over each part of it, and the target's logit; KEEP: and each
// exp(l - maximum) in 16 bits.  The difference is taken first, not in one
// multiply-add with a rounded maximum log2 e: that rounding (2^-18 at 60) would
// be all that is left of a confident token's 1 - p, and of its loss.
template <typename T, bool KEEP>
struct StatsEpilogue {
  static constexpr bool kAux = false;
  static constexpr int kWarps = 16;
  struct Args {
    Targets target;
    float* targetLogit;
    float2* parts;      // [rows][nParts]
    int nParts;
    T* out;             // KEEP: [rows][ld]
    long long ld;
    const XentState* state;
  };
  template <int COLS, class Acc>
  static __device__ __forceinline__ void run(const Args& a, const GemmArgs& g, const Tile& o,
                                             int row, int col0, int M, const Acc& acc) {
    const int t = o.m0 + row;
    const int first = o.n0 + col0;
    const int at = t < M ? a.target.at(t) - first : -1;
    constexpr int STEP = Acc::kStep;
    auto fetch = [&](int c, float(&v)[STEP]) {
      acc(col0 + c, v);
      if (first + c + STEP > g.N) {
#pragma unroll
        for (int i = 0; i < STEP; ++i)
          if (first + c + i >= g.N) v[i] = -INFINITY;
      }
    };
    // (four chains each of maxima and sums, one would wait for itself)
    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sums[4] = {};
#pragma unroll
    for (int c = 0; c < COLS; c += STEP) {
      if (first + c >= g.N) break;
      float v[STEP];
      fetch(c, v);
#pragma unroll
      for (int i = 0; i < STEP; ++i) tops[i % 4] = fmaxf(tops[i % 4], v[i]);
    }
    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    // nothing but -inf: subtract 0, so that exp2 gives 0, not NaN
    const float base = top == -INFINITY ? 0.0f : top;
    const bool store = KEEP && t < M && t < a.state->valid;
    constexpr float up = KEEP ? (float)kShift<T> : 0.0f;  // exact: a power of two
#pragma unroll
    for (int c = 0; c < COLS; c += STEP) {
      if (first + c >= g.N) break;
      float v[STEP];
      fetch(c, v);
#pragma unroll
      for (int i = 0; i < STEP; ++i) {
        v[i] = exp2_fast(fmaf(v[i] - base, kLog2e, up));
        sums[i % 4] += v[i];
      }
      if (store) store_row(a.out + (long long)t * a.ld + first + c, v, STEP, 32);
    }
    const float sum = ((sums[0] + sums[1]) + (sums[2] + sums[3])) *
                      (1.0f / (float)(1 << (KEEP ? kShift<T> : 0)));
    acc.pick(at >= 0 && at < COLS ? col0 + at : -1, [&](float x) { a.targetLogit[t] = x; });
    if (t < M) a.parts[(long long)t * a.nParts + first / COLS] = make_float2(top, sum);
  }
};

// The kept exponentials of the packed tokens made into gradient factors, and
// rows of zeros up to the next whole slice.  The target's factor is made of
// its fp32 logit (target_factor).  One read and one write: 2048 x 32768 in 48 us
// from cold caches (ncu), 5.6 TB/s.
template <typename T>
struct KeptArgs {
  T* out;
  long long ld;
  const float2* parts;
  int nParts, partCols, V;
  const float2* softmax;
  const int* target;
  const float* targetLogit;
  const XentState* state;
};
// p - 1 of the target, of a confident token a small difference: (e - sum) / sum
// with the same e that the sum holds is what the others' sum is.
__device__ __forceinline__ float target_factor(float logit, float2 softmax, float by) {
  return (exp2_fast((logit - softmax.x) * kLog2e) - softmax.y) * by;
}
constexpr int kKeptUnits = 4;  // of 8 values a thread
template <typename T>
__global__ void __launch_bounds__(256) xent_kept_kernel(const __grid_constant__ KeptArgs<T> a) {
  pdl_launch();
  pdl_wait();
  const int valid = a.state->valid, rows = (valid + kTileK - 1) / kTileK * kTileK;
  const int c0 = (blockIdx.x * kKeptUnits * 256 + threadIdx.x) * 8;
  for (int t = blockIdx.y; t < rows; t += gridDim.y) {
    T* out = a.out + t * a.ld;
    const float2 row = t < valid ? a.softmax[t] : make_float2(0.0f, 1.0f);
    const float inv = __fdividef(1.0f, row.y);
    const int y = t < valid ? a.target[t] : -1;
    uint4 q[kKeptUnits];
    float2 part[kKeptUnits];
#pragma unroll
    for (int u = 0; u < kKeptUnits; ++u) {
      const int c = c0 + u * 256 * 8;
      if (t < valid && c < a.V) {
        q[u] = *reinterpret_cast<const uint4*>(out + c);
        part[u] = a.parts[(long long)t * a.nParts + c / a.partCols];
      }
    }
#pragma unroll
    for (int u = 0; u < kKeptUnits; ++u) {
      const int c = c0 + u * 256 * 8;
      if (c >= a.V) break;
      if (t >= valid) {
        *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
        continue;
      }
      const float by = exp2_fast((part[u].x - row.x) * kLog2e) * inv;
      uint32_t* w = reinterpret_cast<uint32_t*>(&q[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = Ty<T>::widen((typename Ty<T>::Bits)(w[i] & 0xffffu)) * by;
        float z = Ty<T>::widen((typename Ty<T>::Bits)(w[i] >> 16)) * by;
        if ((y >> 1) == (c >> 1) + i)
          (y & 1 ? z : x) = target_factor(a.targetLogit[t], row, inv * (float)(1 << kShift<T>));
        w[i] = pack2<T>(x, z);
      }
      *reinterpret_cast<uint4*>(out + c) = q[u];
    }
  }
}

// Gradient factors of a tile of a piece of the vocabulary.
template <typename T>
struct FactorEpilogue {
  static constexpr bool kAux = false;
  static constexpr int kWarps = 16;
  struct Args {
    const int* target;         // packed tokens' targets
    const float* targetLogit;  // and their logits, as the sums hold them
    const float2* softmax;     // maximum and sum of each
    T* out;                    // [tokens][ld]
    long long ld;
    int v0;              // the piece's first row of the vocabulary
  };
  template <int COLS, class Acc>
  static __device__ __forceinline__ void run(const Args& a, const GemmArgs& g, const Tile& o,
                                             int row, int col0, int M, const Acc& acc) {
    const int t = o.m0 + row;
    const bool live = t < M;
    // dW reads whole slices of tokens: zeros up to there.  A tile's rows go on
    // past the buffer's.
    const bool stored = t < (M + kTileK - 1) / kTileK * kTileK;
    const float2 sum = live ? a.softmax[t] : make_float2(0.0f, 1.0f);
    const float by = __fdividef((float)(1 << kShift<T>), sum.y);
    const int at = live ? a.target[t] - a.v0 - o.n0 - col0 : -1;
    T* out = a.out + (long long)t * a.ld + o.n0 + col0;
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      if (o.n0 + col0 + c >= g.N) break;
      float v[32];
      acc(col0 + c, v);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        v[i] = live ? exp2_fast((v[i] - sum.x) * kLog2e) * by : 0.0f;
      if (stored) store_row(out + c, v, 32, 32);
    }
    // the target's factor over the one just written by the same thread
    if (at >= 0 && at < COLS && o.n0 + col0 + at < g.N)
      reinterpret_cast<typename Ty<T>::Bits*>(out)[at] =
          Ty<T>::narrow(target_factor(a.targetLogit[t], sum, by));
  }
};

// dH: the pieces' products added up in fp32 in piece order, rounded once.
template <typename T>
struct HiddenEpilogue {
  static constexpr bool kAux = false;
  static constexpr int kWarps = 16;
  struct Args {
    float* sum;            // [packed tokens][ld]
    long long ld;
    T* out;                // [T][N]
    const int* token;      // packed token -> token
    const XentState* state;
    int first, last, align;
  };
  template <int COLS, class Acc>
  static __device__ __forceinline__ void run(const Args& a, const GemmArgs& g, const Tile& o,
                                             int row, int col0, int M, const Acc& acc) {
    const int t = o.m0 + row;
    const bool live = t < M;
    const float scale = a.last ? a.state->gradScale : 0.0f;
    T* out = a.out + (a.last && live ? (long long)a.token[t] * g.N : 0);
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      const int n = o.n0 + col0 + c;
      if (n >= g.N) break;
      float v[32];
      acc(col0 + c, v);
      if (!live) continue;
      float4* sum = reinterpret_cast<float4*>(a.sum + (long long)t * a.ld + n);
      if (!a.first) {  // rows are padded to whole groups of 32 columns
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 s = sum[i];
          v[4 * i] += s.x, v[4 * i + 1] += s.y, v[4 * i + 2] += s.z, v[4 * i + 3] += s.w;
        }
      }
      if (a.last) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= scale;
        store_row(out + n, v, g.N - n, a.align);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          sum[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
  }
};

// dW: rows of one piece of the vocabulary, whole sums over the tokens.
template <typename T>
struct WeightEpilogue {
  static constexpr bool kAux = false;
  static constexpr int kWarps = 16;
  struct Args {
    T* out;  // the piece's first row
    long long ld;
    const XentState* state;
    int align;
  };
  template <int COLS, class Acc>
  static __device__ __forceinline__ void run(const Args& a, const GemmArgs& g, const Tile& o,
                                             int row, int col0, int M, const Acc& acc) {
    const int v0 = o.m0 + row;
    const float scale = a.state->gradScale;
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      const int n = o.n0 + col0 + c;
      if (n >= g.N) break;
      float v[32];
      acc(col0 + c, v);
      if (v0 >= M) continue;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= scale;
      store_row(a.out + v0 * a.ld + n, v, g.N - n, a.align);
    }
  }
};

// The same through shared memory and tensor copies, for rows of whole 16-byte
// units that are no 32-byte ones.  With few tokens their stores, twice as many
// and across sectors, are what takes the time; with many the products want the
// shared memory for their stages.  Loss and dWeight, bf16, us row by row and
// this way:
//   tokens              64        256        768       1024       1280       2048
//   dim 1032 x 131072   260 204   287 232    478 431   571 533    773 781  1228 1256
//   dim 1000 x 50001    111 104   122 112    192 175   233 220    269 260   387 386
//   dim 2056 x 32768    139 133   152 143    221 197   254 239    300 292   441 436
// Rows of 32-byte units are stored row by row:
//   dim 2048 x 32768     99 112   111 123    176 180   195 214    239 260   375 376
//   dim 1024 x 131072   191 212   215 241    346 357   441 452    623 612  1036 1060
template <typename T>
struct WeightTilesEpilogue {
  static constexpr bool kAux = true;
  static constexpr int kWarps = 8;
  struct Args {
    AuxArgs aux;
    const XentState* state;
  };
  static __device__ __forceinline__ bool skip(const GemmArgs& g, const Tile& o, int n, int M) {
    return n >= g.N || o.m0 >= M;
  }
  template <class Acc>
  static __device__ __forceinline__ void unit(const Args& a, const GemmArgs& g, const Tile& o,
                                              int row, int n, int c, int M, const Acc& acc,
                                              const AuxTile& tile) {
    const float scale = a.state->gradScale;
    float v[32];
    acc(c, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack2<T>(v[8 * i + 2 * j] * scale, v[8 * i + 2 * j + 1] * scale);
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile.piece(0, row, i)),
                   "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                   : "memory");
    }
  }
};
constexpr size_t kTilesMostTokens = 1024;

// One CTA: the targets narrowed (-1: ignored), the tokens that count packed
// in order, their number and the scales.  A target outside the vocabulary is
// reported in the status word and ignored.
struct PrepArgs {
  const long long* targets;
  long long ignore;
  int T, V, mean;
  float gradScale;
  int shift;
  int* target;
  int *token, *skipped;  // the tokens that count, and the others, in order
  XentState* state;
  unsigned* status;
};
__global__ void __launch_bounds__(1024) xent_prep_kernel(const __grid_constant__ PrepArgs a) {
  __shared__ int sWarp[32];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int base = 0;
  for (int t0 = 0; t0 < a.T; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    int y = -1;
    if (t < a.T) {
      const long long raw = a.targets[t];
      if (raw >= 0 && raw < a.V && raw != a.ignore) y = (int)raw;
      else if (raw != a.ignore) atomicCAS(a.status, 0u, (unsigned)VR_ERR_INVALID_ARGUMENT);
      a.target[t] = y;
    }
    const unsigned votes = __ballot_sync(0xffffffffu, y >= 0);
    if (lane == 0) sWarp[warp] = __popc(votes);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      const int n = sWarp[w];
      before += w < warp ? n : 0;
      all += n;
    }
    const int at = base + before + __popc(votes & ((1u << lane) - 1));
    if (y >= 0) a.token[at] = t;
    else if (t < a.T) a.skipped[t - at] = t;
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float per = a.mean ? (base ? 1.0f / (float)base : 0.0f) : 1.0f;
    a.state->valid = base;
    a.state->rows = (base + kTileK - 1) / kTileK * kTileK + a.T - base;
    a.state->lossScale = per;
    a.state->gradScale = per * a.gradScale * exp2f((float)-a.shift);
  }
}

// A (maximum, sum of exp(l - maximum)) pair over more columns: the other's sum
// brought to the common maximum.  -inf: nothing so far.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x), base = top == -INFINITY ? 0.0f : top;
  return make_float2(top, a.y * exp2f((a.x - base) * kLog2e) + b.y * exp2f((b.x - base) * kLog2e));
}

// Joins the rows' pairs, and, in one CTA (ALL), sums the loss.  A warp takes a
// row, or, where one CTA has few rows, several warps do.
struct JoinArgs {
  const float2* parts;
  int nParts, T;
  const int* rowToken;     // packed rows' tokens (-1: none), or null: row = token
  const XentState* state;  // null with raw targets
  Targets target;
  int mean;
  const float* targetLogit;
  float2* softmax;         // the rows' joined pairs
  float *lse, *losses, *loss;
  unsigned* status;
};
// The loss from the tokens' losses, by one CTA of 1024 threads: in 64 bits, in
// a fixed order.  Raw targets are counted here, and bad ones reported.
__device__ __forceinline__ void sum_losses(const JoinArgs& a) {
  __shared__ double sSum[32];
  __shared__ int sCount[32];
  double sum = 0.0;
  int count = 0;
  for (int t = threadIdx.x; t < a.T; t += 1024) {
    sum += (double)a.losses[t];
    if (!a.state) {
      count += a.target.at(t) >= 0;
      if (a.target.bad(a.target.raw[t])) atomicCAS(a.status, 0u, (unsigned)VR_ERR_INVALID_ARGUMENT);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  count = __reduce_add_sync(0xffffffffu, count);
  if (threadIdx.x % 32 == 0) sSum[threadIdx.x / 32] = sum, sCount[threadIdx.x / 32] = count;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) sum += sSum[w], count += sCount[w];
    const float scale = a.state ? a.state->lossScale : a.mean ? 1.0f / (float)max(count, 1) : 1.0f;
    *a.loss = (float)(sum * (double)scale);
  }
}
template <bool ALL>
__global__ void __launch_bounds__(ALL ? 1024 : 256)
    xent_join_kernel(const __grid_constant__ JoinArgs a) {
  constexpr int WARPS = ALL ? 32 : 8;
  __shared__ float2 sPair[WARPS];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int rows = a.rowToken ? a.state->rows : a.T;
  int each = 1;  // warps of a row
  while (ALL && 2 * each * max(rows, 1) <= WARPS) each *= 2;
  const int step = (int)gridDim.x * (WARPS / each);
  // (all warps of a CTA go the same number of rounds)
  for (int t0 = (int)blockIdx.x * (WARPS / each); t0 < rows; t0 += step) {
    const int t = t0 + warp / each;
    const int token = t >= rows ? -1 : a.rowToken ? a.rowToken[t] : t;
    float2 pair = make_float2(-INFINITY, 0.0f);
    if (token >= 0) {
      const float2* p = a.parts + (long long)t * a.nParts;
      const int by = 32 * each;
      int i = lane + 32 * (warp % each);
      for (; i + 3 * by < a.nParts; i += 4 * by) {
        float2 q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = p[i + k * by];
        pair = join(pair, join(join(q[0], q[1]), join(q[2], q[3])));
      }
      for (; i < a.nParts; i += by) pair = join(pair, p[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float2 other = make_float2(__shfl_xor_sync(0xffffffffu, pair.x, o),
                                       __shfl_xor_sync(0xffffffffu, pair.y, o));
      pair = join(pair, other);
    }
    if (ALL && each > 1) {
      if (lane == 0) sPair[warp] = pair;
      __syncthreads();
      if (warp % each == 0)
        for (int w = 1; w < each; ++w) pair = join(pair, sPair[warp + w]);
      __syncthreads();
    }
    if (lane == 0 && warp % each == 0 && token >= 0) {
      const float base = pair.x == -INFINITY ? 0.0f : pair.x;
      const float rest = log2f(pair.y) * kLn2;
      a.softmax[t] = pair;
      a.lse[token] = base + rest;
      // (not lse - l, which keeps only what lse has digits for)
      a.losses[token] = a.target.at(t) >= 0 ? (base - a.targetLogit[t]) + rest : 0.0f;
    }
  }
  if (ALL) {
    __syncthreads();
    sum_losses(a);
  }
}
__global__ void __launch_bounds__(1024) xent_loss_kernel(const __grid_constant__ JoinArgs a) {
  pdl_launch();
  pdl_wait();
  sum_losses(a);
}

// The packed hidden states: the tokens that count, zeros up to whole slices
// of 64 rows, the others; each row's token and target; and zero gradients for
// the others.
struct PackArgs {
  const uint16_t* hidden;
  long long stride;
  int T, D, ld, vec;
  const int *target, *token, *skipped;
  const XentState* state;
  uint16_t* packed;
  int *rowToken, *rowTarget;
  uint16_t* dHidden;  // [T][D] or null
};
__global__ void __launch_bounds__(256) xent_pack_kernel(const __grid_constant__ PackArgs a) {
  pdl_launch();
  pdl_wait();
  const int valid = a.state->valid, rows = a.state->rows;
  const int whole = (valid + kTileK - 1) / kTileK * kTileK;
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const int t = r < valid ? a.token[r] : r < whole ? -1 : a.skipped[r - whole];
    uint16_t* out = a.packed + (long long)r * a.ld;
    const uint16_t* in = a.hidden + (t < 0 ? 0 : t * a.stride);
    if (a.vec) {
      for (int c = threadIdx.x * 8; c < a.ld; c += 256 * 8)
        *reinterpret_cast<uint4*>(out + c) =
            t < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(in + c);
    } else {
      for (int c = threadIdx.x; c < a.ld; c += 256)
        out[c] = t >= 0 && c < a.D ? in[c] : (uint16_t)0;
    }
    if (threadIdx.x == 0) {
      a.rowToken[r] = t;
      a.rowTarget[r] = r < valid ? a.target[t] : -1;
    }
    if (a.dHidden && r >= whole)
      for (int c = threadIdx.x; c < a.D; c += 256) a.dHidden[(long long)t * a.D + c] = 0;
  }
}

// ------------------------------------------------------------- host side
// Rows of the vocabulary taken at a time: a piece of the gradient factors of
// about 256 MB, so that the fp32 sums of dH, read and written once a
// piece, stay a small part of the traffic.
constexpr size_t kPieceBytes = (size_t)256 << 20;
size_t piece_rows(size_t T, size_t V) {  // T: packed rows
  const size_t fit = kPieceBytes / (2 * T) / kBN * kBN;
  return std::min(up(V, kBN), std::max<size_t>(fit, kBN));
}

struct XentPlan {
  bool grads, kept, padHidden, padWeight;
  int partCols;
  // rows: of every buffer of packed tokens; at least T up to whole slices of
  // kTileK, the last row that a kernel stores to
  size_t T, D, V, Dp, rows, nParts, piece, nPieces, sumLd;
  // offsets into the workspace
  size_t state, target, token, skipped, rowToken, rowTarget, softmax, targetLogit, parts, hidden,
      weight, packed, factors, sum, bytes;
};

// `kept`: the gradients' exponentials are kept (where the rule allows it).
bool make_plan(const void* hidden, size_t hiddenStride, const void* weight, size_t weightStride,
               size_t T, size_t D, size_t V, int dtype, bool grads, bool kept, XentPlan* p) {
  constexpr int sms = 152;  // (the workspace's size is asked for without a device, too)
  if ((dtype != VR_FLOAT16 && dtype != VR_BFLOAT16) || T > (1u << 30) || D < 1 || D > (1u << 24) ||
      V < 1 || V > (1u << 30) || hiddenStride < D || weightStride < D ||
      hiddenStride > (1ull << 32) || weightStride > (1ull << 32))
    return false;
  *p = XentPlan{};
  p->grads = grads;
  p->T = T, p->D = D, p->V = V;
  // a packed copy of the hidden states serves the gradients
  p->padHidden = !grads && !packed_rows(hidden, hiddenStride);
  p->padWeight = !packed_rows(weight, weightStride);
  p->Dp = up(D, 16);  // whole 32-byte sectors: rows that straddle them cost a product a fifth
  p->rows = grads ? up(T + kTileK, kTileM) : T;
  // (the rows of the launch: T, or the packed rows' upper bound)
  p->partCols = (grads ? T + kTileK : T) <= kTileM && up(V, kBN) / kBN <= (size_t)sms / 2
                    ? kPartCols / 2
                    : kPartCols;
  p->nParts = up(V, 4 * (size_t)p->partCols) / p->partCols;
  p->kept = grads && kept && (T <= D || 2 * p->rows * up(V, kBN) <= kPieceBytes);
  p->piece = p->kept ? up(V, kBN) : piece_rows(p->rows, V);
  p->nPieces = (V + p->piece - 1) / p->piece;
  p->sumLd = up(D, 32);
  size_t at = 0;
  auto take = [&at](size_t n) {
    const size_t here = at;
    at += op_round(n);
    return here;
  };
  p->state = take(sizeof(XentState));
  p->target = take(T * 4);
  p->token = take(T * 4);
  p->skipped = take(T * 4);
  p->softmax = take(p->rows * sizeof(float2));
  p->targetLogit = take(p->rows * 4);
  p->parts = take(p->rows * p->nParts * sizeof(float2));
  p->hidden = p->padHidden ? take(T * p->Dp * 2) : 0;
  p->weight = p->padWeight ? take(V * p->Dp * 2) : 0;
  if (grads) {
    p->rowToken = take(p->rows * 4);
    p->rowTarget = take(p->rows * 4);
    p->packed = take(p->rows * p->Dp * 2);
    p->factors = take(p->rows * p->piece * 2);
    p->sum = p->nPieces > 1 ? take(p->rows * p->sumLd * 4) : 0;
  }
  p->bytes = at + kOpSlack;
  return true;
}

// One product; pairs of CTAs where the rows fill them.  CHUNK > 0: sums in
// chunks, which one chunk or less does not need; LONG: in long chunks, sums of
// more than kLongSum.
template <typename T, bool AMN, bool BMN, int CHUNK, bool SPLIT, class Epi, bool LONG = false>
vr_result_t product(const OpDevice& dev, const void* a, size_t aLd, const void* b, size_t bLd,
                    size_t M, size_t N, size_t K, const int* dynM, const int* dynK,
                    typename Epi::Args& epi, void* stream, bool narrow = false) {
  const Operand oa = {a, nullptr, aLd}, ob = {b, nullptr, bLd};
  const GemmSize z = {M, N, K, 1, false};
  const bool few = M <= kTileM;
  constexpr int kLong = LONG ? kLongChunk : 0;
#define VR_PRODUCT(C, PAIR, SHARED, SHARES)                                             \
  return gemm_launch<T, kBN, 1, AMN, BMN, C, PAIR, SHARED, Epi>(dev, oa, ob, z, dynM, dynK, \
                                                                epi, SHARES, stream)
  if constexpr (CHUNK > 0) {
    if (narrow && K > kFewRowsChunk * kTileK)
      return gemm_launch<T, 128, 1, AMN, BMN, kFewRowsChunk, false, false, Epi>(
          dev, oa, ob, z, dynM, dynK, epi, 1, stream);
    if (narrow)
      return gemm_launch<T, 128, 1, AMN, BMN, 0, false, false, Epi>(dev, oa, ob, z, dynM, dynK,
                                                                    epi, 1, stream);
  }
  if constexpr (SPLIT) {
    static_assert(CHUNK == 0, "shares are summed in one piece");
    // By the measured times: a slice of 64 k takes 0.31 us on a 256-wide tile
    // of a pair (single CTA 0.33), 0.167 (0.205) on a 128-wide one, a third
    // more where the weight's rows straddle sectors; 36 clusters of four CTAs
    // and 15 of eight are resident at a time (16 are let in: some are empty
    // where tokens are ignored), and a second round of clusters starts slowly;
    // joining s shares takes about s + 2 us.
    const double slices = (double)((K + kTileK - 1) / kTileK);
    const bool odd = bLd % 16 != 0;
    double best = 0;
    int shares = 1;
    bool wide = true;
    auto offer = [&](bool w, int s, size_t tiles, double slice) {
      const int ctas = (few ? 1 : 2) * s;
      const size_t room = ctas > 4 ? 16 : ctas > 2 ? 36 : (size_t)(dev.sms / ctas);
      if (s > 1 && tiles > room) return;
      const double t = (double)((tiles + room - 1) / room) * std::ceil(slices / s) * slice +
                       (s > 1 ? s + 2 : 0);
      if (s == 1 || t < best) best = t, shares = s, wide = w;
    };
    if (few) offer(true, 1, gemm_tiles<kBN, false>(z), 0.33);
    else offer(true, 1, gemm_tiles<kBN, true>(z), 0.31);
    for (int s = 2; s <= (few ? 8 : 4) && s <= slices; s *= 2) {
      if (few) {
        offer(true, s, gemm_tiles<kBN, false>(z), 0.33);
        offer(false, s, gemm_tiles<128, false>(z), 0.205);
      } else {
        offer(true, s, gemm_tiles<kBN, true>(z), odd ? 0.38 : 0.31);
        offer(false, s, gemm_tiles<128, true>(z), odd ? 0.23 : 0.167);
      }
    }
#define VR_SHARED(C, BN, PAIR)                                                                \
  return gemm_launch<T, BN, 1, AMN, BMN, C, PAIR, true, Epi>(dev, oa, ob, z, dynM, dynK, epi, \
                                                             shares, stream)
    if constexpr (kLong > 0) {
      if (shares > 1 && K > kLongSum<T> * shares) {
        if (few && wide) VR_SHARED(kLong, kBN, false);
        if (few) VR_SHARED(kLong, 128, false);
        if (wide) VR_SHARED(kLong, kBN, true);
        VR_SHARED(kLong, 128, true);
      }
    }
    if (shares > 1) {
      if (few && wide) VR_SHARED(0, kBN, false);
      if (few) VR_SHARED(0, 128, false);
      if (wide) VR_SHARED(0, kBN, true);
      VR_SHARED(0, 128, true);
    }
#undef VR_SHARED
  }
  if constexpr (CHUNK > 0) {
    if (few && K > kFewRowsChunk * kTileK) VR_PRODUCT(kFewRowsChunk, false, false, 1);
    if (!few && K > CHUNK * kTileK) VR_PRODUCT(CHUNK, true, false, 1);
  }
  if constexpr (kLong > 0) {
    if (few && K > kLongSum<T>) VR_PRODUCT(kLong, false, false, 1);
    if (K > kLongSum<T>) VR_PRODUCT(kLong, true, false, 1);
  }
  if (few) VR_PRODUCT(0, false, false, 1);
  VR_PRODUCT(0, true, false, 1);
#undef VR_PRODUCT
}

template <typename T>
vr_result_t run(const XentPlan& p, const OpDevice& dev, const void* hidden, size_t hiddenStride,
                const void* weight, size_t weightStride, const long long* targets,
                long long ignoreIndex, int mean, float gradScale, float* losses, float* lse,
                float* loss, void* dHidden, void* dWeight, char* w, void* stream) {
  XentState* state = reinterpret_cast<XentState*>(w + p.state);
  auto ints = [w](size_t at) { return reinterpret_cast<int*>(w + at); };
  int *target = ints(p.target), *token = ints(p.token), *skipped = ints(p.skipped);
  float2* softmax = reinterpret_cast<float2*>(w + p.softmax);
  float* targetLogit = reinterpret_cast<float*>(w + p.targetLogit);
  float2* parts = reinterpret_cast<float2*>(w + p.parts);
  uint16_t* packed = reinterpret_cast<uint16_t*>(w + p.packed);
  T* factors = reinterpret_cast<T*>(w + p.factors);
  vr_result_t e;
  // The loss alone reads the caller's targets where they are.
  Targets rowTarget = {nullptr, targets, ignoreIndex, (int)p.V};
  if (p.grads) {
    PrepArgs a = {targets,   ignoreIndex, (int)p.T, (int)p.V, mean,  gradScale,
                  kShift<T>, target,      token,    skipped,  state, dev.status};
    void* args[] = {&a};
    if ((e = op_launch((const void*)xent_prep_kernel, dim3(1), dim3(1024), args, 0, stream)) !=
        VR_SUCCESS)
      return e;
  }
  auto pad = [&](const void** src, size_t* stride, size_t rows, size_t at) -> vr_result_t {
    PadArgs a = {static_cast<const uint16_t*>(*src), (long long)*stride, (long long)rows,
                 (int)p.D, (int)p.Dp, reinterpret_cast<uint16_t*>(w + at)};
    void* args[] = {&a};
    *src = w + at;
    *stride = p.Dp;
    return op_launch((const void*)pad_kernel,
                     dim3((unsigned)std::min<size_t>((rows + 7) / 8, (size_t)dev.sms * 8)),
                     dim3(256), args, 0, stream);
  };
  if (p.T && p.padHidden && (e = pad(&hidden, &hiddenStride, p.T, p.hidden)) != VR_SUCCESS) return e;
  if (p.T && p.padWeight && (e = pad(&weight, &weightStride, p.V, p.weight)) != VR_SUCCESS) return e;
  if (p.T && p.grads) {
    PackArgs a = {static_cast<const uint16_t*>(hidden), (long long)hiddenStride, (int)p.T,
                  (int)p.D, (int)p.Dp, p.Dp == p.D && packed_rows(hidden, hiddenStride), target,
                  token, skipped, state, packed, ints(p.rowToken), ints(p.rowTarget),
                  static_cast<uint16_t*>(dHidden)};
    void* args[] = {&a};
    if ((e = op_launch((const void*)xent_pack_kernel,
                       dim3((unsigned)std::min<size_t>(p.T + kTileK, (size_t)dev.sms * 8)),
                       dim3(256), args, 0, stream)) != VR_SUCCESS)
      return e;
    hidden = packed;
    hiddenStride = p.Dp;
    rowTarget.of = ints(p.rowTarget);
  }
  if (p.T) {
    // rows: an upper bound where they are packed, their number is on the device
    const size_t rows = p.grads ? p.T + kTileK : p.T;
    const int* dynRows = p.grads ? &state->rows : nullptr;
    if (p.kept) {
      typename StatsEpilogue<T, true>::Args epi = {
          rowTarget, targetLogit, parts, (int)p.nParts, factors, (long long)p.piece, state};
      e = product<T, false, false, kStatsChunk, false, StatsEpilogue<T, true>>(
          dev, hidden, hiddenStride, weight, weightStride, rows, p.V, p.D, dynRows, nullptr, epi,
          stream, p.partCols != kPartCols);
    } else {
      typename StatsEpilogue<T, false>::Args epi = {
          rowTarget, targetLogit, parts, (int)p.nParts, nullptr, 0, state};
      e = product<T, false, false, kStatsChunk, false, StatsEpilogue<T, false>>(
          dev, hidden, hiddenStride, weight, weightStride, rows, p.V, p.D, dynRows, nullptr, epi,
          stream, p.partCols != kPartCols);
    }
    if (e != VR_SUCCESS) return e;
  }
  {
    const size_t rows = !p.T ? 0 : p.grads ? p.T + kTileK : p.T;
    JoinArgs a = {parts,
                  (int)p.nParts,
                  (int)p.T,
                  p.T && p.grads ? ints(p.rowToken) : nullptr,
                  p.grads ? state : nullptr,
                  rowTarget,
                  mean,
                  targetLogit,
                  softmax,
                  lse,
                  losses,
                  loss,
                  dev.status};
    void* args[] = {&a};
    // Few rows: one CTA joins them and sums the loss, a launch less.
    if (rows <= 128) {
      e = op_launch((const void*)xent_join_kernel<true>, dim3(1), dim3(1024), args, 0, stream);
    } else {
      e = op_launch((const void*)xent_join_kernel<false>,
                    dim3((unsigned)std::min<size_t>((rows + 7) / 8, (size_t)dev.sms * 8)),
                    dim3(256), args, 0, stream);
      if (e == VR_SUCCESS)
        e = op_launch((const void*)xent_loss_kernel, dim3(1), dim3(1024), args, 0, stream);
    }
    if (e != VR_SUCCESS) return e;
  }
  if (!p.grads) return VR_SUCCESS;
  if (!p.T) {
    if (dWeight && cudaMemsetAsync(dWeight, 0, p.V * p.D * 2, (cudaStream_t)stream) != cudaSuccess)
      return VR_ERR_CUDA;
    return VR_SUCCESS;
  }
  if (p.kept) {
    KeptArgs<T> a = {factors, (long long)p.piece, parts, (int)p.nParts, p.partCols, (int)p.V, softmax,
                     rowTarget.of, targetLogit, state};
    void* args[] = {&a};
    const size_t columns = 256 * kKeptUnits * 8;
    if ((e = op_launch((const void*)xent_kept_kernel<T>,
                       dim3((unsigned)((p.V + columns - 1) / columns),
                            (unsigned)std::min<size_t>(p.T + kTileK, 32768)),
                       dim3(256), args, 0, stream)) != VR_SUCCESS)
      return e;
  }
  auto aligned = [&](const void* out) {  // of every row of it
    const uintptr_t bits = (uintptr_t)out | (uintptr_t)(2 * p.D);
    return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 2;
  };
  const int alignH = aligned(dHidden), alignW = aligned(dWeight);
  const bool viaPad = dWeight && p.padWeight && alignW == 2;
  for (size_t i = 0; i < p.nPieces; ++i) {
    const size_t v0 = i * p.piece, rows = std::min(p.piece, p.V - v0);
    const T* wPiece = static_cast<const T*>(weight) + v0 * weightStride;
    if (!p.kept) {
      typename FactorEpilogue<T>::Args fa = {rowTarget.of, targetLogit, softmax, factors,
                                             (long long)p.piece, (int)v0};
      if ((e = product<T, false, false, 0, false, FactorEpilogue<T>>(
               dev, packed, p.Dp, wPiece, weightStride, p.T, rows, p.D, &state->valid, nullptr, fa,
               stream)) != VR_SUCCESS)
        return e;
    }
    if (dHidden) {
      typename HiddenEpilogue<T>::Args ha = {
          reinterpret_cast<float*>(w + p.sum), (long long)p.sumLd, static_cast<T*>(dHidden), token,
          state, i == 0, i + 1 == p.nPieces, alignH};
      if ((e = product<T, false, true, 0, true, HiddenEpilogue<T>, true>(
               dev, factors, p.piece, wPiece, weightStride, p.T, p.D, rows, &state->valid, nullptr,
               ha, stream)) != VR_SUCCESS)
        return e;
    }
    if (dWeight) {
      // Rows that are no 16-byte units: into the padded weight's rows, which
      // this piece's products have read, and from there in a pass of its own
      // (stored element by element, 32 rows at a time, they took three times
      // as long as everything else).
      T* out = viaPad ? static_cast<T*>(const_cast<void*>(weight)) + v0 * p.Dp
                      : static_cast<T*>(dWeight) + v0 * p.D;
      const size_t ld = viaPad ? p.Dp : p.D;
      if (p.T <= kTilesMostTokens && !viaPad && alignW == 16) {
        typename WeightTilesEpilogue<T>::Args wa = {};
        wa.aux.nOut = 1;
        wa.state = state;
        if ((e = gemm_operand(&wa.aux.out[0], out, std::is_same<T, __nv_bfloat16>::value, p.D, rows,
                              1, ld * 2, ld * 2 * rows, kTileM, kAuxCols)) != VR_SUCCESS)
          return e;
        e = product<T, true, true, 0, false, WeightTilesEpilogue<T>>(
            dev, factors, p.piece, packed, p.Dp, rows, p.D, p.rows, nullptr, &state->valid, wa,
            stream);
      } else {
        typename WeightEpilogue<T>::Args wa = {out, (long long)ld, state, viaPad ? 32 : alignW};
        e = product<T, true, true, 0, false, WeightEpilogue<T>, true>(
            dev, factors, p.piece, packed, p.Dp, rows, p.D, p.rows, nullptr, &state->valid, wa,
            stream);
      }
      if (e != VR_SUCCESS) return e;
    }
  }
  if (viaPad) {
    PadArgs a = {static_cast<const uint16_t*>(weight), 0, (long long)p.V, (int)p.D, (int)p.Dp,
                 static_cast<uint16_t*>(dWeight)};
    void* args[] = {&a};
    return op_launch((const void*)unpad_kernel,
                     dim3((unsigned)std::min<size_t>((p.V + 7) / 8, (size_t)dev.sms * 8)),
                     dim3(256), args, 0, stream);
  }
  return VR_SUCCESS;
}

}  // namespace
}  // namespace vr

using namespace vr;

extern "C" {

vr_result_t vr_linear_xent_workspace_bytes(const void* hidden, size_t hiddenStride,
                                           const void* weight, size_t weightStride, size_t tokens,
                                           size_t dim, size_t vocab, vr_dtype_t dtype, int grads,
                                           size_t* bytes) {
  XentPlan p = {}, q = {};
  auto plan = [&](bool kept, XentPlan* to) {
    return make_plan(hidden, hiddenStride, weight, weightStride, tokens, dim, vocab, dtype,
                     grads != 0, kept, to);
  };
  if (!bytes || grads < 0 || grads > 2 || !plan(true, &p) || !plan(false, &q))
    return VR_ERR_INVALID_ARGUMENT;
  // a little over one piece, the sums of the pieces take more than keeping all
  *bytes = grads == 2 ? std::min(p.bytes, q.bytes) : p.bytes;
  return VR_SUCCESS;
}

vr_result_t vr_linear_xent(const void* hidden, size_t hiddenStride, const void* weight,
                           size_t weightStride, const long long* targets, size_t tokens,
                           size_t dim, size_t vocab, vr_dtype_t dtype, long long ignoreIndex,
                           int mean, float gradScale, float* losses, float* lse, float* loss,
                           void* dHidden, void* dWeight, void* workspace, size_t workspaceBytes,
                           void* stream) {
  XentPlan p = {};
  const bool grads = dHidden || dWeight;
  auto plan = [&](bool kept) {
    return make_plan(hidden, hiddenStride, weight, weightStride, tokens, dim, vocab, dtype, grads,
                     kept, &p);
  };
  if (!plan(true) || (workspaceBytes < p.bytes && !plan(false)) ||
      !weight || !loss || !workspace || (tokens && (!hidden || !targets || !losses || !lse)) ||
      workspaceBytes < p.bytes || ((uintptr_t)workspace & 15) || ((uintptr_t)targets & 7) ||
      (((uintptr_t)losses | (uintptr_t)lse | (uintptr_t)loss) & 3) ||
      (((uintptr_t)hidden | (uintptr_t)weight | (uintptr_t)dHidden | (uintptr_t)dWeight) & 1))
    return VR_ERR_INVALID_ARGUMENT;
  OpBuffer buf[9] = {
      {hidden, tokens, dim * 2, hiddenStride * 2, false},
      {weight, vocab, dim * 2, weightStride * 2, false},
      {targets, 1, tokens * 8, tokens * 8, false},
      {losses, 1, tokens * 4, tokens * 4, true},
      {lse, 1, tokens * 4, tokens * 4, true},
      {loss, 1, 4, 4, true},
      {workspace, 1, workspaceBytes, workspaceBytes, true},
  };
  int n = 7;
  if (dHidden) buf[n++] = {dHidden, 1, tokens * dim * 2, tokens * dim * 2, true};
  if (dWeight) buf[n++] = {dWeight, 1, vocab * dim * 2, vocab * dim * 2, true};
  if (!op_buffers_ok(buf, n)) return VR_ERR_INVALID_ARGUMENT;
  OpDevice dev;
  vr_result_t e = op_device(&dev);
  if (e != VR_SUCCESS || (e = op_reachable(buf, n, dev.device)) != VR_SUCCESS) return e;
  char* w = op_workspace(workspace);
  return dtype == VR_BFLOAT16
             ? run<__nv_bfloat16>(p, dev, hidden, hiddenStride, weight, weightStride, targets,
                                  ignoreIndex, mean, gradScale, losses, lse, loss, dHidden, dWeight,
                                  w, stream)
             : run<__half>(p, dev, hidden, hiddenStride, weight, weightStride, targets, ignoreIndex,
                           mean, gradScale, losses, lse, loss, dHidden, dWeight, w, stream);
}

}  // extern "C"
