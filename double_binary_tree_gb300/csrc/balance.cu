// Balance loss of R ranks' expert routers (vr_balance_loss).
//
//   p_t = softmax(x_t); c_e = number of tokens that choose expert e among
//   their topK; N valid tokens over all ranks; f_e = c_e / (N topK);
//   P_e = sum_t p_te / N;  L = coef E sum_e f_e P_e
//   dL/dx_te = coef E / N * p_te (f_e - sum_j f_j p_tj)   (f held constant)
//
// f needs every token before the first gradient can be written, so the
// logits are read twice: balance_stats_kernel chooses the experts and sums
// the probabilities and counts of each CTA; every CTA of balance_grad_kernel
// first adds up the CTAs' sums in CTA order (the same bits everywhere and on
// every run; less than the launch of a kernel of its own), then recomputes p
// from the stored maximum and sum and writes its gradients.  A call whose tokens fit
// one CTA twice over runs all of it in one launch (balance_small_kernel).
//
// A token is held by a group of G lanes, VPL logits per lane in registers
// (one 16-byte load per VEC of them, the next tokens' loads in flight).  The
// lanes keep the probability sums of their own experts in registers over all
// tokens the group visits, so the only traffic of the sums is one row per CTA
// at the end.  What bounds the first pass is the choice: topK rounds of a
// warp-wide maximum.  16-bit logits carry their index in the low half of the
// compared word, so a round is one reduction, and with 8 logits a lane they
// are sorted once per lane, so a round looks at one word per lane.
//
// Measured on GB300, 8 ranks x 16384 tokens x 256 experts, topK 8, bf16 (138 MB,
// 21 us at the copy bandwidth): 63 us for the first pass, bound by the integer
// instructions of the choice (about 400 instructions a token, issued in 75 %
// of the cycles), 29 us for the second, near its traffic.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.h"
#include "fold.cuh"
#include "ops.h"

namespace vr {
namespace {

constexpr int kMaxExperts = 1024, kMaxTopK = 32;
constexpr int kAcc = 8192;  // floats of the CTA's probability sums in shared memory

struct BalanceArgs {
  const void* logits[kMaxRanks];
  const unsigned char* mask[kMaxRanks];
  int* chosen[kMaxRanks];
  void* dlogits[kMaxRanks];
  long long tokens;  // per rank
  long long stride;  // elements between rows
  long long total;   // tokens of all ranks
  int E, topK, ctas;
  float coef, gradScale;
  float* loss;
  int* counts;
  // workspace
  // [total] maximum and reciprocal sum of exponentials (apart: joined as a log
  // sum, a row at the type's lowest value would lose the sum); (0, 0): the
  // token does not count
  float2* softmax;
  float* probPart;  // [ctas][E]
  int* countPart;   // [ctas][E]
  int* validPart;   // [ctas]
};

// Order-preserving key of a logit: larger key, larger value; NaN above
// +inf, -0 equal to +0.  Never 0, which marks a taken or absent expert.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (G == 32) {
    v = __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  if constexpr (G == 32) {
    v = __reduce_min_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Logit j of chunk c of lane l: expert (c G + l) VEC + j.
template <int VEC, int G>
__device__ __forceinline__ int expert_of(int c, int l, int j) {
  return (c * G + l) * VEC + j;
}

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's logits as loaded.  Absent experts are -inf: no probability, and
// never chosen, since equal logits go to the lower index and topK <= E.
template <typename T, int VEC, int CHUNKS>
struct RawRow {
  using Load = typename Select<(VEC > 1), uint4, typename Ty<T>::Bits>::type;
  Load q[CHUNKS];
};
template <typename T>
__device__ __forceinline__ uint32_t minus_inf() {
  return sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
}
__device__ __forceinline__ void fill(uint4& q, uint32_t v) { q = make_uint4(v, v, v, v); }
__device__ __forceinline__ void fill(uint32_t& q, uint32_t v) { q = v; }
__device__ __forceinline__ void fill(uint16_t& q, uint32_t v) { q = (uint16_t)v; }

// A token: its rank and row, walked in steps without a division.
struct Place {
  long long t, step;
  int rank, row, stepRanks, stepRows;
  __device__ __forceinline__ Place(const BalanceArgs& a, long long first, long long by)
      : t(first), step(by) {
    const unsigned n = (unsigned)a.tokens;  // below 2^31, as t and the step
    rank = (int)((unsigned)first / n);
    row = (int)((unsigned)first % n);
    stepRanks = (int)((unsigned)by / n);
    stepRows = (int)((unsigned)by % n);
  }
  __device__ __forceinline__ void advance(const BalanceArgs& a) {
    t += step;
    rank += stepRanks;
    row += stepRows;  // both below tokens <= 2^31 - 1
    if ((unsigned)row >= (unsigned)a.tokens) row = (int)((unsigned)row - (unsigned)a.tokens), ++rank;
  }
  __device__ __forceinline__ bool real(const BalanceArgs& a) const { return t < a.total; }
};
template <typename T, int VEC, int CHUNKS, int G>
__device__ __forceinline__ RawRow<T, VEC, CHUNKS> load_row(const BalanceArgs& a, const Place& at,
                                                           int l) {
  using Row = RawRow<T, VEC, CHUNKS>;
  Row r;
  const bool real = at.real(a);
  const typename Ty<T>::Bits* p =
      static_cast<const typename Ty<T>::Bits*>(a.logits[real ? at.rank : 0]) + at.row * a.stride;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int e0 = expert_of<VEC, G>(c, l, 0);  // with VEC > 1, E is a multiple of VEC
    fill(r.q[c], minus_inf<T>());
    if (real && e0 < a.E) r.q[c] = *reinterpret_cast<const typename Row::Load*>(p + e0);
  }
  return r;
}
template <typename T, int VEC, int CHUNKS>
__device__ __forceinline__ float raw_value(const RawRow<T, VEC, CHUNKS>& r, int i) {
  return Ty<T>::widen(reinterpret_cast<const typename Ty<T>::Bits*>(&r.q[i / VEC])[i % VEC]);
}
// exp(x - top) of a row's logits: one multiply-add and exp2 each while the
// rounding of top log2 e, which stays in every exponent and cancels in the
// softmax, is small (at most 2^-4 below 2^20; beyond, it would come to
// exponentials of 0 or infinity: 440 at 1e10).  Larger logits, by which a
// router masks, are subtracted first.
template <typename T, int VEC, int CHUNKS>
__device__ __forceinline__ void exponentials(const RawRow<T, VEC, CHUNKS>& r, float top,
                                             float (&p)[VEC * CHUNKS]) {
  if (std::is_same<T, __half>::value || fabsf(top) < 0x1p20f) {
    const float top2 = top * kLog2e;
#pragma unroll
    for (int i = 0; i < VEC * CHUNKS; ++i)
      p[i] = exp2_fast(fmaf(raw_value(r, i), kLog2e, -top2));
  } else {
#pragma unroll
    for (int i = 0; i < VEC * CHUNKS; ++i) p[i] = exp2_fast((raw_value(r, i) - top) * kLog2e);
  }
}
// Two 16-bit logits as order keys.  Adding zero makes -0 +0 and every NaN
// 0x7fff; then a negative value's bits are inverted, a positive one's sign set.
template <typename T>
__device__ __forceinline__ uint32_t order_keys2(uint32_t b) {
  if (std::is_same<T, __half>::value) {
    const __half2 v = __hadd2(*reinterpret_cast<__half2*>(&b), __float2half2_rn(0.0f));
    b = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v =
        __hadd2(*reinterpret_cast<__nv_bfloat162*>(&b), __float2bfloat162_rn(0.0f));
    b = *reinterpret_cast<const uint32_t*>(&v);
  }
  return b ^ (((b >> 15 & 0x00010001u) * 0x7fffu) | 0x80008000u);
}
// The logit that a key stands for.
template <typename T>
__device__ __forceinline__ float key_value(uint32_t k) {
  if (sizeof(T) == 4) return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
  const uint32_t h = k >> 16;
  return Ty<T>::widen((typename Ty<T>::Bits)(h & 0x8000u ? h & 0x7fffu : h ^ 0xffffu));
}

// The first pass of one CTA: sAcc and sCount get its sums, sValid its tokens
// that count.
template <typename T, int VEC, int CHUNKS, int G, int THREADS>
__device__ __forceinline__ void stats_pass(const BalanceArgs& a, float* sAcc, int* sCount,
                                           int* sValid) {
  constexpr int VPL = VEC * CHUNKS, GROUPS = THREADS / G;
  constexpr bool PACKED = sizeof(T) == 2, SORTED = PACKED && VPL == 8;
  static_assert(GROUPS * G * VPL <= kAcc, "probability sums do not fit");
  const int l = threadIdx.x % G, group = threadIdx.x / G;
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  int valid = 0;
  // Whole warps stay in the loop together (the shuffles name all lanes); a
  // group without a token left works on a row of -inf.
  const long long step = (long long)gridDim.x * GROUPS;
  Place at(a, (long long)blockIdx.x * GROUPS + group, step);
  long long warpAt = at.t - group % (32 / G);
  auto kept_of = [&](const Place& p) -> bool {
    const bool real = p.real(a);
    const unsigned char* m = real ? a.mask[p.rank] : nullptr;
    return real && (!m || m[p.row] != 0);
  };
  RawRow<T, VEC, CHUNKS> next = load_row<T, VEC, CHUNKS, G>(a, at, l);
  bool nextKept = kept_of(at);
  for (; warpAt < a.total; warpAt += step) {
    const Place here = at;
    const RawRow<T, VEC, CHUNKS> raw = next;
    const bool kept = nextKept;
    at.advance(a);
    next = load_row<T, VEC, CHUNKS, G>(a, at, l);
    nextKept = kept_of(at);

    uint32_t key[VPL];
    if (PACKED && VEC > 1) {
#pragma unroll
      for (int i = 0; i < VPL; i += 2) {
        const uint32_t k = order_keys2<T>(reinterpret_cast<const uint32_t*>(&raw.q[i / VEC])[i % VEC / 2]);
        const uint32_t e = 0xffffu - (uint32_t)expert_of<VEC, G>(i / VEC, l, i % VEC);
        key[i] = k << 16 | e;
        key[i + 1] = (k & 0xffff0000u) | (e - 1);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const uint32_t e = (uint32_t)expert_of<VEC, G>(i / VEC, l, i % VEC);
        key[i] = PACKED ? order_keys2<T>((uint32_t) * reinterpret_cast<const typename Ty<T>::Bits*>(
                              &raw.q[i])) << 16 | (0xffffu - e)
                        : order_key(raw_value(raw, i));
      }
    }
    if (SORTED) {
      // the lane's words in descending order (19 comparisons)
      constexpr int net[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6},
                                  {5, 7}, {1, 2}, {5, 6}, {0, 4}, {3, 7}, {1, 5}, {2, 6},
                                  {1, 4}, {3, 6}, {2, 4}, {3, 5}, {3, 4}};
#pragma unroll
      for (int c = 0; c < 19; ++c) {
        const uint32_t x = key[net[c][0] % VPL], y = key[net[c][1] % VPL];
        key[net[c][0] % VPL] = max(x, y);
        key[net[c][1] % VPL] = min(x, y);
      }
    }
    auto largest = [&]() {
      uint32_t best = key[0];
      if (!SORTED) {
#pragma unroll
        for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
      }
      return group_max<G>(best);
    };
    uint32_t best = largest();

    // softmax statistics in fp32; the largest key is the maximum (or NaN)
    const float top = key_value<T>(best);
    float p[VPL], sum = 0.0f;
    exponentials(raw, top, p);
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += p[i];
    sum = group_sum<G>(sum);
    // a row whose logits are all -inf has no softmax: it does not count
    const bool live = kept && top != -INFINITY;
    const float inv = __fdividef(1.0f, sum);
    if (live) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = fmaf(p[i], inv, acc[i]);
      valid += l == 0;
    }
    if (here.real(a) && l == 0)
      a.softmax[here.t] = live ? make_float2(top, inv) : make_float2(0.0f, 0.0f);

    // topK rounds: the largest key left, the lowest index of equals.  Lane r of
    // the group keeps round r's.
    auto take = [&](uint32_t& word) {  // what `best` stands for leaves its lane's keys
      if (PACKED) {
        word = best;
        if (SORTED) {
          if (key[0] == best) {
#pragma unroll
            for (int i = 0; i + 1 < VPL; ++i) key[i] = key[i + 1];
            key[VPL - 1] = 0u;
          }
        } else {
#pragma unroll
          for (int i = 0; i < VPL; ++i) key[i] = key[i] == best ? 0u : key[i];
        }
      } else {
        uint32_t chosen = 0xffffffffu;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
          if (key[i] == best) chosen = (uint32_t)expert_of<VEC, G>(i / VEC, l, i % VEC);
        chosen = group_min<G>(chosen);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if ((uint32_t)expert_of<VEC, G>(i / VEC, l, i % VEC) == chosen) key[i] = 0u;
        word = 0xffffu - chosen;
      }
    };
    for (int from = 0;; from += G) {
      const int n = min(a.topK - from, G);
      uint32_t mine = 0;
      for (int r = 0;;) {
        uint32_t word;
        take(word);
        if (l == r) mine = word;
        if (++r == n) break;
        best = largest();
      }
      if (here.real(a) && l < n) {
        const int e = 0xffff - (int)(mine & 0xffffu);
        if (live) atomicAdd(&sCount[e], 1);
        int* out = a.chosen[here.rank];
        if (out) out[(long long)here.row * a.topK + from + l] = live ? e : -1;
      }
      if (from + n == a.topK) break;
      best = largest();
    }
  }
  if (valid) atomicAdd(sValid, valid);
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    sAcc[group * (G * VPL) + expert_of<VEC, G>(i / VEC, l, i % VEC)] = acc[i];
  __syncthreads();
}

template <typename T, int VEC, int CHUNKS, int G, int THREADS>
__global__ void __launch_bounds__(THREADS) balance_stats_kernel(const __grid_constant__ BalanceArgs a) {
  constexpr int VPL = VEC * CHUNKS, GROUPS = THREADS / G;
  __shared__ float sAcc[kAcc];
  __shared__ int sCount[kMaxExperts];
  __shared__ int sValid;
  for (int e = threadIdx.x; e < a.E; e += THREADS) sCount[e] = 0;
  if (threadIdx.x == 0) sValid = 0;
  __syncthreads();
  pdl_launch();
  pdl_wait();
  stats_pass<T, VEC, CHUNKS, G, THREADS>(a, sAcc, sCount, &sValid);
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    float s = 0.0f;
#pragma unroll 8
    for (int g = 0; g < GROUPS; ++g) s += sAcc[g * (G * VPL) + e];
    a.probPart[(long long)blockIdx.x * a.E + e] = s;
    a.countPart[(long long)blockIdx.x * a.E + e] = sCount[e];
  }
  if (threadIdx.x == 0) a.validPart[blockIdx.x] = sValid;
}

// The shares f, the loss and the counts from one sum of p and one count per
// expert (sum(e), count(e)); CTA 0 writes the results.
template <int THREADS, class Sum, class Count>
__device__ __forceinline__ float shares(const BalanceArgs& a, int valid, float* sShare, float* sPart,
                                        Sum sum, Count count) {
  const float perToken = valid ? 1.0f / (float)valid : 0.0f;
  const float perChoice = valid ? 1.0f / ((float)valid * (float)a.topK) : 0.0f;
  float part = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    const int c = count(e);
    const float f = (float)c * perChoice;
    sShare[e] = f;
    part += f * (sum(e) * perToken);
    if (blockIdx.x == 0) a.counts[e] = c;
  }
  part = group_sum<32>(part);
  if (threadIdx.x % 32 == 0) sPart[threadIdx.x / 32] = part;
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < THREADS / 32; ++w) s += sPart[w];
    *a.loss = a.coef * (float)a.E * s;
  }
  return a.coef * (float)a.E * perToken * a.gradScale;
}

// Values rounded to T in the layout of a load.
template <typename T, int VEC>
__device__ __forceinline__ void store_chunk(typename Ty<T>::Bits* out, const float* v) {
  if constexpr (VEC == 8) {
    uint4 q;
    uint32_t* w = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(out) = q;
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    out[0] = Ty<T>::narrow(v[0]);
  }
}

// The second pass of one CTA: dx = p (F - sum F p), F = factor f.
template <typename T, int VEC, int CHUNKS, int G, int THREADS>
__device__ __forceinline__ void grad_pass(const BalanceArgs& a, const float* sShare, float factor) {
  constexpr int VPL = VEC * CHUNKS, GROUPS = THREADS / G;
  constexpr int TOK = VPL > 8 ? 1 : 2;  // tokens of a group in flight
  const int l = threadIdx.x % G, group = threadIdx.x / G;
  float f[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = expert_of<VEC, G>(i / VEC, l, i % VEC);
    f[i] = e < a.E ? factor * sShare[e] : 0.0f;
  }
  const long long step = (long long)gridDim.x * GROUPS;
  Place at(a, (long long)blockIdx.x * GROUPS + group, step);
  for (long long warpAt = at.t - group % (32 / G); warpAt < a.total; warpAt += TOK * step) {
    RawRow<T, VEC, CHUNKS> raw[TOK];
    float2 sm[TOK];
    typename Ty<T>::Bits* out[TOK];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
      raw[k] = load_row<T, VEC, CHUNKS, G>(a, at, l);
      out[k] = nullptr;
      sm[k] = make_float2(0.0f, 0.0f);
      if (at.real(a)) {
        sm[k] = a.softmax[at.t];
        out[k] = static_cast<typename Ty<T>::Bits*>(a.dlogits[at.rank]) + at.row * a.stride;
      }
      at.advance(a);
    }
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
      if (sm[k].y == 0.0f) {  // does not count: whatever it holds, p = 0
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) fill(raw[k].q[c], 0u);
      }
      float x[VPL], dot = 0.0f;
      exponentials(raw[k], sm[k].x, x);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        dot = fmaf(f[i], x[i], dot);
      }
      const float inv = sm[k].y, less = group_sum<G>(dot) * inv * inv;
#pragma unroll
      for (int i = 0; i < VPL; ++i) x[i] *= fmaf(f[i], inv, -less);
      if (!out[k]) continue;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int e0 = expert_of<VEC, G>(c, l, 0);
        if (e0 < a.E) store_chunk<T, VEC>(out[k] + e0, x + c * VEC);
      }
    }
  }
}

template <typename T, int VEC, int CHUNKS, int G, int THREADS>
__global__ void __launch_bounds__(THREADS) balance_grad_kernel(const __grid_constant__ BalanceArgs a) {
  __shared__ float sShare[kMaxExperts];
  __shared__ float sSum[kMaxExperts];
  __shared__ int sCount[kMaxExperts];
  __shared__ float sPart[THREADS / 32];
  __shared__ int sValid;
  pdl_launch();
  pdl_wait();
  // Every CTA adds up all partial sums: the threads of one expert (a power of
  // two of them) a run of CTAs each, joined in order.
  if (threadIdx.x < 32) {
    int n = 0;
    for (int b = threadIdx.x; b < a.ctas; b += 32) n += a.validPart[b];
    n = __reduce_add_sync(0xffffffffu, n);
    if (threadIdx.x == 0) sValid = n;
  }
  __shared__ float sJoin[THREADS];
  __shared__ int sJoinCount[THREADS];
  int width = 32;  // experts side by side
  while (width < a.E && width < THREADS) width *= 2;
  const int ways = THREADS / width, way = threadIdx.x / width;
  const int run = (a.ctas + ways - 1) / ways;
  for (int e0 = 0; e0 < a.E; e0 += width) {
    const int e = e0 + threadIdx.x % width;
    float s = 0.0f;
    int c = 0;
    if (e < a.E) {
      const int b1 = min(a.ctas, (way + 1) * run);
#pragma unroll 8
      for (int b = way * run; b < b1; ++b) {
        s += a.probPart[(long long)b * a.E + e];
        c += a.countPart[(long long)b * a.E + e];
      }
    }
    sJoin[threadIdx.x] = s;
    sJoinCount[threadIdx.x] = c;
    __syncthreads();
    if (threadIdx.x < width && e < a.E) {
      for (int w = 1; w < ways; ++w) {
        s += sJoin[w * width + threadIdx.x];
        c += sJoinCount[w * width + threadIdx.x];
      }
      sSum[e] = s;
      sCount[e] = c;
    }
    __syncthreads();
  }
  const float factor = shares<THREADS>(
      a, sValid, sShare, sPart, [&](int e) { return sSum[e]; }, [&](int e) { return sCount[e]; });
  if (a.dlogits[0]) grad_pass<T, VEC, CHUNKS, G, THREADS>(a, sShare, factor);
}

// Both passes in one CTA.
template <typename T, int VEC, int CHUNKS, int G, int THREADS>
__global__ void __launch_bounds__(THREADS) balance_small_kernel(const __grid_constant__ BalanceArgs a) {
  constexpr int VPL = VEC * CHUNKS, GROUPS = THREADS / G;
  __shared__ float sAcc[kAcc];
  __shared__ float sShare[kMaxExperts];
  __shared__ int sCount[kMaxExperts];
  __shared__ float sPart[THREADS / 32];
  __shared__ int sValid;
  for (int e = threadIdx.x; e < a.E; e += THREADS) sCount[e] = 0;
  if (threadIdx.x == 0) sValid = 0;
  __syncthreads();
  pdl_launch();
  pdl_wait();
  stats_pass<T, VEC, CHUNKS, G, THREADS>(a, sAcc, sCount, &sValid);
  const float factor = shares<THREADS>(
      a, sValid, sShare, sPart,
      [&](int e) {
        float s = 0.0f;
#pragma unroll 8
        for (int g = 0; g < GROUPS; ++g) s += sAcc[g * (G * VPL) + e];
        return s;
      },
      [&](int e) { return sCount[e]; });
  if (a.dlogits[0]) grad_pass<T, VEC, CHUNKS, G, THREADS>(a, sShare, factor);
}

struct BalanceKernels {
  const void *stats, *grad, *small;
  int threads, groups;  // per CTA
};

template <typename T, int VEC, int CHUNKS, int G>
BalanceKernels kernels_of() {
  constexpr int THREADS = VEC * CHUNKS > 8 ? 256 : 1024;
  return {(const void*)balance_stats_kernel<T, VEC, CHUNKS, G, THREADS>,
          (const void*)balance_grad_kernel<T, VEC, CHUNKS, G, THREADS>,
          (const void*)balance_small_kernel<T, VEC, CHUNKS, G, THREADS>, THREADS, THREADS / G};
}

// The smallest layout that holds E experts: 16-byte loads of V logits where
// the rows allow it, else one logit at a time.
template <typename T, int V>
BalanceKernels pick(int E, bool vec) {
  if (vec) {
    if (E <= 64) return kernels_of<T, V, 8 / V, 8>();
    if (E <= 256) return kernels_of<T, V, 8 / V, 32>();
    return kernels_of<T, V, 32 / V, 32>();
  }
  if (E <= 64) return kernels_of<T, 1, 8, 8>();
  if (E <= 256) return kernels_of<T, 1, 8, 32>();
  return kernels_of<T, 1, 32, 32>();
}

int stats_ctas(int sms, long long total, int groups) {
  return (int)std::max(1LL, std::min<long long>(sms, (total + groups - 1) / groups));
}

constexpr int kMostCtas = 256;  // SMs the workspace provides for

bool valid_sizes(int R, size_t tokens, int experts) {
  return R >= 1 && R <= kMaxRanks && experts >= 1 && experts <= kMaxExperts &&
         tokens <= (size_t)INT_MAX / (size_t)R;
}

size_t workspace(int R, size_t tokens, int experts) {
  const size_t part = op_round((size_t)kMostCtas * experts * 4);
  return op_round((size_t)R * tokens * sizeof(float2)) + 2 * part + op_round(kMostCtas * 4);
}

}  // namespace
}  // namespace vr

using namespace vr;

extern "C" {

vr_result_t vr_balance_loss_workspace_bytes(int R, size_t tokens, int experts, size_t* bytes) {
  if (!bytes || !valid_sizes(R, tokens, experts)) return VR_ERR_INVALID_ARGUMENT;
  *bytes = workspace(R, tokens, experts);
  return VR_SUCCESS;
}

vr_result_t vr_balance_loss(const void* const* logits, size_t rowStride,
                            const unsigned char* const* masks, int R, size_t tokens, int experts,
                            int topK, vr_dtype_t dtype, float coef, float gradScale, float* loss,
                            int* counts, int* const* chosen, void* const* dlogits,
                            void* workspaceBuf, size_t workspaceBytes, void* stream) {
  const size_t E = op_elem_size(dtype);
  if (!E || !valid_sizes(R, tokens, experts) || topK < 1 || topK > kMaxTopK || topK > experts ||
      rowStride < (size_t)experts || rowStride > (size_t)LLONG_MAX / 8 / (tokens ? tokens : 1) ||
      !logits || !loss || !counts || !workspaceBuf ||
      workspaceBytes < workspace(R, tokens, experts) || ((uintptr_t)workspaceBuf & 15) ||
      (((uintptr_t)loss | (uintptr_t)counts) & 3))
    return VR_ERR_INVALID_ARGUMENT;
  BalanceArgs a = {};
  OpBuffer buf[4 * kMaxRanks + 3];
  int n = 0;
  const bool grads = dlogits != nullptr;
  uintptr_t align = (uintptr_t)(rowStride * E) | (uintptr_t)((size_t)experts * E);
  for (int r = 0; r < R; ++r) {
    a.logits[r] = logits[r];
    a.mask[r] = masks ? masks[r] : nullptr;
    a.chosen[r] = chosen ? chosen[r] : nullptr;
    a.dlogits[r] = grads ? dlogits[r] : nullptr;
    if (tokens && (!logits[r] || (grads && !dlogits[r]))) return VR_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a.logits[r] | (uintptr_t)a.dlogits[r]) % E || (uintptr_t)a.chosen[r] % 4)
      return VR_ERR_INVALID_ARGUMENT;
    align |= (uintptr_t)a.logits[r] | (uintptr_t)a.dlogits[r];
    buf[n++] = {a.logits[r], tokens, experts * E, rowStride * E, false};
    if (grads) buf[n++] = {a.dlogits[r], tokens, experts * E, rowStride * E, true};
    if (a.mask[r]) buf[n++] = {a.mask[r], 1, tokens, tokens, false};
    if (a.chosen[r]) buf[n++] = {a.chosen[r], 1, tokens * topK * 4, tokens * topK * 4, true};
  }
  buf[n++] = {loss, 1, 4, 4, true};
  buf[n++] = {counts, 1, (size_t)experts * 4, (size_t)experts * 4, true};
  buf[n++] = {workspaceBuf, 1, workspaceBytes, workspaceBytes, true};
  if (!op_buffers_ok(buf, n)) return VR_ERR_INVALID_ARGUMENT;

  OpDevice dev;
  vr_result_t e = op_device(&dev);
  if (e != VR_SUCCESS || (e = op_reachable(buf, n, dev.device)) != VR_SUCCESS) return e;
  const bool vec = (align & 15) == 0;
  const BalanceKernels k = dtype == VR_FLOAT32   ? pick<float, 4>(experts, vec)
                           : dtype == VR_FLOAT16 ? pick<__half, 8>(experts, vec)
                                                 : pick<__nv_bfloat16, 8>(experts, vec);
  a.tokens = (long long)std::max<size_t>(tokens, 1);
  a.stride = (long long)rowStride;
  a.total = (long long)tokens * R;
  a.E = experts;
  a.topK = topK;
  a.coef = coef;
  a.gradScale = gradScale;
  a.loss = loss;
  a.counts = counts;
  a.ctas = stats_ctas(std::min(dev.sms, kMostCtas), a.total, k.groups);
  char* w = static_cast<char*>(workspaceBuf);
  const size_t part = op_round((size_t)kMostCtas * experts * 4);
  a.softmax = reinterpret_cast<float2*>(w);
  w += op_round((size_t)R * tokens * sizeof(float2));
  a.probPart = reinterpret_cast<float*>(w);
  a.countPart = reinterpret_cast<int*>(w + part);
  a.validPart = reinterpret_cast<int*>(w + 2 * part);
  void* args[] = {&a};
  // Two rounds of one CTA's groups: the second launch and its sums cost more
  // than the idle SMs.
  if (a.total <= 2 * k.groups)
    return op_launch(k.small, dim3(1), dim3(k.threads), args, 0, stream);
  if ((e = op_launch(k.stats, dim3(a.ctas), dim3(k.threads), args, 0, stream)) != VR_SUCCESS)
    return e;
  const int grid = grads ? std::max(1, std::min(dev.sms, (int)((a.total + k.groups - 1) / k.groups)))
                         : 1;
  return op_launch(k.grad, dim3(grid), dim3(k.threads), args, 0, stream);
}

}  // extern "C"
