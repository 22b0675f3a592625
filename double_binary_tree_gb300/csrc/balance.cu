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
// from the stored log sum and writes its gradients.  A call whose tokens fit
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
#include <algorithm>
#include <climits>
#include <cstdint>

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
  unsigned long long divTokens;  // t / tokens = high 64 bits of divTokens * t (0: tokens = 1)
  long long stride;  // elements between rows
  long long total;   // tokens of all ranks
  int E, topK, ctas;
  float coef, gradScale;
  float* loss;
  int* counts;
  // workspace
  float* lse;       // [total]; +inf: the token does not count
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
  if constexpr (G == 32) return __reduce_max_sync(0xffffffffu, v);
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  if constexpr (G == 32) return __reduce_min_sync(0xffffffffu, v);
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int G>
__device__ __forceinline__ float group_maxf(float v) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Logit j of chunk c of lane l: expert (c G + l) VEC + j.
template <int VEC, int G>
__device__ __forceinline__ int expert_of(int c, int l, int j) {
  return (c * G + l) * VEC + j;
}

// A row's logits as loaded; absent experts are -inf when they are widened.
template <typename T, int VEC, int CHUNKS>
struct RawRow {
  typename Select<(VEC > 1), uint4, typename Ty<T>::Bits>::type q[CHUNKS];
};
struct Place {
  int rank;
  long long row;
};
__device__ __forceinline__ Place place_of(const BalanceArgs& a, long long t) {
  Place p;
  p.rank = a.divTokens ? (int)__umul64hi(a.divTokens, (unsigned long long)t) : (int)t;
  p.row = t - (long long)p.rank * a.tokens;
  return p;
}
template <typename T, int VEC, int CHUNKS, int G>
__device__ __forceinline__ RawRow<T, VEC, CHUNKS> load_row(const BalanceArgs& a, const Place& at,
                                                           int l) {
  using Bits = typename Ty<T>::Bits;
  const Bits* p = static_cast<const Bits*>(a.logits[at.rank]) + at.row * a.stride;
  RawRow<T, VEC, CHUNKS> r = {};
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int e0 = expert_of<VEC, G>(c, l, 0);  // with VEC > 1, E is a multiple of VEC
    if (e0 < a.E)
      r.q[c] = *reinterpret_cast<const typename Select<(VEC > 1), uint4, Bits>::type*>(p + e0);
  }
  return r;
}
template <typename T, int VEC, int CHUNKS, int G>
__device__ __forceinline__ typename Ty<T>::Bits raw_bits(const RawRow<T, VEC, CHUNKS>& r, int i) {
  return reinterpret_cast<const typename Ty<T>::Bits*>(&r.q[i / VEC])[i % VEC];
}
template <typename T, int VEC, int CHUNKS, int G>
__device__ __forceinline__ float raw_value(const BalanceArgs& a, const RawRow<T, VEC, CHUNKS>& r,
                                           int l, int i) {
  return expert_of<VEC, G>(i / VEC, l, i % VEC) < a.E
             ? Ty<T>::widen(raw_bits<T, VEC, CHUNKS, G>(r, i))
             : -INFINITY;
}

// The first pass of one CTA: sAcc and sCount get its sums, validOut its
// tokens that count.
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
  // group without a token left repeats the last one and discards it.
  const long long step = (long long)gridDim.x * GROUPS;
  const int inWarp = group % (32 / G);
  const long long first = (long long)blockIdx.x * GROUPS + (group - inWarp);
  auto clamp = [&](long long t) { return t < a.total ? t : a.total - 1; };
  RawRow<T, VEC, CHUNKS> next = {};
  if (first < a.total) next = load_row<T, VEC, CHUNKS, G>(a, place_of(a, clamp(first + inWarp)), l);
  for (long long w = first; w < a.total; w += step) {
    const bool real = w + inWarp < a.total;
    const long long t = clamp(w + inWarp);
    const Place at = place_of(a, t);
    const RawRow<T, VEC, CHUNKS> raw = next;
    if (w + step < a.total)
      next = load_row<T, VEC, CHUNKS, G>(a, place_of(a, clamp(w + step + inWarp)), l);
    const bool kept = !a.mask[at.rank] || a.mask[at.rank][at.row] != 0;

    // softmax statistics in fp32
    float p[VPL], top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = raw_value<T, VEC, CHUNKS, G>(a, raw, l, i);
      top = fmaxf(top, p[i]);
      nan |= p[i] != p[i];
    }
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = expert_of<VEC, G>(i / VEC, l, i % VEC);
      if (PACKED) {
        // 16-bit order key above the complement of the index
        const uint32_t b = raw_bits<T, VEC, CHUNKS, G>(raw, i);
        uint32_t k = b & 0x8000u ? b ^ 0xffffu : b | 0x8000u;
        if (b == 0x8000u) k = 0x8000u;  // -0 as +0
        if (p[i] != p[i]) k = 0xffffu;
        key[i] = e < a.E ? k << 16 | (0xffffu - (uint32_t)e) : 0u;
      } else {
        key[i] = e < a.E ? order_key(p[i]) : 0u;
      }
    }
    top = group_maxf<G>(top);
    nan = __ballot_sync(0xffffffffu, nan) & ((G == 32 ? 0xffffffffu : (1u << (G % 32)) - 1)
                                             << (G == 32 ? 0 : inWarp * G));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = __expf(p[i] - top);
      sum += p[i];
    }
    sum = group_sum<G>(sum);
    // a row whose logits are all -inf has no softmax: it does not count
    const bool live = real && kept && (nan || top != -INFINITY);
    if (live) {
      const float inv = __fdividef(1.0f, sum);
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = fmaf(p[i], inv, acc[i]);
      valid += l == 0;
    }
    if (real && l == 0) a.lse[t] = live ? top + __logf(sum) : INFINITY;

    // topK rounds: the largest key left, the lowest index of equals
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
    int mine = -1;
    for (int r = 0; r < a.topK; ++r) {
      uint32_t at32, best = key[0];
      if (!SORTED) {
#pragma unroll
        for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
      }
      best = group_max<G>(best);
      if (SORTED) {
        const bool won = key[0] == best;
#pragma unroll
        for (int i = 0; i + 1 < VPL; ++i) key[i] = won ? key[i + 1] : key[i];
        if (won) key[VPL - 1] = 0u;
      } else if (PACKED) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (key[i] == best) key[i] = 0u;
      }
      if (PACKED) {
        at32 = 0xffffu - (best & 0xffffu);
      } else {
        at32 = 0xffffffffu;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
          if (key[i] == best) at32 = (uint32_t)expert_of<VEC, G>(i / VEC, l, i % VEC);
        at32 = group_min<G>(at32);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if ((uint32_t)expert_of<VEC, G>(i / VEC, l, i % VEC) == at32) key[i] = 0u;
      }
      if (l == r % G) mine = (int)at32;
      if (r % G == G - 1 || r == a.topK - 1) {
        if (real && l <= r % G) {
          if (live) atomicAdd(&sCount[mine], 1);
          int* out = a.chosen[at.rank];
          if (out) out[at.row * a.topK + (r - r % G) + l] = live ? mine : -1;
        }
      }
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

// The second pass of one CTA.
template <typename T, int VEC, int CHUNKS, int G, int THREADS>
__device__ __forceinline__ void grad_pass(const BalanceArgs& a, const float* sShare, float factor) {
  using Bits = typename Ty<T>::Bits;
  constexpr int VPL = VEC * CHUNKS, GROUPS = THREADS / G;
  constexpr int TOK = VPL > 8 ? 1 : 2;  // tokens of a group in flight
  const int l = threadIdx.x % G, group = threadIdx.x / G, inWarp = group % (32 / G);
  float f[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = expert_of<VEC, G>(i / VEC, l, i % VEC);
    f[i] = e < a.E ? sShare[e] : 0.0f;
  }
  const long long step = (long long)gridDim.x * GROUPS;
  const long long first = (long long)blockIdx.x * GROUPS + (group - inWarp);
  for (long long w0 = first; w0 < a.total; w0 += TOK * step) {
    RawRow<T, VEC, CHUNKS> raw[TOK];
    float lse[TOK];
    Place at[TOK];
    bool real[TOK];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
      const long long want = w0 + k * step + inWarp;
      real[k] = want < a.total;
      const long long t = real[k] ? want : a.total - 1;
      at[k] = place_of(a, t);
      raw[k] = load_row<T, VEC, CHUNKS, G>(a, at[k], l);
      lse[k] = a.lse[t];
    }
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
      const bool live = lse[k] != INFINITY;
      float x[VPL], dot = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float v = raw_value<T, VEC, CHUNKS, G>(a, raw[k], l, i);
        x[i] = live ? __expf(v - lse[k]) : 0.0f;
        dot = fmaf(f[i], x[i], dot);
      }
      dot = group_sum<G>(dot);
      if (!real[k]) continue;
      Bits* out = static_cast<Bits*>(a.dlogits[at[k].rank]) + at[k].row * a.stride;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int e0 = expert_of<VEC, G>(c, l, 0);
        if (e0 >= a.E) continue;
        RawRow<T, VEC, 1> r;
        Bits* b = reinterpret_cast<Bits*>(&r.q[0]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int i = c * VEC + j;
          b[j] = Ty<T>::narrow(live ? factor * x[i] * (f[i] - dot) : 0.0f);
        }
        *reinterpret_cast<typename Select<(VEC > 1), uint4, Bits>::type*>(out + e0) = r.q[0];
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
  return op_round((size_t)R * tokens * 4) + 2 * part + op_round(kMostCtas * 4);
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
  if (e != VR_SUCCESS) return e;
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
  a.lse = reinterpret_cast<float*>(w);
  w += op_round((size_t)R * tokens * 4);
  a.probPart = reinterpret_cast<float*>(w);
  a.countPart = reinterpret_cast<int*>(w + part);
  a.validPart = reinterpret_cast<int*>(w + 2 * part);
  a.divTokens = a.tokens > 1 ? ~0ull / (unsigned long long)a.tokens + 1 : 0ull;
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
