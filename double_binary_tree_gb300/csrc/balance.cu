// Balance loss of R ranks' expert routers (vr_balance_loss).
//
//   p_t = softmax(x_t); c_e = number of tokens that choose expert e among
//   their topK; N valid tokens over all ranks; f_e = c_e / (N topK);
//   P_e = sum_t p_te / N;  L = coef E sum_e f_e P_e
//   dL/dx_te = coef E / N * p_te (f_e - sum_j f_j p_tj)   (f held constant)
//
// f needs every token before the first gradient can be written, so the
// logits are read twice: balance_stats_kernel chooses the experts and sums
// the probabilities and counts of each CTA, balance_finish_kernel adds the
// CTAs' sums in CTA order (the same bits on every run), and
// balance_grad_kernel recomputes p from the stored log sum and writes the
// gradients.
//
// A token is held by a group of G lanes, VPL logits per lane in registers
// (one 16-byte load per VEC of them).  The lanes keep the probability sums
// of their own experts in registers over all tokens the group visits, so the
// only traffic of the sums is one row per CTA at the end.
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
  float* share;     // [E] f, then the gradient's factor
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
  if (G == 32) return __reduce_max_sync(0xffffffffu, v);
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  if (G == 32) return __reduce_min_sync(0xffffffffu, v);
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

// A row's logits into registers; absent experts are -inf.
template <typename T, int VEC, int CHUNKS, int G>
__device__ __forceinline__ void load_row(const BalanceArgs& a, int rank, long long row, int l,
                                         float (&x)[VEC * CHUNKS]) {
  using Bits = typename Ty<T>::Bits;
  const Bits* p = static_cast<const Bits*>(a.logits[rank]) + row * a.stride;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int e0 = expert_of<VEC, G>(c, l, 0);
    if (VEC > 1) {
      uint4 v = {0, 0, 0, 0};
      const bool in = e0 < a.E;  // E is a multiple of VEC here
      if (in) v = *reinterpret_cast<const uint4*>(p + e0);
      const Bits* b = reinterpret_cast<const Bits*>(&v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[c * VEC + j] = in ? Ty<T>::widen(b[j]) : -INFINITY;
    } else {
      x[c] = e0 < a.E ? Ty<T>::widen(p[e0]) : -INFINITY;
    }
  }
}

template <typename T, int VEC, int CHUNKS, int G, int THREADS>
__global__ void __launch_bounds__(THREADS) balance_stats_kernel(const __grid_constant__ BalanceArgs a) {
  constexpr int VPL = VEC * CHUNKS, GROUPS = THREADS / G;
  __shared__ float sAcc[kAcc];
  __shared__ int sCount[kMaxExperts];
  __shared__ int sValid;
  static_assert(GROUPS * G * VPL <= kAcc, "probability sums do not fit");
  for (int e = threadIdx.x; e < a.E; e += THREADS) sCount[e] = 0;
  if (threadIdx.x == 0) sValid = 0;
  __syncthreads();
  pdl_wait();

  const int l = threadIdx.x % G, group = threadIdx.x / G;
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  int valid = 0;
  // Whole warps stay in the loop together (the shuffles name all lanes); a
  // group without a token left repeats the last one and discards it.
  const long long step = (long long)gridDim.x * GROUPS;
  const long long warpFirst = (long long)blockIdx.x * GROUPS + (group - group % (32 / G));
  for (long long w = warpFirst; w < a.total; w += step) {
    const long long want = w + group % (32 / G);
    const bool real = want < a.total;
    const long long t = real ? want : a.total - 1;
    const int rank = (int)(t / a.tokens);
    const long long row = t - rank * a.tokens;
    float x[VPL];
    load_row<T, VEC, CHUNKS, G>(a, rank, row, l, x);
    const bool kept = !a.mask[rank] || a.mask[rank][row] != 0;

    // softmax statistics in fp32
    float top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      top = fmaxf(top, x[i]);
      nan |= x[i] != x[i];
    }
    top = group_maxf<G>(top);
    float p[VPL], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = __expf(x[i] - top);
      sum += p[i];
    }
    sum = group_sum<G>(sum);
    // a row whose logits are all -inf has no softmax: it does not count
    nan = group_max<G>(nan) != 0;
    const bool live = kept && (nan || top != -INFINITY);
    const float inv = live && real ? __fdividef(1.0f, sum) : 0.0f;
    if (live && real) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += p[i] * inv;
      valid += l == 0;
    }
    if (real && l == 0) a.lse[t] = live ? top + __logf(sum) : INFINITY;

    // topK rounds: the largest key left, the lowest index of equals
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = expert_of<VEC, G>(i / VEC, l, i % VEC);
      key[i] = e < a.E ? order_key(x[i]) : 0u;
    }
    int mine = -1;
    for (int r = 0; r < a.topK; ++r) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
      best = group_max<G>(best);
      uint32_t at = 0xffffffffu;
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == best) at = (uint32_t)expert_of<VEC, G>(i / VEC, l, i % VEC);
      at = group_min<G>(at);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if ((uint32_t)expert_of<VEC, G>(i / VEC, l, i % VEC) == at) key[i] = 0u;
      if (l == r % G) mine = (int)at;
      if (r % G == G - 1 || r == a.topK - 1) {
        if (real && l <= r % G) {
          if (live) atomicAdd(&sCount[mine], 1);
          int* out = a.chosen[rank];
          if (out) out[row * a.topK + (r - r % G) + l] = live ? mine : -1;
        }
      }
    }
  }
  if (valid) atomicAdd(&sValid, valid);
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    sAcc[group * (G * VPL) + expert_of<VEC, G>(i / VEC, l, i % VEC)] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    float s = 0.0f;
    for (int g = 0; g < GROUPS; ++g) s += sAcc[g * (G * VPL) + e];
    a.probPart[(long long)blockIdx.x * a.E + e] = s;
    a.countPart[(long long)blockIdx.x * a.E + e] = sCount[e];
  }
  if (threadIdx.x == 0) a.validPart[blockIdx.x] = sValid;
}

// One CTA: the CTAs' sums added in order, the counts, the shares, the loss.
__global__ void __launch_bounds__(1024) balance_finish_kernel(const __grid_constant__ BalanceArgs a) {
  __shared__ float sSum[32];
  __shared__ int sValid;
  pdl_wait();
  if (threadIdx.x == 0) {
    int n = 0;
    for (int b = 0; b < a.ctas; ++b) n += a.validPart[b];
    sValid = n;
  }
  __syncthreads();
  const float n = (float)sValid;
  const float perToken = sValid ? 1.0f / n : 0.0f;
  const float perChoice = sValid ? 1.0f / (n * (float)a.topK) : 0.0f;
  float part = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += 1024) {
    float s = 0.0f;
    int c = 0;
    for (int b = 0; b < a.ctas; ++b) {
      s += a.probPart[(long long)b * a.E + e];
      c += a.countPart[(long long)b * a.E + e];
    }
    a.counts[e] = c;
    const float f = (float)c * perChoice;
    a.share[e] = f;
    part += f * (s * perToken);
  }
  part = group_sum<32>(part);
  if (threadIdx.x % 32 == 0) sSum[threadIdx.x / 32] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < 32; ++w) s += sSum[w];
    *a.loss = a.coef * (float)a.E * s;
    a.share[a.E] = a.coef * (float)a.E * perToken * a.gradScale;
  }
}

template <typename T, int VEC, int CHUNKS, int G, int THREADS>
__global__ void __launch_bounds__(THREADS) balance_grad_kernel(const __grid_constant__ BalanceArgs a) {
  using Bits = typename Ty<T>::Bits;
  constexpr int VPL = VEC * CHUNKS, GROUPS = THREADS / G;
  pdl_wait();
  const int l = threadIdx.x % G, group = threadIdx.x / G;
  float f[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = expert_of<VEC, G>(i / VEC, l, i % VEC);
    f[i] = e < a.E ? a.share[e] : 0.0f;
  }
  const float factor = a.share[a.E];
  const long long step = (long long)gridDim.x * GROUPS;
  const long long warpFirst = (long long)blockIdx.x * GROUPS + (group - group % (32 / G));
  for (long long w = warpFirst; w < a.total; w += step) {
    const long long want = w + group % (32 / G);
    const bool real = want < a.total;
    const long long t = real ? want : a.total - 1;
    const int rank = (int)(t / a.tokens);
    const long long row = t - rank * a.tokens;
    float x[VPL];
    load_row<T, VEC, CHUNKS, G>(a, rank, row, l, x);
    const float lse = a.lse[t];
    const bool live = lse != INFINITY;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      x[i] = live ? __expf(x[i] - lse) : 0.0f;
      dot += f[i] * x[i];
    }
    dot = group_sum<G>(dot);
    if (!real) continue;
    Bits* out = static_cast<Bits*>(a.dlogits[rank]) + row * a.stride;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int e0 = expert_of<VEC, G>(c, l, 0);
      if (e0 >= a.E) continue;
      Bits b[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int i = c * VEC + j;
        b[j] = Ty<T>::narrow(live ? factor * x[i] * (f[i] - dot) : 0.0f);
      }
      if (VEC > 1) {
        uint4 v;
        Bits* d = reinterpret_cast<Bits*>(&v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] = b[j];
        *reinterpret_cast<uint4*>(out + e0) = v;
      } else {
        out[e0] = b[0];
      }
    }
  }
}

struct BalanceKernels {
  const void* stats;
  const void* grad;
  int threads, groups;  // per CTA
};

template <typename T, int VEC, int CHUNKS, int G>
BalanceKernels kernels_of() {
  constexpr int THREADS = VEC * CHUNKS > 8 ? 256 : 1024;
  return {(const void*)balance_stats_kernel<T, VEC, CHUNKS, G, THREADS>,
          (const void*)balance_grad_kernel<T, VEC, CHUNKS, G, 256>, THREADS, THREADS / G};
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
  return op_round((size_t)R * tokens * 4) + 2 * part + op_round(kMostCtas * 4) +
         op_round((experts + 1) * 4);
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
  a.share = reinterpret_cast<float*>(w + 2 * part + op_round(kMostCtas * 4));
  void* args[] = {&a};
  if ((e = op_launch(k.stats, dim3(a.ctas), dim3(k.threads), args, 0, stream)) != VR_SUCCESS)
    return e;
  if ((e = op_launch((const void*)balance_finish_kernel, dim3(1), dim3(1024), args, 0, stream)) !=
      VR_SUCCESS)
    return e;
  if (!grads || !a.total) return VR_SUCCESS;
  const int groups = k.threads > 256 ? k.groups / 4 : k.groups;
  const long long want = (a.total + groups - 1) / groups;
  const int grid = (int)std::min<long long>(want, (long long)dev.sms * 8);
  return op_launch(k.grad, dim3(grid), dim3(256), args, 0, stream);
}

}  // extern "C"
