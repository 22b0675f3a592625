// One AdamW step over many tensors at once (vr_adamw), and the values of its
// 8-bit states (vr_adamw_values).
//
//   g = gradScale grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// All tensors of a launch are cut into chunks, which the CTAs take in turn; a
// warp updates blocks of 256 elements, eight consecutive ones a lane, in one
// pass over every array.
//
// States of 8 bits.  256 elements share a power of two as scale, by the
// largest of them.  m keeps a sign, four bits of exponent and three of
// mantissa; v, which is positive and ranges over twice the exponents, five and
// three.  Both are a 32-bit number, multiplied so that the format's lowest
// exponent becomes a denormal's, without its last 20 bits: the codes are the
// remaining ones.  20 random bits are added before they are cut off, so that
// a code is the value on average.  (Rounded to the nearest, v would never move:
// one step changes it by 1 - b2 of itself, a thousandth, and its neighbours are
// a sixteenth away.)  The random bits are a function of seed, step and element.
// A positive v does not become zero: its code is 1 at least, or m, whose
// smallest code is about as large against sqrt(v)'s, would be divided by eps.
//
// The states are computed with each operation rounded by itself, so that the
// codes are the same wherever the formulas are evaluated in 32 bits.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <vector>

#include "common.h"
#include "fold.cuh"
#include "ops.h"

namespace vr {
namespace {

constexpr int kBlock = 256;  // elements that share a scale, and a warp's
constexpr int kLane = kBlock / 32;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 2 * kWarps * kBlock;  // elements that a CTA takes at a time
constexpr int kTensors = 52;                 // of one launch

struct Tensor {
  void* param;
  const void* grad;
  void *m, *v;
  float *mScale, *vScale, *master;
  long long size;
  long long block;  // blocks of the call's earlier tensors
};
struct AdamArgs {
  Tensor tensor[kTensors];
  int first[kTensors + 1];  // chunk that a tensor begins with
  int count;
  unsigned vec[2];          // tensors whose rows allow vector accesses
  float beta1, beta2, eps, weightDecay;
  float gradScale, up, down, keep;  // up: lr / (1 - b1^t); down: 1 / (1 - b2^t)
  float logBeta1, logBeta2;
  const float* control;
  unsigned seedKey;
  long long step;
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments exceed 4 KB");

// A bijection of 32-bit numbers in which every bit depends on all bits.
__host__ __device__ __forceinline__ unsigned mix(unsigned x) {
  x ^= x >> 16;
  x *= 0x6a09e667u;
  x ^= x >> 15;
  x *= 0xbb67ae85u;
  return x ^ x >> 16;
}

// Eight consecutive elements, of which those below n are there.
template <typename T>
struct Eight {
  using Bits = typename Ty<T>::Bits;
  static constexpr int kWords = 8 * (int)sizeof(Bits) / 4;
  static __device__ __forceinline__ void load(const void* p, int n, bool vec, float (&x)[kLane]) {
    const Bits* b = static_cast<const Bits*>(p);
    if (vec && n >= kLane) {
      uint32_t w[kWords];
      load_words(p, w);
      const Bits* r = reinterpret_cast<const Bits*>(w);
#pragma unroll
      for (int i = 0; i < kLane; ++i) x[i] = Ty<T>::widen(r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kLane; ++i) x[i] = i < n ? Ty<T>::widen(b[i]) : 0.0f;
    }
  }
  static __device__ __forceinline__ void store(void* p, int n, bool vec,
                                               const float (&x)[kLane]) {
    Bits* b = static_cast<Bits*>(p);
    if (vec && n >= kLane) {
      uint32_t w[kWords];
      Bits* r = reinterpret_cast<Bits*>(w);
#pragma unroll
      for (int i = 0; i < kLane; ++i) r[i] = Ty<T>::narrow(x[i]);
      store_words(p, w);
    } else {
#pragma unroll
      for (int i = 0; i < kLane; ++i)
        if (i < n) b[i] = Ty<T>::narrow(x[i]);
    }
  }
  static __device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[4]) {
    const uint4 q = *static_cast<const uint4*>(p);
    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
  }
  static __device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  }
  static __device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[4]) {
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  }
};

// Codes of eight elements, and what they stand for: the code's digits as those
// of a 32-bit number, times 2^LIFT and the block's scale.
__device__ __forceinline__ uint2 load_codes(const void* p, int n, bool vec) {
  if (vec && n >= kLane) return *static_cast<const uint2*>(p);
  const uint8_t* b = static_cast<const uint8_t*>(p);
  uint2 q = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < kLane; ++i)
    if (i < n) (i < 4 ? q.x : q.y) |= (unsigned)b[i] << (8 * (i % 4));
  return q;
}
__device__ __forceinline__ void store_codes(void* p, int n, bool vec, uint2 q) {
  if (vec && n >= kLane) {
    *static_cast<uint2*>(p) = q;
    return;
  }
  uint8_t* b = static_cast<uint8_t*>(p);
#pragma unroll
  for (int i = 0; i < kLane; ++i)
    if (i < n) b[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i % 4)));
}
__device__ __forceinline__ unsigned code_at(uint2 q, int i) {
  return (i < 4 ? q.x : q.y) >> (8 * (i % 4)) & 255u;
}
// 2^e, e in [-126, 127]
__device__ __forceinline__ float power(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }

template <bool SECOND>
struct State8 {
  static constexpr int kTop = SECOND ? 15 : 7;       // exponent of a block's largest value
  static constexpr int kLift = SECOND ? 112 : 120;   // of a code's value above the 32-bit number's
  static __device__ __forceinline__ void decode(uint2 q, float scale, float (&x)[kLane]) {
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      const unsigned c = code_at(q, i);
      const float y =
          __fmul_rn(__fmul_rn(__uint_as_float((SECOND ? c : c & 127u) << 20), power(kLift)), scale);
      x[i] = __uint_as_float(__float_as_uint(y) | (SECOND ? 0u : (c & 128u) << 24));
    }
  }
  // The codes of a warp's block and its scale; `cut`: 20 random bits each.
  // A NaN or an infinity makes the scale NaN.
  static __device__ __forceinline__ uint2 encode(const float (&x)[kLane],
                                                 const unsigned (&cut)[kLane], float* scale) {
    unsigned top = 0;  // of the absolute values; NaN is above infinity
#pragma unroll
    for (int i = 0; i < kLane; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    uint2 q = make_uint2(0, 0);
    if (top >= 0x7f800000u) {
      *scale = __uint_as_float(0x7fffffffu);
      return q;
    }
    const int e = max((int)(top >> 23) - 127, -110);
    *scale = power(e - kTop);
    const float up = power(kTop - e);
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      const float y = __fmul_rn(__fmul_rn(fabsf(x[i]), up), power(-kLift));
      unsigned c = (__float_as_uint(y) + cut[i]) >> 20;
      if (SECOND) c = x[i] > 0.0f ? max(c, 1u) : c;
      else c |= x[i] < 0.0f && c ? 128u : 0u;
      (i < 4 ? q.x : q.y) |= c << (8 * (i % 4));
    }
    return q;
  }
};

__device__ __forceinline__ bool bit_of(const unsigned (&w)[2], int i) {
  return (w[i / 32] >> (i % 32) & 1) != 0;
}

// The tensor that chunk c belongs to.
__device__ __forceinline__ int tensor_of(const AdamArgs& a, int c) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// P: of the parameters, G: of the gradients; BITS of the states; MASTER: 32-bit
// parameters beside P's, which are written only.
template <typename P, typename G, int BITS, bool MASTER>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamArgs a) {
  pdl_launch();
  pdl_wait();
  float gradScale = a.gradScale, up = a.up, down = a.down, keep = a.keep;
  long long step = a.step;
  if (a.control) {
    const float lr = a.control[0], t = a.control[1];
    gradScale = a.control[2];
    if (!(fabsf(gradScale) < INFINITY)) return;  // no step
    step = (long long)t;
    up = lr / -expm1f(t * a.logBeta1);
    down = 1.0f / -expm1f(t * a.logBeta2);
    keep = 1.0f - lr * a.weightDecay;
  }
  unsigned key = 0;
  if (BITS == 8) key = mix(mix(a.seedKey ^ (unsigned)step) ^ (unsigned)(step >> 32));
  const float rest1 = 1.0f - a.beta1, rest2 = 1.0f - a.beta2;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int chunks = a.first[a.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int lo = tensor_of(a, c);
    const Tensor& t = a.tensor[lo];
    const bool vec = bit_of(a.vec, lo);
    const long long from = (long long)(c - a.first[lo]) * kChunk;
#pragma unroll 1
    for (int part = 0; part < kChunk / (kWarps * kBlock); ++part) {
      const long long at = from + (part * kWarps + warp) * kBlock;  // of the warp's block
      if (at >= t.size) break;
      const long long i0 = at + lane * kLane;
      const int n = (int)max(min(t.size - i0, (long long)kLane), 0LL);
      float g[kLane], p[kLane], m[kLane], v[kLane];
      uint2 qm, qv;
      float scaleM, scaleV;
      char *codesM = static_cast<char*>(t.m) + i0, *codesV = static_cast<char*>(t.v) + i0;
      float *wordsM = static_cast<float*>(t.m) + i0, *wordsV = static_cast<float*>(t.v) + i0;
      if (BITS == 8) {
        qm = load_codes(codesM, n, vec);
        qv = load_codes(codesV, n, vec);
        scaleM = t.mScale[at / kBlock];
        scaleV = t.vScale[at / kBlock];
      } else {
        Eight<float>::load(wordsM, n, vec, m);
        Eight<float>::load(wordsV, n, vec, v);
      }
      Eight<G>::load(static_cast<const G*>(t.grad) + i0, n, vec, g);
      if (MASTER) Eight<float>::load(t.master + i0, n, vec, p);
      else Eight<P>::load(static_cast<const P*>(t.param) + i0, n, vec, p);
      if (BITS == 8) {
        State8<false>::decode(qm, scaleM, m);
        State8<true>::decode(qv, scaleV, v);
      }
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        const float x = __fmul_rn(g[i], gradScale);
        m[i] = __fadd_rn(__fmul_rn(m[i], a.beta1), __fmul_rn(x, rest1));
        v[i] = __fadd_rn(__fmul_rn(v[i], a.beta2), __fmul_rn(__fmul_rn(x, x), rest2));
        float root;
        asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v[i] * down));
        p[i] = p[i] * keep - __fdividef(up * m[i], root + a.eps);
      }
      if (MASTER) Eight<float>::store(t.master + i0, n, vec, p);
      Eight<P>::store(static_cast<P*>(t.param) + i0, n, vec, p);
      if (BITS == 8) {
        const unsigned long long place =
            (unsigned long long)(t.block + at / kBlock) * kBlock + lane * kLane;
        const unsigned by = mix(key ^ (unsigned)(place >> 32));
        unsigned cutM[kLane], cutV[kLane];
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
          const unsigned r = mix(by ^ ((unsigned)place + i));
          cutM[i] = (r & 0xffffu) << 4;
          cutV[i] = r >> 16 << 4;
        }
        qm = State8<false>::encode(m, cutM, &scaleM);
        qv = State8<true>::encode(v, cutV, &scaleV);
        store_codes(codesM, n, vec, qm);
        store_codes(codesV, n, vec, qv);
        if (lane == 0) t.mScale[at / kBlock] = scaleM, t.vScale[at / kBlock] = scaleV;
      } else {
        Eight<float>::store(wordsM, n, vec, m);
        Eight<float>::store(wordsV, n, vec, v);
      }
    }
  }
}

// The values of 8-bit states in 32 bits: `param` is m's, `master` v's (each may
// be null).
__global__ void __launch_bounds__(kThreads) adamw_values_kernel(
    const __grid_constant__ AdamArgs a) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int chunks = a.first[a.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int lo = tensor_of(a, c);
    const Tensor& t = a.tensor[lo];
    const bool vec = bit_of(a.vec, lo);
    const long long from = (long long)(c - a.first[lo]) * kChunk;
#pragma unroll
    for (int part = 0; part < kChunk / (kWarps * kBlock); ++part) {
      const long long at = from + (part * kWarps + warp) * kBlock;
      if (at >= t.size) break;
      const long long i0 = at + lane * kLane;
      const int n = (int)max(min(t.size - i0, (long long)kLane), 0LL);
      float x[kLane];
      if (t.param) {
        State8<false>::decode(load_codes(static_cast<const char*>(t.m) + i0, n, vec),
                              t.mScale[at / kBlock], x);
        Eight<float>::store(static_cast<float*>(t.param) + i0, n, vec, x);
      }
      if (t.master) {
        State8<true>::decode(load_codes(static_cast<const char*>(t.v) + i0, n, vec),
                             t.vScale[at / kBlock], x);
        Eight<float>::store(t.master + i0, n, vec, x);
      }
    }
  }
}

// ------------------------------------------------------------- host side
template <typename P, typename G>
const void* kernel_of(int bits, bool master) {
  if constexpr (std::is_same<P, float>::value) {
    return bits == 8 ? (const void*)adamw_kernel<P, G, 8, false>
                     : (const void*)adamw_kernel<P, G, 32, false>;
  } else {
    if (master)
      return bits == 8 ? (const void*)adamw_kernel<P, G, 8, true>
                       : (const void*)adamw_kernel<P, G, 32, true>;
    return bits == 8 ? (const void*)adamw_kernel<P, G, 8, false>
                     : (const void*)adamw_kernel<P, G, 32, false>;
  }
}
template <typename P>
const void* kernel_of(int gradDtype, int bits, bool master) {
  return gradDtype == VR_FLOAT32   ? kernel_of<P, float>(bits, master)
         : gradDtype == VR_FLOAT16 ? kernel_of<P, __half>(bits, master)
                                   : kernel_of<P, __nv_bfloat16>(bits, master);
}

constexpr size_t kMostSize = (size_t)1 << 40;

// The buffers of a call: extents, and whether each is written.
struct Spans {
  std::vector<OpSpan> v;
  void add(const void* p, size_t bytes, bool write) {
    if (p && bytes) v.push_back({(uintptr_t)p, (uintptr_t)p + bytes, write});
  }
};

// Launches `fn` over the tensors, kTensors at a time.  `fill` writes tensor i
// and returns the address bits of its rows.
template <class Fill>
vr_result_t over_tensors(const void* fn, AdamArgs& a, const size_t* sizes, int count,
                         const OpDevice& dev, void* stream, Fill fill) {
  long long block = 0;
  int i = 0;
  while (i < count) {
    long long chunks = 0;
    a.count = 0;
    a.vec[0] = a.vec[1] = 0;
    for (; i < count && a.count < kTensors; ++i) {
      const long long n = (long long)sizes[i];
      if (!n) continue;
      const long long more = (n + kChunk - 1) / kChunk;
      if (a.count && chunks + more > INT_MAX) break;
      Tensor& t = a.tensor[a.count];
      if (fill(i, &t)) a.vec[a.count / 32] |= 1u << (a.count % 32);
      t.size = n;
      t.block = block;
      block += (n + kBlock - 1) / kBlock;
      a.first[a.count++] = (int)chunks;
      chunks += more;
    }
    if (!a.count) break;
    a.first[a.count] = (int)chunks;
    void* args[] = {&a};
    const vr_result_t e =
        op_launch(fn, dim3((unsigned)std::min<long long>(chunks, dev.sms * 8LL)), dim3(kThreads),
                  args, 0, stream);
    if (e != VR_SUCCESS) return e;
  }
  return VR_SUCCESS;
}

}  // namespace
}  // namespace vr

using namespace vr;

extern "C" {

vr_result_t vr_adamw(void* const* params, const void* const* grads, void* const* m,
                     void* const* v, float* const* mScales, float* const* vScales,
                     float* const* masters, const size_t* sizes, int count, vr_dtype_t dtype,
                     vr_dtype_t gradDtype, int stateBits, float lr, float beta1, float beta2,
                     float eps, float weightDecay, long long step, float gradScale,
                     unsigned long long seed, const float* control, void* stream) {
  const size_t E = op_elem_size(dtype), GE = op_elem_size(gradDtype);
  const bool few = stateBits == 8;
  auto beta_ok = [](float b) { return b >= 0.0f && b < 1.0f; };
  if (!E || !GE || (stateBits != 8 && stateBits != 32) || count < 1 || !params || !grads || !m ||
      !v || !sizes || few != (mScales != nullptr) || few != (vScales != nullptr) ||
      (masters && dtype == VR_FLOAT32) || !beta_ok(beta1) || !beta_ok(beta2) || !(eps >= 0.0f) ||
      !std::isfinite(eps) || ((uintptr_t)control & 3) ||
      (!control && (!std::isfinite(lr) || !std::isfinite(gradScale) || step < 1)) ||
      !std::isfinite(weightDecay))
    return VR_ERR_INVALID_ARGUMENT;
  const size_t SE = few ? 1 : 4;
  try {
    Spans spans;
    spans.v.reserve((size_t)count * 7 + 1);
    std::vector<const void*> reach;
    for (int i = 0; i < count; ++i) {
      const size_t n = sizes[i], blocks = (n + kBlock - 1) / kBlock;
      if (n > kMostSize) return VR_ERR_INVALID_ARGUMENT;
      if (!n) continue;
      if (!params[i] || !grads[i] || !m[i] || !v[i] || (few && (!mScales[i] || !vScales[i])) ||
          (masters && !masters[i]) || (uintptr_t)params[i] % E || (uintptr_t)grads[i] % GE ||
          ((uintptr_t)m[i] | (uintptr_t)v[i]) % SE ||
          (few && ((uintptr_t)mScales[i] | (uintptr_t)vScales[i]) % 4) ||
          (masters && (uintptr_t)masters[i] % 4))
        return VR_ERR_INVALID_ARGUMENT;
      spans.add(params[i], n * E, true);
      spans.add(grads[i], n * GE, false);
      spans.add(m[i], n * SE, true);
      spans.add(v[i], n * SE, true);
      if (few) {
        spans.add(mScales[i], blocks * 4, true);
        spans.add(vScales[i], blocks * 4, true);
      }
      if (masters) spans.add(masters[i], n * 4, true);
    }
    spans.add(control, 12, false);
    if (!op_spans_ok(spans.v.data(), spans.v.size())) return VR_ERR_INVALID_ARGUMENT;
    OpDevice dev;
    vr_result_t e = op_device(&dev);
    if (e != VR_SUCCESS) return e;
    for (const OpSpan& s : spans.v) {
      const void* p = (const void*)s.lo;
      if ((e = op_reachable(&p, 1, dev.device)) != VR_SUCCESS) return e;
    }
    AdamArgs a;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.eps = eps;
    a.weightDecay = weightDecay;
    a.gradScale = gradScale;
    const double log1 = std::log((double)beta1), log2 = std::log((double)beta2);
    a.logBeta1 = (float)log1;
    a.logBeta2 = (float)log2;
    a.up = (float)((double)lr / -std::expm1((double)step * log1));
    a.down = (float)(1.0 / -std::expm1((double)step * log2));
    a.keep = (float)(1.0 - (double)lr * (double)weightDecay);
    a.control = control;
    a.seedKey = mix(mix((unsigned)seed) ^ (unsigned)(seed >> 32));
    a.step = step;
    const void* fn = dtype == VR_FLOAT32   ? kernel_of<float>(gradDtype, stateBits, false)
                     : dtype == VR_FLOAT16 ? kernel_of<__half>(gradDtype, stateBits, masters)
                                           : kernel_of<__nv_bfloat16>(gradDtype, stateBits, masters);
    return over_tensors(fn, a, sizes, count, dev, stream, [&](int i, Tensor* t) {
      *t = {params[i],
            grads[i],
            m[i],
            v[i],
            few ? mScales[i] : nullptr,
            few ? vScales[i] : nullptr,
            masters ? masters[i] : nullptr,
            0,
            0};
      return (uintptr_t)params[i] % (8 * E) == 0 && (uintptr_t)grads[i] % (8 * GE) == 0 &&
             ((uintptr_t)m[i] | (uintptr_t)v[i]) % (8 * SE) == 0 && (uintptr_t)t->master % 32 == 0;
    });
  } catch (...) {  // no host memory for the list
    return VR_ERR_INTERNAL;
  }
}

vr_result_t vr_adamw_values(const void* const* m, const void* const* v,
                            const float* const* mScales, const float* const* vScales,
                            const size_t* sizes, int count, float* const* mValues,
                            float* const* vValues, void* stream) {
  if (count < 1 || !sizes || (mValues && (!m || !mScales)) || (vValues && (!v || !vScales)) ||
      (!mValues && !vValues))
    return VR_ERR_INVALID_ARGUMENT;
  try {
    Spans spans;
    spans.v.reserve((size_t)count * 6);
    for (int i = 0; i < count; ++i) {
      const size_t n = sizes[i], blocks = (n + kBlock - 1) / kBlock;
      if (n > kMostSize) return VR_ERR_INVALID_ARGUMENT;
      auto one = [&](const void* const* codes, const float* const* scales, float* const* out) {
        if (!n || !out) return true;
        if (!codes[i] || !scales[i] || !out[i] ||
            ((uintptr_t)scales[i] | (uintptr_t)out[i]) % 4)
          return false;
        spans.add(codes[i], n, false);
        spans.add(scales[i], blocks * 4, false);
        spans.add(out[i], n * 4, true);
        return true;
      };
      if (!one(m, mScales, mValues) || !one(v, vScales, vValues)) return VR_ERR_INVALID_ARGUMENT;
    }
    if (!op_spans_ok(spans.v.data(), spans.v.size())) return VR_ERR_INVALID_ARGUMENT;
    OpDevice dev;
    vr_result_t e = op_device(&dev);
    if (e != VR_SUCCESS) return e;
    for (const OpSpan& s : spans.v) {
      const void* p = (const void*)s.lo;
      if ((e = op_reachable(&p, 1, dev.device)) != VR_SUCCESS) return e;
    }
    AdamArgs a;
    return over_tensors((const void*)adamw_values_kernel, a, sizes, count, dev, stream,
                        [&](int i, Tensor* t) {
                          *t = {mValues ? mValues[i] : nullptr,
                                nullptr,
                                mValues ? const_cast<void*>(m[i]) : nullptr,
                                vValues ? const_cast<void*>(v[i]) : nullptr,
                                mValues ? const_cast<float*>(mScales[i]) : nullptr,
                                vValues ? const_cast<float*>(vScales[i]) : nullptr,
                                vValues ? vValues[i] : nullptr,
                                0,
                                0};
                          return ((uintptr_t)t->m | (uintptr_t)t->v) % 8 == 0 &&
                                 ((uintptr_t)t->param | (uintptr_t)t->master) % 32 == 0;
                        });
  } catch (...) {  // no host memory for the list
    return VR_ERR_INTERNAL;
  }
}

}  // extern "C"
