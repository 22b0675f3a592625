// One AdamW step over many tensors at once (vr_adamw), and the values of its
// 8-bit states (vr_adamw_values).
//
//   g = gradScale grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// All tensors of a launch are cut into chunks, which the CTAs take in turn; a
// warp updates blocks of 256 elements, eight consecutive ones a lane, in one
// pass over every array.  With states of 32 bits that is bound by memory: 147 M
// parameters in bf16 with masters, 28 bytes each, take 620 to 638 us (6.4 to 6.6
// TB/s).  With states of 8 bits it is 16 bytes and 67 instructions an element: 122
// M take 365 to 370 us (5.2 to 5.3 TB/s), the issue slots 61 % busy (82
// instructions and 430 us before codes were packed four at a time and decoded by
// conversions).
//
// Tensors of which a buffer does not begin at a multiple of eight elements go
// element by element, as ends of tensors do: 100 M in bf16 with masters take 865 to
// 1050 us instead of 440 (states of 32 bits), 660 to 800 instead of 298 (8 bits).
//
// States of 8 bits.  256 elements share a power of two as scale, by the
// largest of them.  m keeps a sign, four bits of exponent and three of
// mantissa; v, which is positive and ranges over twice the exponents, five and
// three.  Both are a 32-bit number, multiplied so that the format's lowest
// exponent becomes a denormal's, without its last 20 bits: the codes are the
// remaining ones.  A random number is added before they are cut off (16 bits, at
// the upper end of the 20), so that a code is the value on average.  (Rounded to
// the nearest, v would never move: one step changes it by 1 - b2 of itself, a
// thousandth, and its neighbours are a sixteenth away.)  The random bits are a
// function of seed, step and element.
// A positive v does not become zero: its code is 1 at least, or m, whose
// smallest code is about as large against sqrt(v)'s, would be divided by eps.
//
// The states are computed with each operation rounded by itself, so that the
// codes are the same wherever the formulas are evaluated in 32 bits.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <vector>

#include <cuda_fp16.h>

#include "common.h"
#include "fold.cuh"
#include "gemm_host.h"

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
  float gradScale, up, down, decay;  // up: lr / (1 - b1^t); down: (1 - b2^t)^(-1/2)
  float logBeta1, logBeta2;
  const float* control;
  unsigned seedKey;
  long long step;
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments exceed 4 KB");

// A bijection of 32-bit numbers in which every bit depends on all bits.  (A
// changed bit of x changes each bit of the result with a probability within
// 0.004 of a half, what 200000 samples resolve; the factors are digits of the
// roots of 2 and 3.)
constexpr unsigned kMix1 = 0x6a09e667u, kMix2 = 0xbb67ae85u;
__host__ __device__ __forceinline__ unsigned mix(unsigned x) {
  x = (x ^ x >> 16) * kMix1;
  x = (x ^ x >> 15) * kMix2;
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
      widen(w, x);
    } else {
#pragma unroll
      for (int i = 0; i < kLane; ++i) x[i] = i < n ? Ty<T>::widen(b[i]) : 0.0f;
    }
  }
  static __device__ __forceinline__ void widen(const uint32_t (&w)[kWords], float (&x)[kLane]) {
    const Bits* r = reinterpret_cast<const Bits*>(w);
#pragma unroll
    for (int i = 0; i < kLane; ++i) x[i] = Ty<T>::widen(r[i]);
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

// Codes of eight elements.
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
// 2^e, e in [-126, 127]
__device__ __forceinline__ float power(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }
// The top bytes of four words.
__device__ __forceinline__ unsigned top_bytes(const unsigned (&x)[kLane], int first) {
  const unsigned lo = __byte_perm(x[first], x[first + 1], 0x0073);
  return __byte_perm(lo, __byte_perm(x[first + 2], x[first + 3], 0x0073), 0x5410);
}

// Exponents: of a block's largest value, and of a code's value above that of
// the 32-bit number with its digits.
constexpr int kTopM = 7, kLiftM = 120, kTopV = 15, kLiftV = 112;

__device__ __forceinline__ void decode_m(uint2 q, float scale, float (&x)[kLane]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(i ? q.y : q.x));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[4 * i] = a.x * scale, x[4 * i + 1] = a.y * scale;
    x[4 * i + 2] = b.x * scale, x[4 * i + 3] = b.y * scale;
  }
}
__device__ __forceinline__ void decode_v(uint2 q, float scale, float (&x)[kLane]) {
  // (2^lift scale in one factor where that is a 32-bit number)
  const bool large = scale >= power(127 - kLiftV);
  const float by = large ? power(kLiftV) : scale * power(kLiftV);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // two codes: 20 bits up each
    const unsigned two = __byte_perm(i < 2 ? q.x : q.y, 0, i % 2 ? 0x4342 : 0x4140) * 16u;
    x[2 * i] = __fmul_rn(__uint_as_float(two << 16), by);
    x[2 * i + 1] = __fmul_rn(__uint_as_float(two & 0xffff0000u), by);
  }
  if (large) {
#pragma unroll
    for (int i = 0; i < kLane; ++i) x[i] = __fmul_rn(x[i], scale);
  }
}
// max of |a| and b that keeps NaN
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %1;\n\tmax.NaN.f32 %0, t, %2;\n\t}"
      : "=f"(r)
      : "f"(a), "f"(b));
  return r;
}
// x, an infinity made the largest number.  (One instruction: two of min and max, or a
// comparison and a choice, take 1 % of the step with 8-bit states, and a comparison
// 0.3 us of the shortest one's 4.)
__device__ __forceinline__ float finite(float x) {
  float r;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(FLT_MAX));
  return r;
}
// A warp's block by its largest absolute value: its scale, 2^(exponent - top),
// and x multiplied so that the codes' digits are those of 32-bit numbers from
// bit 20 on.  (One factor, which may be a denormal; where it would be less, x
// goes down by 2^100 first.  What that rounds is below 2^-126 of a block above
// 2^36, nothing in its codes.)  An infinity or a NaN makes the scale NaN.
template <int TOP, int LIFT>
__device__ __forceinline__ float block_scale(const float (&x)[kLane], float (&y)[kLane]) {
  float largest = 0.0f;
#pragma unroll
  for (int i = 0; i < kLane; ++i) largest = max_abs(x[i], largest);
  const unsigned all = __reduce_max_sync(0xffffffffu, __float_as_uint(largest));
  int e = max((int)(all >> 23) - 127, -110);
  const float scale = all >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : power(e - TOP);
  constexpr int kDown = 100;
  static_assert(TOP - LIFT - (127 - kDown) >= -149, "the factor of the largest blocks");
  if (e > 149 + TOP - LIFT) {
    e -= kDown;
#pragma unroll
    for (int i = 0; i < kLane; ++i) y[i] = __fmul_rn(x[i], power(-kDown));
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) y[i] = x[i];
  }
  const int k = TOP - LIFT - e;
  const float by = __uint_as_float(k >= -126 ? (unsigned)(k + 127) << 23 : 1u << (k + 149));
#pragma unroll
  for (int i = 0; i < kLane; ++i) y[i] = __fmul_rn(y[i], by);
  return scale;
}
// A block's largest values may be rounded up to the next power of two, but not
// to 2^128: they keep the code below, 1.875 2^127.
template <int TOP>
__device__ __forceinline__ void hold_finite(unsigned (&u)[kLane], float scale) {
  if (scale == power(127 - TOP)) {
    constexpr unsigned kMost = ((unsigned)(2 * TOP + 1) << 3) << 24;  // code of 2^(TOP + 1)
#pragma unroll
    for (int i = 0; i < kLane; ++i) u[i] = min(u[i], kMost - 1);
  }
}
// New codes; `cut`: 16 random bits each, from bit 8.  (Shifted up by 4, a code
// is a word's top byte.)
__device__ __forceinline__ uint2 encode_m(const float (&x)[kLane], const unsigned (&cut)[kLane],
                                          float* scale) {
  float y[kLane];
  *scale = block_scale<kTopM, kLiftM>(x, y);
  unsigned t[kLane], u[kLane];
#pragma unroll
  for (int i = 0; i < kLane; ++i) {
    t[i] = __float_as_uint(y[i]);
    u[i] = t[i] * 16u + cut[i];
  }
  hold_finite<kTopM>(u, *scale);
  if (*scale != *scale) return make_uint2(0, 0);
  return make_uint2((top_bytes(t, 0) & 0x80808080u) | top_bytes(u, 0),
                    (top_bytes(t, 4) & 0x80808080u) | top_bytes(u, 4));
}
__device__ __forceinline__ uint2 encode_v(const float (&x)[kLane], const unsigned (&cut)[kLane],
                                          float* scale) {
  float y[kLane];
  *scale = block_scale<kTopV, kLiftV>(x, y);
  unsigned t[kLane], u[kLane], least = ~0u;
#pragma unroll
  for (int i = 0; i < kLane; ++i) {
    t[i] = __float_as_uint(y[i]);
    least = min(least, t[i]);
  }
  if (least < 1u << 20) {  // a positive one does not become zero
#pragma unroll
    for (int i = 0; i < kLane; ++i)
      if (x[i] > 0.0f) t[i] = max(t[i], 1u << 20);
  }
#pragma unroll
  for (int i = 0; i < kLane; ++i) u[i] = t[i] * 16u + cut[i];
  hold_finite<kTopV>(u, *scale);
  if (*scale != *scale) return make_uint2(0, 0);
  return make_uint2(top_bytes(u, 0), top_bytes(u, 4));
}

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

// The chunks that a CTA takes one after the other, and a warp's place in each:
// kParts blocks kStride elements apart.  States of 32 bits: those of the warps
// interleaved (620 to 638 us for 147 M parameters; 645 where a warp's follow one
// another), states of 8 bits: a warp's side by side (365 to 380 us for 122 M;
// 390 interleaved).
constexpr int kParts = kChunk / (kWarps * kBlock);
template <int BITS>
constexpr int kStride = BITS == 8 ? kBlock : kWarps * kBlock;
struct Cursor {
  int chunk, tensor;
  __device__ __forceinline__ Cursor(const AdamArgs& a)
      : chunk((int)blockIdx.x), tensor(tensor_of(a, min(chunk, a.first[a.count] - 1))) {}
  __device__ __forceinline__ bool more(const AdamArgs& a) const { return chunk < a.first[a.count]; }
  __device__ __forceinline__ void advance(const AdamArgs& a) {
    chunk += gridDim.x;
    while (more(a) && chunk >= a.first[tensor + 1]) ++tensor;
  }
  // the first element of the warp's first block
  template <int BITS>
  __device__ __forceinline__ long long at(const AdamArgs& a) const {
    constexpr int kWarp = BITS == 8 ? kParts * kBlock : kBlock;
    return (long long)(chunk - a.first[tensor]) * kChunk + (int)(threadIdx.x / 32) * kWarp;
  }
};
// Whole blocks with vector accesses.
template <int BITS>
__device__ __forceinline__ bool whole(const AdamArgs& a, int tensor, const Tensor& t, long long at) {
  return bit_of(a.vec, tensor) && t.size - at >= (kParts - 1) * kStride<BITS> + kBlock;
}

// Blocks on their way.  With states of 8 bits a block is 2 KB, too little to
// keep the memory busy while it is computed on: each lane copies its share of
// the next chunk's blocks into shared memory (cp.async, no registers).
constexpr int kAhead = 2;
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, int bytes) {
  if (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else if (bytes == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
// A block of a warp's slot: planes of 16 bytes a lane, the codes, the scales.
template <typename P, typename G>
struct Slot {
  static constexpr int kG = Eight<G>::kWords / 4, kP = Eight<P>::kWords / 4;  // planes
  static constexpr int kCodes = (kG + kP) * 512, kScales = kCodes + 512, kBytes = kScales + 16;
  // (blocks that are not whole: the scales of those that are there)
  static __device__ __forceinline__ void fill(uint32_t slot, const Tensor& t, const void* param,
                                              long long at, bool whole) {
    const int lane = threadIdx.x % 32;
    if (whole) {
      const long long i0 = at + lane * kLane;
      const char* g = reinterpret_cast<const char*>(static_cast<const G*>(t.grad) + i0);
      const char* p = reinterpret_cast<const char*>(static_cast<const P*>(param) + i0);
      const char *m = static_cast<const char*>(t.m) + i0, *v = static_cast<const char*>(t.v) + i0;
      const uint32_t to = slot + lane * 16, codes = slot + kCodes + lane * 8;
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
#pragma unroll
        for (int i = 0; i < kG; ++i)
          copy_async(to + k * kBytes + i * 512, g + k * (kStride<8> * (int)sizeof(G)) + i * 16, 16);
#pragma unroll
        for (int i = 0; i < kP; ++i)
          copy_async(to + k * kBytes + (kG + i) * 512, p + k * (kStride<8> * (int)sizeof(P)) + i * 16,
                     16);
        copy_async(codes + k * kBytes, m + k * kStride<8>, 8);
        copy_async(codes + k * kBytes + 256, v + k * kStride<8>, 8);
      }
    }
    const int k = lane / 2;
    if (k < kParts && at + k * kStride<8> < t.size)
      copy_async(slot + k * kBytes + kScales + lane % 2 * 4,
                 (lane % 2 ? t.vScale : t.mScale) + (at / kBlock + k * (kStride<8> / kBlock)), 4);
  }
  template <int PLANES>
  static __device__ __forceinline__ void read(uint32_t plane, uint32_t (&w)[4 * PLANES]) {
#pragma unroll
    for (int i = 0; i < PLANES; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(plane + i * 512 + threadIdx.x % 32 * 16)
                   : "memory");
  }
  static __device__ __forceinline__ void gradient(uint32_t slot, float (&x)[kLane]) {
    uint32_t w[4 * kG];
    read<kG>(slot, w);
    Eight<G>::widen(w, x);
  }
  static __device__ __forceinline__ void parameter(uint32_t slot, float (&x)[kLane]) {
    uint32_t w[4 * kP];
    read<kP>(slot + kG * 512, w);
    Eight<P>::widen(w, x);
  }
  static __device__ __forceinline__ uint2 codes(uint32_t slot, int which) {
    uint2 q;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(q.x), "=r"(q.y)
                 : "r"(slot + kCodes + which * 256 + threadIdx.x % 32 * 8)
                 : "memory");
    return q;
  }
  static __device__ __forceinline__ float scale(uint32_t slot, int which) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(slot + kScales + which * 4) : "memory");
    return x;
  }
};

// What a step multiplies by.
struct Step {
  float gradScale, up, down, decay;
  unsigned key;
};

// Where a lane's elements of a warp's first block are.
template <typename P, typename G, bool MASTER>
struct Lane {
  using Read = typename Select<MASTER, float, P>::type;  // the parameters that are read
  const G* grad;
  P* param;
  Read* read;
  char *m, *v;
  float *mScale, *vScale;
  unsigned long long place;  // among the call's tensors
  __device__ __forceinline__ Lane(const Tensor& t, long long at, int bytes) {
    const long long i0 = at + (int)(threadIdx.x % 32) * kLane;
    grad = static_cast<const G*>(t.grad) + i0;
    param = static_cast<P*>(t.param) + i0;
    if constexpr (MASTER) read = t.master + i0;
    else read = param;
    m = static_cast<char*>(t.m) + i0 * bytes;
    v = static_cast<char*>(t.v) + i0 * bytes;
    if (bytes == 1) {
      const long long block = (long long)((unsigned long long)at / kBlock);
      mScale = t.mScale + block;
      vScale = t.vScale + block;
      place = (unsigned long long)(t.block + block) * kBlock + threadIdx.x % 32 * kLane;
    }
  }
};

// Block `part` of a warp's, its inputs in `slot` of shared memory (states of 8
// bits, WHOLE blocks) or where they are.  n: elements of the lane that are there.
template <typename P, typename G, int BITS, bool MASTER, bool WHOLE>
__device__ __forceinline__ void update_block(const AdamArgs& a, const Step& s,
                                             const Lane<P, G, MASTER>& l, int part, int n,
                                             uint32_t slot) {
  using Read = typename Select<MASTER, float, P>::type;
  using S = Slot<Read, G>;
  const int off = part * kStride<BITS>;
  float g[kLane], p[kLane], m[kLane], v[kLane];
  char *codesM = l.m + off, *codesV = l.v + off;
  float *wordsM = reinterpret_cast<float*>(l.m) + off, *wordsV = reinterpret_cast<float*>(l.v) + off;
  if (BITS == 8) {
    uint2 qm, qv;
    if (WHOLE) {
      S::gradient(slot, g);
      S::parameter(slot, p);
      qm = S::codes(slot, 0);
      qv = S::codes(slot, 1);
    } else {
      qm = load_codes(codesM, n, false);
      qv = load_codes(codesV, n, false);
    }
    decode_m(qm, S::scale(slot, 0), m);
    decode_v(qv, S::scale(slot, 1), v);
  } else {
    Eight<float>::load(wordsM, n, WHOLE, m);
    Eight<float>::load(wordsV, n, WHOLE, v);
  }
  if (BITS != 8 || !WHOLE) {
    Eight<G>::load(l.grad + off, n, WHOLE, g);
    Eight<Read>::load(l.read + off, n, WHOLE, p);
  }
  const float rest1 = 1.0f - a.beta1, rest2 = 1.0f - a.beta2;
#pragma unroll
  for (int i = 0; i < kLane; ++i) {
    const float x = __fmul_rn(g[i], s.gradScale);
    m[i] = __fadd_rn(__fmul_rn(m[i], a.beta1), __fmul_rn(x, rest1));
    v[i] = __fadd_rn(__fmul_rn(v[i], a.beta2), __fmul_rn(__fmul_rn(x, x), rest2));
    // (root + eps is 0 or above 2^-75: no denormal to be flushed; v / (1 - b2^t)
    // could pass 2^128)
    float root, inv;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v[i]));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(root, s.down, a.eps)));
    // What p loses by its decay, lr wd p, is added to its move before the one
    // rounding of p: 1 - lr wd in 32 bits would be 1, or off by a half, where lr wd is
    // about 2^-24.  (A parameter that is infinite, a mask, stays so: its decay is
    // that of the largest number.)
    p[i] -= fmaf(s.decay, finite(p[i]), s.up * m[i] * inv);
  }
  if (MASTER) Eight<Read>::store(l.read + off, n, WHOLE, p);
  Eight<P>::store(l.param + off, n, WHOLE, p);
  if (BITS == 8) {
    // mix(x ^ i) of the lane's eight places (i < 8 leaves x >> 16 as it is): the
    // upper half of r for v, its lower half after r ^= r >> 16 for m
    const unsigned long long place = l.place + (unsigned)off;
    const unsigned x = mix(s.key ^ (unsigned)(place >> 32)) ^ (unsigned)place;
    unsigned cutM[kLane], cutV[kLane];
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      unsigned r = ((x ^ x >> 16) ^ (unsigned)i) * kMix1;
      r = (r ^ r >> 15) * kMix2;
      cutV[i] = __byte_perm(r, 0, 0x4324);
      cutM[i] = __byte_perm(r, 0, 0x4104) ^ cutV[i];
    }
    float scaleM, scaleV;
    const uint2 qm = encode_m(m, cutM, &scaleM), qv = encode_v(v, cutV, &scaleV);
    store_codes(codesM, n, WHOLE, qm);
    store_codes(codesV, n, WHOLE, qv);
    if (threadIdx.x % 32 == 0) l.mScale[off / kBlock] = scaleM, l.vScale[off / kBlock] = scaleV;
  } else {
    Eight<float>::store(wordsM, n, WHOLE, m);
    Eight<float>::store(wordsV, n, WHOLE, v);
  }
}
// The blocks of a warp that are not whole.
template <typename P, typename G, int BITS, bool MASTER>
__device__ __noinline__ void update_rest(const AdamArgs& a, const Step& s, const Tensor& t,
                                         long long at, uint32_t slot) {
  const Lane<P, G, MASTER> l(t, at, BITS / 8);
#pragma unroll 1
  for (int k = 0; k < kParts && at + k * kStride<BITS> < t.size; ++k) {
    const long long left = t.size - at - k * kStride<BITS> - (int)(threadIdx.x % 32) * kLane;
    update_block<P, G, BITS, MASTER, false>(
        a, s, l, k, (int)max(min(left, (long long)kLane), 0LL),
        slot + (unsigned)(k * Slot<typename Lane<P, G, MASTER>::Read, G>::kBytes));
  }
}

// P: of the parameters, G: of the gradients; BITS of the states; MASTER: 32-bit
// parameters beside P's, which are written only.
template <typename P, typename G, int BITS, bool MASTER>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 2 : 4) adamw_kernel(const __grid_constant__ AdamArgs a) {
  using S = Slot<typename Lane<P, G, MASTER>::Read, G>;
  extern __shared__ uint4 smem[];
  pdl_launch();
  pdl_wait();
  Step s = {a.gradScale, a.up, a.down, a.decay, 0};
  long long step = a.step;
  if (a.control) {
    const float lr = a.control[0], t = a.control[1];
    s.gradScale = a.control[2];
    if (!(fabsf(s.gradScale) < INFINITY)) return;  // no step
    step = (long long)t;
    s.up = lr / -expm1f(t * a.logBeta1);
    s.down = sqrtf(1.0f / -expm1f(t * a.logBeta2));
    s.decay = lr * a.weightDecay;
  }
  if (BITS == 8) s.key = mix(mix(a.seedKey ^ (unsigned)step) ^ (unsigned)(step >> 32));
  constexpr unsigned kSlot = kParts * S::kBytes;
  const uint32_t slot0 = BITS == 8 ? smem_addr(smem) + threadIdx.x / 32 * (kAhead * kSlot) : 0u;
  Cursor now(a), ahead(a);
  auto fill = [&](int slot) {
    if (BITS == 8) {
      if (ahead.more(a)) {
        const Tensor& t = a.tensor[ahead.tensor];
        const long long at = ahead.at<BITS>(a);
        S::fill(slot0 + (unsigned)slot * kSlot, t, MASTER ? (void*)t.master : t.param, at,
                whole<BITS>(a, ahead.tensor, t, at));
        ahead.advance(a);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  fill(0);
  for (int slot = 0; now.more(a); now.advance(a), slot ^= 1) {
    __syncwarp();  // (the scales of the slot that is filled next have been read)
    fill(slot ^ 1);
    const Tensor& t = a.tensor[now.tensor];
    const long long at = now.at<BITS>(a);
    const uint32_t from = slot0 + (unsigned)slot * kSlot;
    if (BITS == 8) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
    }
    if (whole<BITS>(a, now.tensor, t, at)) {
      const Lane<P, G, MASTER> l(t, at, BITS / 8);
#pragma unroll(BITS == 8 ? kParts : 1)
      for (int k = 0; k < kParts; ++k)
        update_block<P, G, BITS, MASTER, true>(a, s, l, k, kLane, from + k * S::kBytes);
    } else {
      update_rest<P, G, BITS, MASTER>(a, s, t, at, from);
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
        decode_m(load_codes(static_cast<const char*>(t.m) + i0, n, vec), t.mScale[at / kBlock], x);
        Eight<float>::store(static_cast<float*>(t.param) + i0, n, vec, x);
      }
      if (t.master) {
        decode_v(load_codes(static_cast<const char*>(t.v) + i0, n, vec), t.vScale[at / kBlock], x);
        Eight<float>::store(t.master + i0, n, vec, x);
      }
    }
  }
}

// ------------------------------------------------------------- host side
struct AdamKernel {
  const void* fn;
  size_t smem;
};
template <typename P, typename G, bool MASTER>
AdamKernel kernel_of(int bits) {
  using Read = typename Select<MASTER, float, P>::type;
  if (bits == 32) return {(const void*)adamw_kernel<P, G, 32, MASTER>, 0};
  return {(const void*)adamw_kernel<P, G, 8, MASTER>,
          (size_t)kWarps * kAhead * kParts * Slot<Read, G>::kBytes};
}
template <typename P, typename G>
AdamKernel kernel_of(int bits, bool master) {
  if constexpr (!std::is_same<P, float>::value)
    if (master) return kernel_of<P, G, true>(bits);
  return kernel_of<P, G, false>(bits);
}
template <typename P>
AdamKernel kernel_of(int gradDtype, int bits, bool master) {
  return gradDtype == VR_FLOAT32   ? kernel_of<P, float>(bits, master)
         : gradDtype == VR_FLOAT16 ? kernel_of<P, __half>(bits, master)
                                   : kernel_of<P, __nv_bfloat16>(bits, master);
}

constexpr size_t kMostSize = (size_t)1 << 40;

// The buffers of a call: extents, and whether each is written.
struct Spans {
  std::vector<OpSpan> v;
  void add(const void* p, size_t bytes, bool write) {
    if (bytes && p) v.push_back({(uintptr_t)p, (uintptr_t)p + bytes, write});
  }
};

// Launches `fn` over the tensors, kTensors at a time.  `fill` writes tensor i
// and returns the address bits of its rows.
template <class Fill>
vr_result_t over_tensors(const AdamKernel& k, AdamArgs& a, const size_t* sizes, int count,
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
        op_launch(k.fn, dim3((unsigned)std::min<long long>(chunks, dev.sms * 8LL)), dim3(kThreads),
                  args, k.smem, stream);
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
      !std::isfinite(eps) || (eps > 0.0f && eps < FLT_MIN) || ((uintptr_t)control & 3) ||
      (!control && (!std::isfinite(lr) || !std::isfinite(gradScale) || step < 1)) ||
      !std::isfinite(weightDecay))
    return VR_ERR_INVALID_ARGUMENT;
  const size_t SE = few ? 1 : 4;
  try {
    Spans spans;
    spans.v.reserve((size_t)count * 7 + 1);
    for (int i = 0; i < count; ++i) {
      const size_t n = sizes[i];
      if (n > kMostSize) return VR_ERR_INVALID_ARGUMENT;
      if (!n) continue;
      if (!params[i] || !grads[i] || !m[i] || !v[i] || (few && (!mScales[i] || !vScales[i])) ||
          (masters && !masters[i]) || (uintptr_t)params[i] & (E - 1) ||
          (uintptr_t)grads[i] & (GE - 1) || ((uintptr_t)m[i] | (uintptr_t)v[i]) & (SE - 1) ||
          (few && ((uintptr_t)mScales[i] | (uintptr_t)vScales[i]) & 3) ||
          (masters && (uintptr_t)masters[i] & 3))
        return VR_ERR_INVALID_ARGUMENT;
    }
    auto list = [&](auto p, size_t elem, bool write) {
      for (int i = 0; p && i < count; ++i) spans.add(p[i], sizes[i] * elem, write);
    };
    auto scales = [&](auto p) {
      for (int i = 0; p && i < count; ++i) spans.add(p[i], (sizes[i] + kBlock - 1) / kBlock * 4, true);
    };
    list(params, E, true);
    list(grads, GE, false);
    list(m, SE, true);
    list(v, SE, true);
    scales(mScales);
    scales(vScales);
    list(masters, 4, true);
    spans.add(control, 12, false);
    if (!op_spans_ok(spans.v.data(), spans.v.size())) return VR_ERR_INVALID_ARGUMENT;
    OpDevice dev;
    vr_result_t e = op_device(&dev);
    if (e != VR_SUCCESS) return e;
    if ((e = op_reachable(spans.v.data(), spans.v.size(), dev.device)) != VR_SUCCESS) return e;
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
    a.down = (float)std::sqrt(1.0 / -std::expm1((double)step * log2));
    a.decay = (float)((double)lr * (double)weightDecay);
    a.control = control;
    a.seedKey = mix(mix((unsigned)seed) ^ (unsigned)(seed >> 32));
    a.step = step;
    const AdamKernel k = dtype == VR_FLOAT32   ? kernel_of<float>(gradDtype, stateBits, false)
                         : dtype == VR_FLOAT16 ? kernel_of<__half>(gradDtype, stateBits, masters)
                                               : kernel_of<__nv_bfloat16>(gradDtype, stateBits,
                                                                          masters);
    if (k.smem && (e = gemm_prepare(k.fn, dev.device, k.smem)) != VR_SUCCESS) return e;
    return over_tensors(k, a, sizes, count, dev, stream, [&](int i, Tensor* t) {
      *t = {params[i],
            grads[i],
            m[i],
            v[i],
            few ? mScales[i] : nullptr,
            few ? vScales[i] : nullptr,
            masters ? masters[i] : nullptr,
            0,
            0};
      return !((uintptr_t)params[i] & (8 * E - 1)) && !((uintptr_t)grads[i] & (8 * GE - 1)) &&
             !(((uintptr_t)m[i] | (uintptr_t)v[i]) & (8 * SE - 1)) &&
             !((uintptr_t)t->master & 31);
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
      const size_t n = sizes[i];
      if (n > kMostSize) return VR_ERR_INVALID_ARGUMENT;
      auto bad = [&](const void* const* codes, const float* const* scales, float* const* out) {
        return n && out &&
               (!codes[i] || !scales[i] || !out[i] ||
                ((uintptr_t)scales[i] | (uintptr_t)out[i]) % 4);
      };
      if (bad(m, mScales, mValues) || bad(v, vScales, vValues)) return VR_ERR_INVALID_ARGUMENT;
    }
    auto list = [&](auto p, auto out, size_t elem, size_t per, bool write) {
      for (int i = 0; out && i < count; ++i)
        if (sizes[i]) spans.add(p[i], (sizes[i] + per - 1) / per * elem, write);
    };
    list(m, mValues, 1, 1, false);
    list(mScales, mValues, 4, kBlock, false);
    list(mValues, mValues, 4, 1, true);
    list(v, vValues, 1, 1, false);
    list(vScales, vValues, 4, kBlock, false);
    list(vValues, vValues, 4, 1, true);
    if (!op_spans_ok(spans.v.data(), spans.v.size())) return VR_ERR_INVALID_ARGUMENT;
    OpDevice dev;
    vr_result_t e = op_device(&dev);
    if (e != VR_SUCCESS) return e;
    if ((e = op_reachable(spans.v.data(), spans.v.size(), dev.device)) != VR_SUCCESS) return e;
    AdamArgs a;
    return over_tensors({(const void*)adamw_values_kernel, 0}, a, sizes, count, dev, stream,
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
