// Rows of 16-bit matrices as the products' epilogues store them, and copies of
// rows that tensor copies cannot read where they lie.
#pragma once

#include "gemm.cuh"

namespace vr {
namespace {

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)Ty<T>::narrow(a) | (uint32_t)Ty<T>::narrow(b) << 16;
}

// Consecutive 16-bit values of one row.  `align`: bytes that a store may
// take (2, 16 or 32); a warp's rows are 32 lines apart, so half as many
// stores are half the time.
template <typename T, int N>
__device__ __forceinline__ void store_row(T* out, const float (&v)[N], int cols, int align) {
  typename Ty<T>::Bits* o = reinterpret_cast<typename Ty<T>::Bits*>(out);
  if (align >= 16 && cols >= N) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    if (align == 32) {
#pragma unroll
      for (int i = 0; i < N / 2; i += 8)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + 2 * i),
                     "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                     "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                     : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; i += 4)
        *reinterpret_cast<uint4*>(o + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cols) o[i] = Ty<T>::narrow(v[i]);
  }
}

// Rows of `cols` elements between a dense buffer of any alignment and one
// whose rows are whole sectors (ld): in, with zeros after the last column, or
// out.  A warp takes a row, so that its accesses are one run of bytes.
struct PadArgs {
  const uint16_t* src;
  long long stride, rows;
  int cols, ld;
  uint16_t* dst;
  // in: batches of so many rows, of which those with a positive count are copied
  // (null: all)
  const int* counts;
  long long perCount;
};
__global__ void __launch_bounds__(256) pad_kernel(const __grid_constant__ PadArgs a) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  for (long long r = (long long)blockIdx.x * 8 + threadIdx.x / 32; r < a.rows;
       r += (long long)gridDim.x * 8) {
    if (a.counts && a.counts[r / a.perCount] <= 0) continue;
    const uint16_t* in = a.src + r * a.stride;
    uint4* out = reinterpret_cast<uint4*>(a.dst + r * a.ld);
#pragma unroll 2
    for (int u = lane; u < a.ld / 8; u += 32) {
      alignas(16) uint16_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = u * 8 + i < a.cols ? in[u * 8 + i] : (uint16_t)0;
      out[u] = *reinterpret_cast<const uint4*>(v);
    }
  }
}
__global__ void __launch_bounds__(256) unpad_kernel(const __grid_constant__ PadArgs a) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  for (long long r = (long long)blockIdx.x * 8 + threadIdx.x / 32; r < a.rows;
       r += (long long)gridDim.x * 8) {
    const uint16_t* in = a.src + r * a.ld;
    uint16_t* out = a.dst + r * a.cols;
    const int odd = (int)((uintptr_t)out >> 1 & 1);  // 32-bit stores begin after it
    const int words = (a.cols - odd) / 2;
    if (lane == 0 && odd) out[0] = in[0];
    if (lane == 1 && odd + 2 * words < a.cols) out[a.cols - 1] = in[a.cols - 1];
#pragma unroll 4
    for (int w = lane; w < words; w += 32) {
      const int c = odd + 2 * w;
      *reinterpret_cast<uint32_t*>(out + c) = (uint32_t)in[c] | (uint32_t)in[c + 1] << 16;
    }
  }
}

inline size_t up(size_t n, size_t to) { return (n + to - 1) / to * to; }

inline bool packed_rows(const void* p, size_t stride) {
  return ((uintptr_t)p & 15) == 0 && stride % 8 == 0;
}

}  // namespace
}  // namespace vr
