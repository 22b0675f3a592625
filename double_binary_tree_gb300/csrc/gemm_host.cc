// Tensor maps for the matrix products of the training operators.
#include "gemm_host.h"

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>
#include <set>
#include <utility>

namespace vr {
namespace {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, found through the runtime (the library links no
// driver library, so that it loads where there is none).
EncodeFn encoder() {
  static std::atomic<EncodeFn> found{nullptr};
  EncodeFn f = found.load();
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeFn>(p);
  found.store(f);
  return f;
}

std::mutex g_mu;
std::set<std::pair<const void*, int>> g_prepared;

}  // namespace

vr_result_t gemm_operand(CUtensorMap* map, const void* p, bool bf16, size_t inner, size_t rows,
                         size_t batch, size_t rowStride, size_t batchStride, int boxRows,
                         int boxCols) {
  const EncodeFn encode = encoder();
  if (!encode) return VR_ERR_CUDA;
  const cuuint64_t dims[3] = {inner, rows, batch};
  const cuuint64_t strides[2] = {rowStride, batchStride};
  const cuuint32_t box[3] = {(cuuint32_t)boxCols, (cuuint32_t)boxRows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = encode(
      map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
      const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
      boxCols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? VR_SUCCESS : VR_ERR_CUDA;
}

vr_result_t gemm_prepare(const void* fn, int device, size_t smem) {
  try {
    std::lock_guard<std::mutex> g(g_mu);
    const auto key = std::make_pair(fn, device);
    if (g_prepared.count(key)) return VR_SUCCESS;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
      return VR_ERR_CUDA;
    g_prepared.insert(key);
    return VR_SUCCESS;
  } catch (...) {  // no host memory for the entry
    return VR_ERR_INTERNAL;
  }
}

}  // namespace vr
