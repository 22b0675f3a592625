// Host side of the tensor-core products (gemm.cuh): operands and launches.
#pragma once

#include <cuda.h>

#include "ops.h"

namespace vr {

// An operand of `batch` matrices of `rows` rows of `inner` 16-bit elements,
// fetched in boxes of 64 elements by boxRows rows into 128-byte swizzled
// shared memory.  `p` and both strides are multiples of 16 bytes.
// (boxCols = 32: boxes of 32 elements, 64-byte swizzled.)
vr_result_t gemm_operand(CUtensorMap* map, const void* p, bool bf16, size_t inner, size_t rows,
                         size_t batch, size_t rowStride, size_t batchStride, int boxRows,
                         int boxCols = 64);
// Allows `fn` its dynamic shared memory (once per kernel and device).
vr_result_t gemm_prepare(const void* fn, int device, size_t smem);

}  // namespace vr
