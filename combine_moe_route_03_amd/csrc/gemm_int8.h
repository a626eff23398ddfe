// gemm_int8.h -- pieces shared by the grouped products of 8-bit integer operands.
#pragma once

#include "device.h"
#include "gemm_fp8.h"

namespace moe {

// One 16 x 16 x 64 product of 8-bit integers added to 32-bit sums, exact: lane l holds 16
// columns from 16 (l / 16) on of row l % 16 of each operand, and of the result rows
// 4 (l / 16) + 0..3 of the first operand, column l % 16 (the second's row).
__device__ __forceinline__ i32x4 mfma_int8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// A sum with the scales of its row and its column, each product rounded to fp32.
__device__ __forceinline__ float scaled(int sum, float row_scale, float col_scale) {
  return (float)sum * row_scale * col_scale;
}

}  // namespace moe
