// Shared by the kernels of moe_int8_matmul.
#pragma once

#include <cuda_runtime.h>

#include "ops.h"

namespace moe {

// Tiles of 16 weight rows and 8 or 16 tokens; right for every size, fast for a few rows a group.
cudaError_t launch_int8_few(const moe_int8_matmul_args& a, cudaStream_t s);

// A value of the result from its integer sum, rounded to fp32.
__device__ __forceinline__ float int8_scaled(float c, float b_scale, float a_scale) { return __fmul_rn(__fmul_rn(c, b_scale), a_scale); }

}  // namespace moe
