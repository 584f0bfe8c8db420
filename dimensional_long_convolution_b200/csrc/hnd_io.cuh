// hnd_io.cuh -- activation types of the block operators: fp32 arithmetic on
// fp32 or bf16 storage, each stored value rounded once (to nearest even).
#pragma once

#include <cuda_bf16.h>

#include "hnd_bounds.cuh"

namespace hnd {

__device__ __forceinline__ float ld1(const float* p) { return *HND_G(p); }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*HND_G(p)); }
__device__ __forceinline__ void st1(float* p, float v) { *HND_G(p) = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *HND_G(p) = __float2bfloat16_rn(v); }

}  // namespace hnd
