// An fp32 value as three bf16 parts, which the tensor cores multiply exactly.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace conv2d_gb300 {

// The bf16 nearest to x (toward zero where that would overflow), and what is
// left for the next part: three parts hold all 24 bits of a float.
__device__ __forceinline__ float part_of(float x) {
    __nv_bfloat16 a = __float2bfloat16_rn(x);
    if (__hisinf(a) && !isinf(x)) a = __float2bfloat16_rz(x);
    return __bfloat162float(a);
}
__device__ __forceinline__ float rest_of(float x, float part) { return isfinite(part) ? x - part : 0.f; }
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
    p[0] = part_of(x);
    x = rest_of(x, p[0]);
    p[1] = part_of(x);
    p[2] = part_of(rest_of(x, p[1]));
}

}  // namespace conv2d_gb300
