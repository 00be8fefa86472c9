// sta_ops.cuh -- device helpers of the plan-less operators: e4m3 conversions.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace sta {
namespace ops {

// Two floats to e4m3, `lo` in bits 0-7: to nearest even, magnitudes above 448 to 448, NaN kept.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes (bits 0-7, 8-15) to fp16, exactly.
__device__ __forceinline__ uint32_t e4m3_half2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}
// Four codes to floats.
__device__ __forceinline__ void e4m3_floats(uint32_t u, float& a, float& b, float& c, float& d) {
    const uint32_t lo = e4m3_half2(uint16_t(u & 0xffffu)), hi = e4m3_half2(uint16_t(u >> 16));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    a = x.x;
    b = x.y;
    c = y.x;
    d = y.y;
}

}  // namespace ops
}  // namespace sta
