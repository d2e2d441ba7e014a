// 8-bit floating point (e4m3: 4 exponent bits, 3 of fraction, no infinities, 448
// the largest) and the scales that go with it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rowops {

// two numbers, `lo` in the lower byte: nearest even, 448 beyond it, NaN stays
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint8_t to_e4m3(float v) { return uint8_t(to_e4m3x2(v, 0.f)); }

// The scale that takes `top` to 448: at least the smallest normal number, so that
// its reciprocal is finite. NaN stays.
__device__ __forceinline__ float quant_scale(float top) {
    const float s = top * (1.f / 448.f);
    return s < 0x1p-126f ? 0x1p-126f : s;
}

}  // namespace rowops
