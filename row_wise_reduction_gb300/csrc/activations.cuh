// The activations of the fused normalisations and their derivatives, on pairs with
// packed arithmetic: none, SiLU, and the two GELUs of the LayerNorm kernels.
#pragma once

#include "ln_gelu_kernels.cuh"
#include "rowops.h"

namespace rowops {

// the nearest to z within bound of 0; a NaN stays
__device__ __forceinline__ float within(float z, float bound) {
    float y;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(z), "f"(bound));
    return y;
}

// e = 2^a and q = 1 / (1 + e) of two values from one reciprocal, that of the
// product (1 + e_x) (1 + e_y). a is kept to 84 (a NaN as well, which would pass to the
// other value; the callers' z carries it on), so q stays at 2^-84 where it is smaller.
// Where the product passes 2^126, its reciprocal and with it both q are 0: one is at
// 2^-84 there and the other below 2^-42. What is built from q, z q or z q (1 - q), is then
// off by at most |z| 2^-84 (5e-6 at |z| = 10^20) or 7e-12. One and a half special-function
// results a value instead of two, which an SM makes 16 of a cycle: a pass that reads
// from L2 and the backward pass, which evaluates the slope twice, would be bound by them.
__device__ __forceinline__ float2 sigmoids2(float2 a, float2& e) {
    e = make_float2(ex2_approx(fminf(a.x, 84.f)), ex2_approx(fminf(a.y, 84.f)));
    const float2 d = f2_add(e, f2(1.f));
    const float r = rcp_approx(d.x * d.y);
    return f2_mul(make_float2(d.y, d.x), f2(r));
}

// z for the slope of the tanh form: within 7.4 of 0, where a is 58.8 (and -58.8: e =
// 2^-58.8). The slope is within 2.1e-16 of 0 (or 1) there and beyond, and its cubic
// factor z (1 + 3 k1 z^2) stays below 100: kept at large z it would make of q's 2^-84,
// or of e = 0 once it overflows, any number or a NaN.
__device__ __forceinline__ float2 tanh_slope_range(float2 z) {
    return make_float2(within(z.x, 7.4f), within(z.y, 7.4f));
}

template <int ACT>
__device__ __forceinline__ float2 act_of2(float2 z) {
    if constexpr (ACT == ROWOPS_ACT_SILU) {
        float2 e;
        return f2_mul(z, sigmoids2(f2_mul(z, f2(-kLog2eF)), e));
    } else if constexpr (ACT == ROWOPS_ACT_GELU) {
        return gelu_erf2(z);
    } else if constexpr (ACT == ROWOPS_ACT_GELU_TANH) {
        return gelu_tanh_approx2(z);
    } else {
        return z;
    }
}

// With q = 1 / (1 + e), 1 - q = e q (no cancellation):
//   SiLU   q + z q (1 - q)
//   tanh   q + z q (1 - q) 2 du/dz,  q = 0.5 (1 + tanh u), du/dz = k0 (1 + 3 k1 z^2)
//   exact  Phi(z) + z phi(z), Phi by the forward's fit
template <int ACT>
__device__ __forceinline__ float2 act_grad2(float2 z) {
    if constexpr (ACT == ROWOPS_ACT_SILU) {
        float2 e;
        const float2 q = sigmoids2(f2_mul(z, f2(-kLog2eF)), e);
        return f2_fma(f2_mul(z, q), f2_mul(e, q), q);
    } else if constexpr (ACT == ROWOPS_ACT_GELU) {
        using F = GeluErfFit;
        const float2 z2 = f2_mul(z, z);
        float2 p = f2_fma(z2, f2(F::q6), f2(F::q5));
        p = f2_fma(z2, p, f2(F::q4));
        p = f2_fma(z2, p, f2(F::q3));
        p = f2_fma(z2, p, f2(F::q2));
        p = f2_fma(z2, p, f2(F::q1));
        p = f2_fma(z2, p, f2(F::q0));
        const float2 h = f2_mul(z2, f2(-0.5f * kLog2eF));
        const float2 phi = f2_mul(make_float2(ex2_approx(h.x), ex2_approx(h.y)), f2(0.3989422804014327f));
        float2 e;
        return f2_fma(z, phi, sigmoids2(f2_mul(p, z), e));
    } else if constexpr (ACT == ROWOPS_ACT_GELU_TANH) {
        constexpr float c0 = float(-2.0 * 0.79788456 * kLog2e), c1 = float(-2.0 * 0.79788456 * 0.044715 * kLog2e);
        constexpr float d0 = float(2.0 * 0.79788456), d1 = float(6.0 * 0.79788456 * 0.044715);
        z = tanh_slope_range(z);
        const float2 z2 = f2_mul(z, z);
        float2 e;
        const float2 q = sigmoids2(f2_mul(f2_fma(z2, f2(c1), f2(c0)), z), e);
        return f2_fma(f2_mul(f2_mul(e, q), q), f2_mul(z, f2_fma(z2, f2(d1), f2(d0))), q);
    } else {
        return f2(1.f);
    }
}

}  // namespace rowops
