// The activations of the fused normalisations and their derivatives, one value
// at a time: none, SiLU, and the two GELUs of the LayerNorm kernels. One exp2
// and one reciprocal each (the exact GELU's derivative: two exp2).
#pragma once

#include "ln_gelu_kernels.cuh"
#include "rowops.h"

namespace rowops {

// 1 / (1 + 2^a)
__device__ __forceinline__ float sigmoid2(float a) { return rcp_approx(1.f + ex2_approx(a)); }

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == ROWOPS_ACT_SILU) return z * sigmoid2(-kLog2eF * z);
    else if constexpr (ACT == ROWOPS_ACT_GELU) return gelu_erf(z);
    else if constexpr (ACT == ROWOPS_ACT_GELU_TANH) return gelu_tanh_approx(z);
    else return z;
}

// With q = 1 / (1 + e), 1 - q = e q (no cancellation); e is kept from
// overflowing, where q = 0 would meet an infinite e.
//   SiLU   q + z q (1 - q)
//   tanh   q + z q (1 - q) 2 du/dz,  q = 0.5 (1 + tanh u), du/dz = k0 (1 + 3 k1 z^2)
//   exact  Phi(z) + z phi(z), Phi by the forward's fit
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
    if constexpr (ACT == ROWOPS_ACT_SILU) {
        const float e = ex2_approx(fminf(-kLog2eF * z, 126.f)), q = rcp_approx(1.f + e);
        return fmaf(z * q, e * q, q);
    } else if constexpr (ACT == ROWOPS_ACT_GELU) {
        using F = GeluErfFit;
        const float z2 = z * z;
        float p = fmaf(z2, F::q6, F::q5);
        p = fmaf(z2, p, F::q4);
        p = fmaf(z2, p, F::q3);
        p = fmaf(z2, p, F::q2);
        p = fmaf(z2, p, F::q1);
        p = fmaf(z2, p, F::q0);
        const float phi = 0.3989422804014327f * ex2_approx(-0.5f * kLog2eF * z2);
        return fmaf(z, phi, sigmoid2(p * z));
    } else if constexpr (ACT == ROWOPS_ACT_GELU_TANH) {
        constexpr float c0 = float(-2.0 * 0.79788456 * kLog2e), c1 = float(-2.0 * 0.79788456 * 0.044715 * kLog2e);
        constexpr float d0 = float(2.0 * 0.79788456), d1 = float(6.0 * 0.79788456 * 0.044715);
        const float z2 = z * z;
        const float e = ex2_approx(fminf(fmaf(c1, z2, c0) * z, 126.f)), q = rcp_approx(1.f + e);
        return fmaf((e * q) * q, z * fmaf(d1, z2, d0), q);
    } else {
        return 1.f;
    }
}

}  // namespace rowops
