// RMSNorm (with the residual's addition) and its result in 8 bits with scales:
//   s = x + residual as the I/O type stores it;  y = s w / sqrt(mean(s^2) + eps)
//   scale = max(max|y| / 448, 2^-126) over a row or `group` columns;  q = e4m3(y / scale)
// y itself is never rounded nor stored. e4m3 has 448 as its largest number.
#include <algorithm>

#include "e4m3.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace rowops {
namespace {

// One CTA per row, any length and layout. Pass 1 forms s (writing residual_out)
// and the sum of squares; then a warp takes a group at a time, its largest
// magnitude and its quotients (the whole row is one group of the CTA).
constexpr int kLoopBlock = 512;

template <typename T, bool RES>
__global__ void __launch_bounds__(kLoopBlock) rms_quant_looped_kernel(const QuantArgs a) {
    using E = Elem<T>;
    __shared__ float red[2][2][kLoopBlock / 32];  // alternate per row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* w = static_cast<const T*>(a.w);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        const T* x = static_cast<const T*>(a.x) + row * a.ld;
        const T* src = RES ? static_cast<const T*>(a.residual_out) + row * a.ld : x;
        uint8_t* q = static_cast<uint8_t*>(a.q) + row * a.ldq;
        float sum = 0.f, top = 0.f;
        for (int64_t c = threadIdx.x; c < a.N; c += kLoopBlock) {
            float s = E::load(x + c);
            if constexpr (RES) {
                s = E::round(s + E::load(static_cast<const T*>(a.residual) + row * a.ld + c));
                E::store(static_cast<T*>(a.residual_out) + row * a.ld + c, s);
            }
            sum = fmaf(s, s, sum);
            if (a.group == a.N) top = max_nan(top, fabsf(w ? s * E::load(w + c) : s));
        }
        sum = group_reduce<kLoopBlock>(sum, red[turn][0], OpSum());
        const float inv = rsqrtf(sum / float(a.N) + a.eps);
        if (a.group == a.N) {
            top = group_reduce<kLoopBlock>(top, red[turn][1], OpMaxNan());
            const float scale = quant_scale(top * inv);
            if (threadIdx.x == 0) a.scales[row] = scale;
            const float f = 1.f / scale;  // (apart from inv: the product of the two may overflow)
            for (int64_t c = threadIdx.x; c < a.N; c += kLoopBlock) {
                const float s = E::load(src + c);
                q[c] = to_e4m3(s * (w ? E::load(w + c) : 1.f) * inv * f);
            }
            continue;
        }
        const int64_t groups = (a.N + a.group - 1) / a.group;
        for (int64_t g = warp; g < groups; g += kLoopBlock / 32) {
            const int64_t c0 = g * a.group, c1 = c0 + a.group < a.N ? c0 + a.group : a.N;
            top = 0.f;
            for (int64_t c = c0 + lane; c < c1; c += 32)
                top = max_nan(top, fabsf(E::load(src + c) * (w ? E::load(w + c) : 1.f)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float scale = quant_scale(top * inv), f = 1.f / scale;
            if (lane == 0) a.scales[row * groups + g] = scale;
            for (int64_t c = c0 + lane; c < c1; c += 32)
                q[c] = to_e4m3(E::load(src + c) * (w ? E::load(w + c) : 1.f) * inv * f);
        }
    }
}

template <typename T>
cudaError_t launch(const QuantArgs& a, bool, const LaunchCfg& cfg) {
    auto k = a.residual ? rms_quant_looped_kernel<T, true> : rms_quant_looped_kernel<T, false>;
    const int grid = grid_for(reinterpret_cast<const void*>(k), kLoopBlock, 0, a.M, cfg);
    k<<<grid, kLoopBlock, 0, cfg.stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

QuantLaunch rms_quant_f32() { return launch<float>; }
QuantLaunch rms_quant_bf16() { return launch<bf16_t>; }

}  // namespace rowops
