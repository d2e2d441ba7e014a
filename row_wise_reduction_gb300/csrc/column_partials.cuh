// Column sums left as P partial rows: out0[c], for the columns below N0, and
// out1[c - N0] for those from there on, are the sums of part[p * pitch + c] over
// p. A CTA takes W columns by H = 1024 / W threads; thread (x, y) adds the partials
// p = y, y + H, ... of column x in order, eight of them on their way, then the H sums
// are added in order of y: a fixed order, so the result does not depend on
// scheduling. W is 32 (whole lines), and 8 (whole sectors) where that leaves most
// SMs without a CTA. May be launched while the kernel that leaves the partials
// runs (it waits for that one's end). With one partial at a time 152 x 8192 took
// 5.6 us and 640 x 640 8.6 us alone on the GPU.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rowops_launch.h"

namespace rowops {

template <int W>
static __global__ void __launch_bounds__(1024) column_partials_kernel(const float* part, int P, int64_t pitch,
                                                                      int64_t N, int64_t N0, float* out0,
                                                                      float* out1) {
    constexpr int H = 1024 / W, U = 8;
    __shared__ float acc[H][W + 1];
    const int x = threadIdx.x % W, y = threadIdx.x / W;
    const int64_t c = int64_t(blockIdx.x) * W + x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.f;
    if (c < N) {
        for (int p0 = y; p0 < P; p0 += U * H) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = p0 + u * H < P ? part[int64_t(p0 + u * H) * pitch + c] : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) s += v[u];
        }
    }
    acc[y][x] = s;
    __syncthreads();
    if (y == 0 && c < N) {
        float t = 0.f;
#pragma unroll 16
        for (int k = 0; k < H; ++k) t += acc[k][x];
        if (c < N0) out0[c] = t;
        else out1[c - N0] = t;
    }
}

// out1 NULL: one set of N0 columns; else two.
inline cudaError_t reduce_partials(const float* part, int64_t P, int64_t pitch, int64_t N0, float* out0, float* out1,
                                   const LaunchCfg& cfg) {
    const int64_t N = out1 ? 2 * N0 : N0;
    cudaLaunchConfig_t lc = {};
    const int W = N > 32 * 76 ? 32 : 8;
    lc.gridDim = dim3(unsigned((N + W - 1) / W));
    lc.blockDim = dim3(1024);
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, W == 32 ? column_partials_kernel<32> : column_partials_kernel<8>, part, int(P), pitch, N, N0, out0, out1);
}

}  // namespace rowops
