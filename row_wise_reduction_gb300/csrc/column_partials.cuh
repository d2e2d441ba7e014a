// Column sums left as P partial rows: out0[c], for the columns below N0, and
// out1[c - N0] for those from there on, are the sums of part[p * pitch + c] over
// p. A CTA takes 32 columns; thread (x, y) adds the partials p = y, y + 32, ... of
// column x in order, then the 32 sums are added in order of y: a fixed order, so
// the result does not depend on scheduling. May be launched while the kernel
// that leaves the partials drains (it waits for that one's end).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rowops_launch.h"

namespace rowops {

static __global__ void __launch_bounds__(1024) column_partials_kernel(const float* part, int P, int64_t pitch,
                                                                      int64_t N, int64_t N0, float* out0,
                                                                      float* out1) {
    __shared__ float acc[32][33];
    const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.f;
    if (c < N) {
#pragma unroll 16
        for (int p = threadIdx.y; p < P; p += 32) s += part[p * pitch + c];
    }
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < N) {
        float t = 0.f;
#pragma unroll 8
        for (int y = 0; y < 32; ++y) t += acc[y][threadIdx.x];
        if (c < N0) out0[c] = t;
        else out1[c - N0] = t;
    }
}

// out1 NULL: one set of N0 columns; else two.
inline cudaError_t reduce_partials(const float* part, int64_t P, int64_t pitch, int64_t N0, float* out0, float* out1,
                                   const LaunchCfg& cfg) {
    const int64_t N = out1 ? 2 * N0 : N0;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(unsigned((N + 31) / 32));
    lc.blockDim = dim3(32, 32);
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, column_partials_kernel, part, int(P), pitch, N, N0, out0, out1);
}

}  // namespace rowops
