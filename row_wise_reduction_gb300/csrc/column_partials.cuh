// Column sums left as P partial rows of N floats: out[c] = the sum of part[p *
// pitch + c] over p. A CTA takes 32 columns; thread (x, y) adds the partials p
// = y, y + 32, ... of column x in order, then the 32 sums are added in order of
// y: a fixed order, so the result does not depend on scheduling.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rowops {

static __global__ void __launch_bounds__(1024) column_partials_kernel(const float* part, int P, int64_t pitch,
                                                                      int64_t N, float* out) {
    __shared__ float acc[32][33];
    const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.f;
    if (c < N)
        for (int p = threadIdx.y; p < P; p += 32) s += part[p * pitch + c];
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < N) {
        float t = 0.f;
#pragma unroll 8
        for (int y = 0; y < 32; ++y) t += acc[y][threadIdx.x];
        out[c] = t;
    }
}

}  // namespace rowops
