// Philox4x32-10, the counter-based generator of Salmon, Moraes, Dror and Shaw,
// "Parallel Random Numbers: As Easy as 1, 2, 3" (SC 2011): ten rounds of two
// 32 x 32 -> 64 bit products on a 128-bit counter, keyed with 64 bits. A block
// of four words depends on its counter and key alone, so any thread can make
// any block at any time and nothing has to be stored.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rowops {

// The rounds' keys: key + round (golden ratio, sqrt(3) - 1), computed once on the host
// and read from the kernel's arguments, so a round is four instructions.
struct PhiloxKeys {
    uint2 k[10];
    __host__ explicit PhiloxKeys(uint64_t key) {
        for (unsigned r = 0; r < 10; ++r) {
            k[r].x = uint32_t(key) + r * 0x9E3779B9u;
            k[r].y = uint32_t(key >> 32) + r * 0xBB67AE85u;
        }
    }
};

__device__ __forceinline__ uint4 philox4x32_10(uint4 c, const PhiloxKeys& keys) {
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t a = uint64_t(0xD2511F53u) * c.x, b = uint64_t(0xCD9E8D57u) * c.z;
        c = make_uint4(uint32_t(b >> 32) ^ c.y ^ keys.k[round].x, uint32_t(b),
                       uint32_t(a >> 32) ^ c.w ^ keys.k[round].y, uint32_t(a));
    }
    return c;
}

}  // namespace rowops
