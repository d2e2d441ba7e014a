// A thread's ring of data on its way into shared memory: D steps of N words (of 16
// bytes, or 4), in slots of its own, so no barrier stands between a copy and its use and what is
// in flight takes no registers.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rowops {

// BYTES (4, 8 or 16) from global to shared memory, both aligned to it
template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* global) {
    const unsigned to = unsigned(__cvta_generic_to_shared(smem));
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(to), "l"(global) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(global), "n"(BYTES) : "memory");
}

// 16 bytes under an L2 policy
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void copy_async16(void* smem, const void* global, uint64_t policy) {
    const unsigned to = unsigned(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2;" ::"r"(to), "l"(global),
                 "l"(policy)
                 : "memory");
}

// the first `bytes` of 16 (no others are read), zeros behind them
__device__ __forceinline__ void copy_async_part(void* smem, const void* global, unsigned bytes) {
    const unsigned to = unsigned(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(to), "l"(global), "r"(bytes)
                 : "memory");
}

template <int D, int N, int THREADS, typename Word = uint4>
struct Ring {
    Word* at;  // [D][N][THREADS], this thread's
    int in = 0, out = 0;
    __device__ __forceinline__ explicit Ring(Word* smem) : at(smem + threadIdx.x) {}
    __device__ __forceinline__ void ask(int n, const void* p) {
        copy_async<sizeof(Word)>(at + (in * N + n) * THREADS, p);
    }
    __device__ __forceinline__ void ask_part(int n, const void* p, unsigned bytes) {
        copy_async_part(at + (in * N + n) * THREADS, p, bytes);
    }
    // the step's copies are all asked for (or there were none)
    __device__ __forceinline__ void asked() {
        asm volatile("cp.async.commit_group;" ::: "memory");
        in = in + 1 == D ? 0 : in + 1;
    }
    // the oldest step's copies are here, D - 1 later ones may not be
    __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory"); }
    __device__ __forceinline__ Word get(int n) const { return at[(out * N + n) * THREADS]; }
    __device__ __forceinline__ void done() { out = out + 1 == D ? 0 : out + 1; }
};

}  // namespace rowops
