// Attention over a paged cache, fp32 (paged_kernels.cuh), by fused multiply-adds: G heads
// take 2 G operations for each element read, 16 cycles a position, head dimension of 128 and 8
// heads, where the memory takes 44 for its 1 KB. Few warps an SM and chains of shuffles between the two
// products leave it bound by latency all the same: one sequence of 32768 positions, 8 heads of 128 with 4 queries
// each, 57.9 us (39.5 at the rate of a copy); 9 sequences, a window of 1999, 3 heads of 80 with 5 each, 20.6 us (3.9).
#pragma once

#include "paged_kernels.cuh"

namespace rowops {

// A warp's state for a unit of at most G heads. Pieces of 8 positions. For the scores lane
// 8 p + t has position t and every fourth vector of the row, from p on; the quarters are
// added up so that it keeps G / 4 heads. For the values a lane has vectors of the columns (of 64
// columns half a warp has them, and each half four positions).
template <int DT, int G>
struct PagedF32 {
    using T = float;
    static constexpr int kRows = G, kD = DT, kOwn = G;
    using Ring = PagedRing<T, DT, kRows>;
    static constexpr int kTokens = Ring::kShape.tokens, kPitch = Ring::kShape.joined, kScratch = Ring::kShape.scratch;
    static_assert(kTokens == 8 && kPitch == DT);
    static constexpr int kVectors = DT / 4, kHalves = kVectors <= 16 ? 2 : 1, kEach = (kVectors + 31) / 32;
    static constexpr int kHeads = G > 4 ? G / 4 : 1;
    float *q, *weights, *keeps;  // [G][DT] of the CTA; [G][8] and [G] of the warp
    float o[G][kEach][4], m[kHeads], l[kHeads];

    __device__ __forceinline__ explicit PagedF32(float* scratch) {
        const int warp = threadIdx.x >> 5;
        q = scratch;
        weights = scratch + G * DT + warp * G * 8;
        keeps = scratch + G * DT + kPagedWarps * G * 8 + warp * G;
    }
    __device__ __forceinline__ static int lane() { return threadIdx.x & 31; }
    __device__ __forceinline__ static int row(int i) { return i; }
    // the first of the heads whose scores this lane keeps
    __device__ __forceinline__ static int own() {
        const int p = lane() >> 3;
        return G >= 4 ? p * kHeads : 0;
    }

    __device__ __forceinline__ void begin(const T* from, int rows, int D) {
        for (int i = threadIdx.x; i < G * DT; i += kPagedBlock) {
            const int r = i / DT, d = i % DT;
            q[i] = r < rows && d < D ? from[r * D + d] : 0.f;
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < kEach; ++i) o[g][i][0] = o[g][i][1] = o[g][i][2] = o[g][i][3] = 0.f;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) m[h] = -INFINITY, l[h] = 0.f;
        __syncthreads();
    }

    __device__ __forceinline__ void step(const char* k, const char* v, int lo, int hi, float scale) {
        const int p = lane() >> 3, t = lane() & 7;
        float s[G] = {};
        const float4* kr = reinterpret_cast<const float4*>(k + t * Ring::kPitch) + p;
#pragma unroll 4
        for (int i = 0; i < DT / 16; ++i) {
            const float4 x = kr[4 * i];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float4 y = reinterpret_cast<const float4*>(q + g * DT)[4 * i + p];
                s[g] = fmaf(x.x, y.x, s[g]);
                s[g] = fmaf(x.y, y.y, s[g]);
                s[g] = fmaf(x.z, y.z, s[g]);
                s[g] = fmaf(x.w, y.w, s[g]);
            }
        }
        // over the quarters: lanes 16 apart, then 8 apart, keep half of the heads each
        if constexpr (G >= 4) {
            const bool up = p & 2, odd = p & 1;
#pragma unroll
            for (int g = 0; g < G / 2; ++g) {
                const float mine = up ? s[g + G / 2] : s[g], theirs = up ? s[g] : s[g + G / 2];
                s[g] = mine + __shfl_xor_sync(0xffffffffu, theirs, 16);
            }
#pragma unroll
            for (int g = 0; g < G / 4; ++g) {
                const float mine = odd ? s[g + G / 4] : s[g], theirs = odd ? s[g] : s[g + G / 4];
                s[g] = mine + __shfl_xor_sync(0xffffffffu, theirs, 8);
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                s[g] += __shfl_xor_sync(0xffffffffu, s[g], 16);
                s[g] += __shfl_xor_sync(0xffffffffu, s[g], 8);
            }
        }
        bool moved = false;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            const float x = t >= lo && t < hi ? s[h] * scale : -INFINITY;
            float top = x;
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(top, m[h]);
            const float zero = top == -INFINITY ? 0.f : top, keep = ex2_approx(m[h] - zero), w = ex2_approx(x - zero);
            m[h] = top;
            l[h] = l[h] * keep + w;
            weights[(own() + h) * 8 + t] = w;
            if (t == 0) keeps[own() + h] = keep;
            moved = moved || keep != 1.f;
        }
        moved = __any_sync(0xffffffffu, moved);
        __syncwarp();
        if (moved) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float keep = keeps[g];
#pragma unroll
                for (int i = 0; i < kEach; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[g][i][e] *= keep;
            }
        }
        const int half = kHalves == 2 ? lane() >> 4 : 0, at = kHalves == 2 ? lane() & 15 : lane();
#pragma unroll
        for (int u = 0; u < 8 / kHalves; u += 4) {
            const int t0 = half * 4 + u;
            float4 x[kEach][4];
#pragma unroll
            for (int i = 0; i < kEach; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i][j] = at + 32 * i < kVectors
                                  ? reinterpret_cast<const float4*>(v + (t0 + j) * Ring::kPitch)[at + 32 * i]
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float4 w = *reinterpret_cast<const float4*>(weights + g * 8 + t0);
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[g][i][0] = fmaf(ws[j], x[i][j].x, o[g][i][0]);
                        o[g][i][1] = fmaf(ws[j], x[i][j].y, o[g][i][1]);
                        o[g][i][2] = fmaf(ws[j], x[i][j].z, o[g][i][2]);
                        o[g][i][3] = fmaf(ws[j], x[i][j].w, o[g][i][3]);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void spoil() {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) l[h] = NAN;
    }
    __device__ __forceinline__ void tell(float* tops, float* sums) {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
            if ((lane() & 7) == 0) tops[own() + h] = m[h], sums[own() + h] = l[h];
        }
    }
    __device__ __forceinline__ void add(float* joined, const float (&factor)[G], bool first) {
        const int at = kHalves == 2 ? lane() & 15 : lane();
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if constexpr (kHalves == 2) o[g][i][e] += __shfl_xor_sync(0xffffffffu, o[g][i][e], 16);
                if (at + 32 * i < kVectors && lane() < 32 / kHalves) {
                    float4* to = reinterpret_cast<float4*>(joined + g * DT) + at + 32 * i;
                    const float4 v = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *to;
                    *to = make_float4(v.x + o[g][i][0] * factor[g], v.y + o[g][i][1] * factor[g],
                                      v.z + o[g][i][2] * factor[g], v.w + o[g][i][3] * factor[g]);
                }
            }
    }
};

template <int G>
cudaError_t paged_f32(const PagedArgs& a, void* workspace, const LaunchCfg& cfg) {
    const int blocks = int((a.heads / a.kv_heads + G - 1) / G);
    switch (paged_width(a.D)) {
        case 64: return paged_launch<PagedF32<64, G>>(a, workspace, blocks, cfg);
        case 80: return paged_launch<PagedF32<80, G>>(a, workspace, blocks, cfg);
        case 96: return paged_launch<PagedF32<96, G>>(a, workspace, blocks, cfg);
        case 128: return paged_launch<PagedF32<128, G>>(a, workspace, blocks, cfg);
        case 160: return paged_launch<PagedF32<160, G>>(a, workspace, blocks, cfg);
        case 192: return paged_launch<PagedF32<192, G>>(a, workspace, blocks, cfg);
        default: return paged_launch<PagedF32<256, G>>(a, workspace, blocks, cfg);
    }
}

}  // namespace rowops
