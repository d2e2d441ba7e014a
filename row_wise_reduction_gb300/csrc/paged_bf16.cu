// Attention over a paged cache, bf16 (paged_kernels.cuh): the products on the tensor
// cores by mma.sync, whose accumulators are registers. At one query a sequence a key or value
// is used for the heads of one group only: 2 operations a byte and head, where the memory
// feeds 24 bytes a cycle and SM; the instruction's sixteen rows, of which a group
// fills what it has heads, still leave the tensor cores idle most of the time, so the larger
// tiles of tcgen05 and its accumulators' way through tensor memory would buy nothing.
#include "paged_kernels.cuh"

namespace rowops {
namespace {

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A warp's state for a unit of at most 16 heads: the rows of the products, a lane holding rows
// lane / 4 and lane / 4 + 8. Pieces of 16 positions.
template <int DT>
struct PagedBf16 {
    using T = bf16_t;
    static constexpr int kTokens = 16, kRows = 16, kD = DT, kOwn = 2;
    // Long heads' queries stay in shared memory: 64 registers less, which D = 256 spilled
    static constexpr bool kKept = DT < 192;
    static constexpr size_t kScratch = kKept ? 0 : size_t(DT / 16) * 32 * 16;
    using Ring = PagedRing<T, DT, kTokens>;
    uint32_t q[kKept ? DT / 16 : 1][4];
    uint4* far;  // [DT / 16][32], every warp writes the same
    float o[DT / 8][4], m[2], l[2];
    int rows;

    __device__ __forceinline__ explicit PagedBf16(float* scratch) : far(reinterpret_cast<uint4*>(scratch)) {}
    __device__ __forceinline__ static int lane() { return threadIdx.x & 31; }
    __device__ __forceinline__ static int row(int i) { return lane() / 4 + 8 * i; }

    __device__ __forceinline__ void begin(const T* from, int rows_, int D) {
        rows = rows_;
        const bool pairs = (reinterpret_cast<uintptr_t>(from) & 3) == 0 && D % 2 == 0;
#pragma unroll
        for (int s = 0; s < DT / 16; ++s) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row(i & 1), d = 16 * s + 8 * (i >> 1) + lane() % 4 * 2;
                const T* at = from + r * D + d;
                uint32_t v = 0;
                if (r < rows && d < D)
                    v = pairs ? *reinterpret_cast<const uint32_t*>(at)
                              : at[0].bits | (d + 1 < D ? uint32_t(at[1].bits) << 16 : 0u);
                q[kKept ? s : 0][i] = v;
            }
            if constexpr (!kKept) far[s * 32 + lane()] = make_uint4(q[0][0], q[0][1], q[0][2], q[0][3]);
        }
#pragma unroll
        for (int n = 0; n < DT / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // positions [lo, hi) of the piece count; scale takes a product to the exponent of 2
    __device__ __forceinline__ void step(const char* k, const char* v, int lo, int hi, float scale) {
        const uint32_t g = lane() / 8, r = lane() % 8;
        const uint32_t ka = uint32_t(__cvta_generic_to_shared(k)) + ((g >> 1) * 8 + r) * Ring::kPitch + (g & 1) * 16;
        const uint32_t va = uint32_t(__cvta_generic_to_shared(v)) + ((g & 1) * 8 + r) * Ring::kPitch + (g >> 1) * 16;
        float s[2][4] = {};
#pragma unroll
        for (int i = 0; i < DT / 16; ++i) {
            uint32_t b[4];
            ldmatrix4(b, ka + i * 32);
            if constexpr (!kKept) {
                const uint4 f = far[i * 32 + lane()];
                q[0][0] = f.x, q[0][1] = f.y, q[0][2] = f.z, q[0][3] = f.w;
            }
            mma(s[0], q[kKept ? i : 0], b[0], b[1]);
            mma(s[1], q[kKept ? i : 0], b[2], b[3]);
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 8 * n + lane() % 4 * 2 + (e & 1);
                s[n][e] = t >= lo && t < hi ? s[n][e] * scale : -INFINITY;
                top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
            }
        float keep[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            top[i] = fmaxf(top[i], m[i]);
            const float zero = top[i] == -INFINITY ? 0.f : top[i];
            keep[i] = ex2_approx(m[i] - zero);
            m[i] = top[i];
            top[i] = zero;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = ex2_approx(s[n][e] - top[e >> 1]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            l[i] = l[i] * keep[i] + ((s[0][2 * i] + s[0][2 * i + 1]) + (s[1][2 * i] + s[1][2 * i + 1]));
        if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
            for (int n = 0; n < DT / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] *= keep[e >> 1];
        }
        // the weights as two bf16 numbers each, right to 2^-17 together: one alone would round
        // a weight by 2^-9, which a few large ones do not average out
        uint32_t hi16[4], lo16[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = s[i >> 1][2 * (i & 1)], y = s[i >> 1][2 * (i & 1) + 1];
            hi16[i] = pack_bf16x2(x, y);
            lo16[i] = pack_bf16x2(x - __uint_as_float(hi16[i] << 16), y - __uint_as_float(hi16[i] & 0xffff0000u));
        }
#pragma unroll
        for (int i = 0; i < DT / 16; ++i) {
            uint32_t b[4];
            ldmatrix4_t(b, va + i * 32);
            mma(o[2 * i], hi16, b[0], b[1]);
            mma(o[2 * i + 1], hi16, b[2], b[3]);
            mma(o[2 * i], lo16, b[0], b[1]);
            mma(o[2 * i + 1], lo16, b[2], b[3]);
        }
    }
    __device__ __forceinline__ void spoil() { l[0] = l[1] = NAN; }
    __device__ __forceinline__ void tell(float* tops, float* sums) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (lane() % 4 == 0) tops[row(i)] = m[i], sums[row(i)] = l[i];
        }
    }
    __device__ __forceinline__ void add(float* joined, const float (&factor)[2], bool first) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (row(i) < rows)
#pragma unroll
                for (int n = 0; n < DT / 8; ++n) {
                    float2* at = reinterpret_cast<float2*>(joined + row(i) * DT + 8 * n) + lane() % 4;
                    const float2 v = first ? make_float2(0.f, 0.f) : *at;
                    *at = make_float2(v.x + o[n][2 * i] * factor[i], v.y + o[n][2 * i + 1] * factor[i]);
                }
    }
};

}  // namespace

cudaError_t paged_attention_bf16(const PagedArgs& a, void* workspace, const LaunchCfg& cfg) {
    const int blocks = int((a.heads / a.kv_heads + 15) / 16);
    switch (paged_width(a.D)) {
        case 64: return paged_launch<PagedBf16<64>>(a, workspace, blocks, cfg);
        case 80: return paged_launch<PagedBf16<80>>(a, workspace, blocks, cfg);
        case 96: return paged_launch<PagedBf16<96>>(a, workspace, blocks, cfg);
        case 128: return paged_launch<PagedBf16<128>>(a, workspace, blocks, cfg);
        case 160: return paged_launch<PagedBf16<160>>(a, workspace, blocks, cfg);
        case 192: return paged_launch<PagedBf16<192>>(a, workspace, blocks, cfg);
        default: return paged_launch<PagedBf16<256>>(a, workspace, blocks, cfg);
    }
}

}  // namespace rowops
