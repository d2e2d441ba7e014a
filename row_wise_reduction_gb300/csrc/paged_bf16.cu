// Attention over a paged cache, bf16 (paged_kernels.cuh): the products on the tensor
// cores by mma.sync, whose accumulators are registers. At one query a sequence a key or value
// is used for the heads of one group only: 2 operations a byte and head, where the memory
// feeds 24 bytes a cycle and SM, which leaves the tensor cores idle most of the time even so: the larger
// tiles of tcgen05, most of them empty, and its accumulators' way through tensor memory would buy nothing.
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

// the 8 x 8 matrix whose row lane / 4 a lane holds a pair of, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// A warp's state for a unit of at most 8 H heads. Pieces of 16 positions. The heads are the
// columns of both products, keys (positions x d) times queries and values transposed (d x
// positions) times weights, as their tiles are 8 wide where rows come by 16: with the heads as
// rows a group of 8 took twice the products, exponentials and accumulators (64 sequences of up to 8192: 190 us).
// A lane holds the heads 2 (lane mod 4) and one more, of every 8. The weights, positions by
// heads as they come, are transposed for the second product.
// Long heads in blocks of 16 are bound by one CTA an SM with four warps: 32 sequences of up to 8192, 96 heads over 8, D 192
// 427 us and D 256 647, whose accumulators take 255 registers and spill 250 to 300 bytes; blocks of 8 (64 heads over 8)
// take 171 and 249.
template <int DT, int H>
struct PagedBf16 {
    using T = bf16_t;
    static constexpr int kRows = 8 * H, kD = DT, kOwn = 2 * H;
    using Ring = PagedRing<T, DT, kRows>;
    static constexpr int kTokens = Ring::kShape.tokens, kPitch = Ring::kShape.joined, kScratch = Ring::kShape.scratch;
    static constexpr bool kKept = kScratch == 0;  // long heads' queries stay in shared memory
    static_assert(kKept || kScratch == DT / 16 * H * 32 * 8);
    uint2 q[kKept ? DT / 16 : 1][H];
    uint2* far;  // [DT / 16][H][32], every warp writes the same
    float o[DT / 16][H][4], m[H][2], l[H][2];
    int rows;

    __device__ __forceinline__ explicit PagedBf16(float* scratch) : far(reinterpret_cast<uint2*>(scratch)) {}
    __device__ __forceinline__ static int lane() { return threadIdx.x & 31; }
    __device__ __forceinline__ static int row(int i) { return 8 * (i >> 1) + lane() % 4 * 2 + (i & 1); }

    __device__ __forceinline__ void begin(const T* from, int rows_, int D) {
        rows = rows_;
        const bool pairs = (reinterpret_cast<uintptr_t>(from) & 3) == 0 && D % 2 == 0;
#pragma unroll
        for (int s = 0; s < DT / 16; ++s)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                uint32_t v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 8 * h + lane() / 4, d = 16 * s + 8 * i + lane() % 4 * 2;
                    const T* at = from + r * D + d;
                    v[i] = 0;
                    if (r < rows && d < D)
                        v[i] = pairs ? *reinterpret_cast<const uint32_t*>(at)
                                     : at[0].bits | (d + 1 < D ? uint32_t(at[1].bits) << 16 : 0u);
                }
                if constexpr (kKept) q[s][h] = make_uint2(v[0], v[1]);
                else far[(s * H + h) * 32 + lane()] = make_uint2(v[0], v[1]);
            }
#pragma unroll
        for (int i = 0; i < DT / 16; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) o[i][h][0] = o[i][h][1] = o[i][h][2] = o[i][h][3] = 0.f;
#pragma unroll
        for (int h = 0; h < H; ++h) m[h][0] = m[h][1] = -INFINITY, l[h][0] = l[h][1] = 0.f;
    }

    // positions [lo, hi) of the piece count; scale takes a product to the exponent of 2
    __device__ __forceinline__ void step(const char* k, const char* v, int lo, int hi, float scale) {
        const uint32_t g = lane() / 8, r = lane() % 8;
        const uint32_t ka = uint32_t(__cvta_generic_to_shared(k)) + ((g & 1) * 8 + r) * Ring::kPitch + (g >> 1) * 16;
        const uint32_t va = uint32_t(__cvta_generic_to_shared(v)) + ((g >> 1) * 8 + r) * Ring::kPitch + (g & 1) * 16;
        float s[H][4] = {}, odd[H][4] = {};  // two chains of products
#pragma unroll
        for (int i = 0; i < DT / 16; ++i) {
            uint32_t a[4];
            ldmatrix4(a, ka + i * 32);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                uint2 b;
                if constexpr (kKept) b = q[i][h];
                else b = far[(i * H + h) * 32 + lane()];
                mma(i & 1 ? odd[h] : s[h], a, b.x, b.y);
            }
        }
        const int t = lane() / 4;
        const bool in[2] = {t >= lo && t < hi, t + 8 >= lo && t + 8 < hi};
        float keep[H][2];
        bool moved = false;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = in[0] ? (s[h][e] + odd[h][e]) * scale : -INFINITY;
                float y = in[1] ? (s[h][e + 2] + odd[h][e + 2]) * scale : -INFINITY;
                float top = fmaxf(x, y);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                top = fmaxf(top, m[h][e]);
                const float zero = top == -INFINITY ? 0.f : top;
                keep[h][e] = ex2_approx(m[h][e] - zero);
                m[h][e] = top;
                x = ex2_approx(x - zero);
                y = ex2_approx(y - zero);
                l[h][e] = l[h][e] * keep[h][e] + (x + y);
                s[h][e] = x;
                s[h][e + 2] = y;
                moved = moved || keep[h][e] != 1.f;
            }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int i = 0; i < DT / 16; ++i)
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][h][e] *= keep[h][e & 1];
        }
        // the weights as two bf16 numbers each, right to 2^-17 together: one alone would round
        // a weight by 2^-9, which a few large ones do not average out
        uint32_t hi16[H][2], lo16[H][2];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = s[h][2 * i], y = s[h][2 * i + 1];
                const uint32_t two = pack_bf16x2(x, y);
                hi16[h][i] = transpose8(two);
                lo16[h][i] = transpose8(pack_bf16x2(x - __uint_as_float(two << 16), y - __uint_as_float(two & 0xffff0000u)));
            }
#pragma unroll
        for (int i = 0; i < DT / 16; ++i) {
            uint32_t a[4];
            ldmatrix4_t(a, va + i * 32);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                mma(o[i][h], a, hi16[h][0], hi16[h][1]);
                mma(o[i][h], a, lo16[h][0], lo16[h][1]);
            }
        }
    }
    __device__ __forceinline__ void spoil() {
#pragma unroll
        for (int h = 0; h < H; ++h) l[h][0] = l[h][1] = NAN;
    }
    __device__ __forceinline__ void tell(float* tops, float* sums) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            float& x = l[i >> 1][i & 1];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            if (lane() < 4) tops[row(i)] = m[i >> 1][i & 1], sums[row(i)] = x;
        }
    }
    __device__ __forceinline__ void add(float* joined, const float (&factor)[kOwn], bool first) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            if (row(i) < rows)
#pragma unroll
                for (int n = 0; n < DT / 8; ++n) {
                    float* at = joined + row(i) * kPitch + 8 * n + lane() / 4;
                    const float v = o[n >> 1][i >> 1][2 * (n & 1) + (i & 1)] * factor[i];
                    *at = first ? v : *at + v;
                }
    }
};

template <int H>
cudaError_t paged_bf16(const PagedArgs& a, void* workspace, const LaunchCfg& cfg) {
    const int blocks = int((a.heads / a.kv_heads + 8 * H - 1) / (8 * H));
    switch (paged_width(a.D)) {
        case 64: return paged_launch<PagedBf16<64, H>>(a, workspace, blocks, cfg);
        case 80: return paged_launch<PagedBf16<80, H>>(a, workspace, blocks, cfg);
        case 96: return paged_launch<PagedBf16<96, H>>(a, workspace, blocks, cfg);
        case 128: return paged_launch<PagedBf16<128, H>>(a, workspace, blocks, cfg);
        case 160: return paged_launch<PagedBf16<160, H>>(a, workspace, blocks, cfg);
        case 192: return paged_launch<PagedBf16<192, H>>(a, workspace, blocks, cfg);
        default: return paged_launch<PagedBf16<256, H>>(a, workspace, blocks, cfg);
    }
}

}  // namespace

cudaError_t paged_attention_bf16(const PagedArgs& a, void* workspace, const LaunchCfg& cfg) {
    return paged_rows(a.heads / a.kv_heads, 2) == 8 ? paged_bf16<1>(a, workspace, cfg) : paged_bf16<2>(a, workspace, cfg);
}

}  // namespace rowops
