// Bias + dropout + residual, and its backward with the bias's gradient:
//   y = r + keep (x + b) / (1 - p);    dx = keep dy / (1 - p), db = column sums of dx
// (the backward is the same kernel on dy without bias and residual). Whether
// an element is kept follows from 16 random bits of Philox4x32-10: element (row,
// col) takes half-word col mod 8 of the block with counter (col / 8, row,
// offset) and key seed, and is kept where they reach round(65536 p). The mask is
// a function of position alone: never stored, and the same for every layout,
// launch shape and type. Sixteen bits an element instead of 32 halve the
// generator's share of the instructions: ten rounds cost about 60 instructions
// for eight elements.
//
// A team of TL lanes holds 8 TL consecutive columns of a row; lane l makes the
// block of columns 8 l .. 8 l + 7 and keeps its eight decisions as a byte. Each
// lane moves the columns that coalesce best for the type and alignment (bf16:
// its own eight as one 16-byte vector; fp32: two 16-byte vectors; rows that
// start at odd offsets: eight single elements, TL apart) and gets the bytes of
// those columns from the lanes that made them. The lanes keep their columns
// over all rows of a chunk, so the bias is loaded once and column sums stay in
// registers until the chunk's end; they leave one partial row per chunk, added
// up by a second kernel in a fixed order.
#include "column_partials.cuh"
#include "philox.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace rowops {
namespace {

constexpr int kWarps = 8;

struct DropArgs {
    int64_t M, N, ld, chunk_rows;
    int tl_log2, wx_log2;  // lanes of a team; warps of a CTA side by side
    uint32_t lim;          // round(65536 p) 2^16 - 1: kept where the bits, as the upper half-word, are above
    float scale;           // 1 / (1 - p) for p = round(65536 p) / 65536
    uint64_t seed, offset;
    const uint64_t* device_offset;
};

// the decisions of a block's eight half-words, bit e for column e
__device__ __forceinline__ uint32_t keep_bits(const uint4& q, uint32_t lim) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m |= (w[i] << 16) > lim ? 1u << (2 * i) : 0u;
        m |= w[i] > lim ? 2u << (2 * i) : 0u;
    }
    return m;
}

// VEC: 16-byte vectors (16-byte aligned rows, N a multiple of the vector), else
// single elements. RNG: p > 0. SUM: column sums of the results into `part`.
// U: rows of a team in flight.
template <typename T, bool VEC, bool RNG, bool SUM, int U>
__global__ void __launch_bounds__(kWarps * 32)
    dropout_kernel(const T* x, const T* r, const T* b, T* y, float* part, DropArgs a) {
    using E = Elem<T>;
    constexpr int PE = VEC ? E::kVec : 1;  // elements of a piece
    constexpr int NP = 8 / PE;             // pieces of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int TL = 1 << a.tl_log2, tl = lane & (TL - 1), sub = lane >> a.tl_log2;
    const int WX = 1 << a.wx_log2, wx = warp & (WX - 1), wy = warp >> a.wx_log2;
    const int SR = 32 >> a.tl_log2, RY = (kWarps >> a.wx_log2) * SR;  // rows of a warp and of the CTA at a time
    const int64_t c0 = (int64_t(blockIdx.x) * WX + wx) * 8 * TL;     // the team's first column
    const int64_t r0 = int64_t(blockIdx.y) * a.chunk_rows;
    const int64_t r1 = r0 + a.chunk_rows < a.M ? r0 + a.chunk_rows : a.M;
    const uint2 key = make_uint2(uint32_t(a.seed), uint32_t(a.seed >> 32));
    uint64_t off = a.offset;
    if (RNG && a.device_offset) off += *a.device_offset;

    int64_t col[NP];
    bool in[NP];
    float bias[NP][PE];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        col[j] = c0 + PE * (TL * j + tl);
        in[j] = col[j] < a.N;
#pragma unroll
        for (int e = 0; e < PE; ++e) bias[j][e] = b && in[j] ? E::load(b + col[j] + e) : 0.f;
    }
    float acc[NP][PE] = {};

    for (int64_t rb = r0 + wy * SR; rb < r1; rb += int64_t(RY) * U) {
        uint4 xv[U][NP], rv[U][NP];
        float xs[U][NP], rs[U][NP];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = rb + sub + int64_t(u) * RY;
#pragma unroll
            for (int j = 0; j < NP; ++j)
                if (row < r1 && in[j]) {
                    const int64_t at = row * a.ld + col[j];
                    if constexpr (VEC) {
                        xv[u][j] = ld_stream16(x + at);
                        if (r) rv[u][j] = ld_stream16(r + at);
                    } else {
                        xs[u][j] = E::load(x + at);
                        if (r) rs[u][j] = E::load(r + at);
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = rb + sub + int64_t(u) * RY;
            uint32_t own = 0xffu;
            if constexpr (RNG)
                own = keep_bits(philox4x32_10(make_uint4(uint32_t(c0 >> 3) + tl, uint32_t(row), uint32_t(off),
                                                         uint32_t(off >> 32)),
                                              key),
                                a.lim);
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                uint32_t keep = own;
                if constexpr (RNG && PE < 8) {
                    const int at = PE * (TL * j + tl);  // column within the team's
                    keep = __shfl_sync(0xffffffffu, own, (lane & ~(TL - 1)) + (at >> 3)) >> (at & 7);
                }
                if (row < r1 && in[j]) {
                    const int64_t at = row * a.ld + col[j];
                    float v[PE], q[PE];
                    if constexpr (VEC) {
                        E::unpack(xv[u][j], v);
                        if (r) E::unpack(rv[u][j], q);
                    } else {
                        v[0] = xs[u][j];
                        if (r) q[0] = rs[u][j];
                    }
#pragma unroll
                    for (int e = 0; e < PE; ++e) {
                        v[e] = keep >> e & 1u ? (v[e] + bias[j][e]) * a.scale : 0.f;
                        if constexpr (SUM) acc[j][e] += v[e];
                        if (r) v[e] += q[e];
                    }
                    if constexpr (VEC) st_stream16(y + at, E::pack(v));
                    else E::store(y + at, v[0]);
                }
            }
        }
    }

    if constexpr (SUM) {
        // over the warp's teams, then over the CTA's warps of the same columns
        __shared__ float red[kWarps][256];
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int e = 0; e < PE; ++e) {
                for (int o = TL; o < 32; o <<= 1) acc[j][e] += __shfl_xor_sync(0xffffffffu, acc[j][e], o);
                if (sub == 0) red[warp][PE * (TL * j + tl) + e] = acc[j][e];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < WX * 8 * TL; i += kWarps * 32) {
            const int w = i / (8 * TL), c = i - w * 8 * TL;
            float s = 0.f;
            for (int k = w; k < kWarps; k += WX) s += red[k][c];
            const int64_t at = int64_t(blockIdx.x) * WX * 8 * TL + i;
            if (at < a.N) part[int64_t(blockIdx.y) * a.N + at] = s;
        }
    }
}

template <typename T, bool VEC, bool RNG, bool SUM>
cudaError_t launch(const void* x, const void* r, const void* b, void* y, float* part, int max_partials,
                   float* db, DropArgs a, const LaunchCfg& cfg) {
    constexpr int U = VEC ? 4 : 2;
    auto kern = dropout_kernel<T, VEC, RNG, SUM, U>;
    // the widest team, then the most warps side by side, that leave at most 1/8
    // of their columns idle; else those that leave the fewest
    auto pick = [](int64_t n, int64_t unit, int top) {
        int best = 0;
        int64_t least = -1;
        for (int l = top; l >= 0; --l) {
            const int64_t step = unit << l, span = (n + step - 1) / step * step;
            if (span - n <= n / 8) return l;
            if (least < 0 || span < least) {
                best = l;
                least = span;
            }
        }
        return best;
    };
    a.tl_log2 = pick(a.N, 8, 5);
    const int64_t segs = (a.N + (int64_t(8) << a.tl_log2) - 1) / (int64_t(8) << a.tl_log2);
    a.wx_log2 = pick(segs, 1, 3);
    const int64_t gx = (segs + (1 << a.wx_log2) - 1) >> a.wx_log2;
    const int64_t step = int64_t(kWarps >> a.wx_log2) * (32 >> a.tl_log2) * U;  // rows of a CTA at a time
    const int64_t want = int64_t(grid_for(reinterpret_cast<const void*>(kern), kWarps * 32, 0, INT64_MAX, cfg)) *
                         (SUM ? 1 : 4);
    int64_t chunks = (want + gx - 1) / gx;
    if (SUM && chunks > max_partials) chunks = max_partials;
    if (chunks > 65535) chunks = 65535;
    a.chunk_rows = (a.M + chunks - 1) / chunks;
    if (!SUM || (a.M + step - 1) / step >= chunks) a.chunk_rows = (a.chunk_rows + step - 1) / step * step;
    const int64_t gy = (a.M + a.chunk_rows - 1) / a.chunk_rows;
    kern<<<dim3(unsigned(gx), unsigned(gy)), kWarps * 32, 0, cfg.stream>>>(
        static_cast<const T*>(x), static_cast<const T*>(r), static_cast<const T*>(b), static_cast<T*>(y), part, a);
    cudaError_t e = cudaGetLastError();
    if (SUM && e == cudaSuccess) e = reduce_partials(part, gy, a.N, a.N, db, nullptr, cfg);
    return e;
}

template <typename T>
cudaError_t dropout(const void* x, const void* r, const void* b, void* y, float* part, int max_partials, float* db,
                    int64_t M, int64_t N, int64_t ld, const DropoutMask& m, bool vec, const LaunchCfg& cfg) {
    DropArgs a{M, N, ld, 0, 0, 0, (m.drop << 16) - 1u, m.drop < 65536u ? 65536.f / float(65536u - m.drop) : 0.f,
               m.seed, m.offset, m.device_offset};
    const int k = (vec ? 4 : 0) | (m.drop ? 2 : 0) | (db ? 1 : 0);
    switch (k) {
        case 0: return launch<T, false, false, false>(x, r, b, y, part, max_partials, db, a, cfg);
        case 1: return launch<T, false, false, true>(x, r, b, y, part, max_partials, db, a, cfg);
        case 2: return launch<T, false, true, false>(x, r, b, y, part, max_partials, db, a, cfg);
        case 3: return launch<T, false, true, true>(x, r, b, y, part, max_partials, db, a, cfg);
        case 4: return launch<T, true, false, false>(x, r, b, y, part, max_partials, db, a, cfg);
        case 5: return launch<T, true, false, true>(x, r, b, y, part, max_partials, db, a, cfg);
        case 6: return launch<T, true, true, false>(x, r, b, y, part, max_partials, db, a, cfg);
        default: return launch<T, true, true, true>(x, r, b, y, part, max_partials, db, a, cfg);
    }
}

}  // namespace

DropoutLaunch dropout_f32() { return dropout<float>; }
DropoutLaunch dropout_bf16() { return dropout<bf16_t>; }

}  // namespace rowops
