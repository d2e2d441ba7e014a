// Group norm with an activation on channels-last data: B samples of S positions
// of C channels (position stride ld), G groups of L = C / G channels. Over the m =
// S L elements of a sample's group, mean and biased variance;
//   xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  y = act(xh w + b)
// Backward, with dz = dy act'(xh w + b) and per sample and channel
// A_c = sum_s dz, Q_c = sum_s dz xh:
//   dx = rstd (dz w - c1 - xh c2),  c1 = sum_{c in group} w_c A_c / m, c2 = sum w_c Q_c / m
//   dw_c = sum over the samples of Q_c,  db_c = sum over the samples of A_c
//
// Bound by memory traffic. Two passes: the first leaves each chunk of a sample's
// positions with its groups' sums, the second adds up the chunks of its sample
// and writes the result, reading the tensors again (from L2 where they fit).
//
// A thread keeps one vector of channels over the positions of its chunk, so a
// channel's parameters and sums live in registers and a group may hold any
// number of channels, straddling vectors. The variance is never a difference of
// large sums: a thread sums x - k and (x - k)^2 about its own first value k, and
// (count, mean, sum of squares about the mean) are merged from there on, each
// merge taking the squares of the means' differences.
#pragma once

#include "activations.cuh"
#include "column_partials.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace rowops {

constexpr int kGnBlock = 256;

// (count, mean, sum of squares about the mean) of two sets as those of their union
struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ Moments merge(Moments a, Moments b) {
    if (b.n == 0.f) return a;
    if (a.n == 0.f) return b;
    const float n = a.n + b.n, d = b.mean - a.mean, f = b.n / n;
    return Moments{n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * (a.n * f)};
}
__device__ __forceinline__ Moments warp_merge(Moments v) {
    for (int o = 16; o > 0; o >>= 1)
        v = merge(v, Moments{__shfl_xor_sync(0xffffffffu, v.n, o), __shfl_xor_sync(0xffffffffu, v.mean, o),
                             __shfl_xor_sync(0xffffffffu, v.m2, o)});
    return v;
}

// VEC elements at p as fp32 (VEC 1: one element)
template <typename T, int VEC>
struct Piece {
    using E = Elem<T>;
    uint4 v;
    float s;
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC == 1) s = E::load(p);
        else v = ld_stream16(p);
    }
    __device__ __forceinline__ void load_keep(const T* p) {
        if constexpr (VEC == 1) s = E::load(p);
        else v = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        if constexpr (VEC == 1) f[0] = s;
        else E::unpack(v, f);
    }
    __device__ __forceinline__ static void store(T* p, const float (&f)[VEC]) {
        if constexpr (VEC == 1) E::store(p, f[0]);
        else st_stream16(p, E::pack(f));
    }
};

// Pass 1 of the forward: part[(sample chunks + chunk) G + g] = (mean, sum of
// squares about it) of the chunk's positions.
template <typename T, int VEC>
__global__ void __launch_bounds__(kGnBlock) gn_stats_kernel(const T* x, float2* part, GnArgs a) {
    extern __shared__ float sm[];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int TX = a.tx, TY = kGnBlock / TX, tx = t % TX, ty = t / TX;
    const int W = TX * VEC;                     // channels of a tile
    float* pm = sm;                             // [TY][W] means
    float* pq = pm + TY * W;                    // [TY][W] squares
    Moments* group = reinterpret_cast<Moments*>(pq + TY * W);  // [G]
    const int64_t r0 = int64_t(blockIdx.y) * a.chunk_rows;
    const int64_t r1 = r0 + a.chunk_rows < a.S ? r0 + a.chunk_rows : a.S;
    const T* xs = x + int64_t(blockIdx.x) * a.S * a.ld;
    for (int g = t; g < a.G; g += kGnBlock) group[g] = Moments{0.f, 0.f, 0.f};

    for (int tile = 0; tile < a.tiles; ++tile) {
        const int c0 = tile * W, c = c0 + tx * VEC;
        float k[VEC] = {}, s1[VEC] = {}, s2[VEC] = {};
        int n = 0;
        if (ty < TY && c < a.C && r0 + ty < r1) {
            Piece<T, VEC> first;
            first.load_keep(xs + (r0 + ty) * a.ld + c);
            first.get(k);
            constexpr int U = 4;
            for (int64_t r = r0 + ty; r < r1; r += int64_t(TY) * U) {
                Piece<T, VEC> p[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r + u * TY < r1) p[u].load_keep(xs + (r + u * TY) * a.ld + c);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r + u * TY < r1) {
                        float v[VEC];
                        p[u].get(v);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float d = v[e] - k[e];
                            s1[e] += d;
                            s2[e] = fmaf(d, d, s2[e]);
                        }
                        ++n;
                    }
            }
        }
        if (ty < TY) {
            const float inv = n ? 1.f / float(n) : 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = s1[e] * inv;
                pm[ty * W + tx * VEC + e] = k[e] + d;
                const float q = fmaf(-s1[e], d, s2[e]);
                pq[ty * W + tx * VEC + e] = q < 0.f ? 0.f : q;  // a NaN stays
            }
        }
        __syncthreads();
        // a warp per group of the tile
        const int cend = min(c0 + W, a.C);
        for (int g = c0 / a.L + warp; g * a.L < cend; g += kGnBlock / 32) {
            const int ca = max(g * a.L, c0) - c0, width = min((g + 1) * a.L, cend) - c0 - ca;
            Moments m{0.f, 0.f, 0.f};
            for (int i = lane; i < TY * width; i += 32) {
                const int y = i / width, q = y * W + ca + (i - y * width);
                const int64_t left = r1 - r0 - y;
                if (left > 0) m = merge(m, Moments{float((left + TY - 1) / TY), pm[q], pq[q]});
            }
            m = warp_merge(m);
            if (lane == 0) group[g] = merge(group[g], m);
        }
        __syncthreads();
    }
    float2* out = part + (int64_t(blockIdx.x) * a.chunks + blockIdx.y) * a.G;
    for (int g = t; g < a.G; g += kGnBlock) out[g] = make_float2(group[g].mean, group[g].m2);
}

// The sample's (mean, rstd) of every group from its chunks' moments, into shared
// memory; a warp per group.
__device__ __forceinline__ void gn_merge_stats(const float2* part, const GnArgs& a, float2* stats) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float2* p = part + int64_t(blockIdx.x) * a.chunks * a.G;
    for (int g = warp; g < a.G; g += kGnBlock / 32) {
        Moments m{0.f, 0.f, 0.f};
        for (int k = lane; k < a.chunks; k += 32) {
            const float2 q = p[int64_t(k) * a.G + g];
            const int64_t r0 = int64_t(k) * a.chunk_rows;
            const int64_t rows = r0 + a.chunk_rows < a.S ? a.chunk_rows : a.S - r0;
            m = merge(m, Moments{float(rows) * float(a.L), q.x, q.y});
        }
        m = warp_merge(m);
        if (lane == 0) stats[g] = make_float2(m.mean, 1.f / sqrtf(m.m2 / m.n + a.eps));
    }
}

// Pass 2 of the forward.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock)
    gn_apply_kernel(const T* x, T* y, const T* w, const T* b, const float2* part, float2* stats_out, GnArgs a) {
    using E = Elem<T>;
    extern __shared__ float2 stats[];  // [G]
    const int t = threadIdx.x;
    const int TX = a.tx, TY = kGnBlock / TX, tx = t % TX, ty = t / TX;
    gn_merge_stats(part, a, stats);
    __syncthreads();
    if (stats_out && blockIdx.y == 0)
        for (int g = t; g < a.G; g += kGnBlock) stats_out[int64_t(blockIdx.x) * a.G + g] = stats[g];
    const int64_t r0 = int64_t(blockIdx.y) * a.rows;
    const int64_t r1 = r0 + a.rows < a.S ? r0 + a.rows : a.S;
    const int64_t sample = int64_t(blockIdx.x) * a.S * a.ld;
    if (ty >= TY) return;
    for (int tile = 0; tile < a.tiles; ++tile) {
        const int c = (tile * TX + tx) * VEC;
        if (c >= a.C) continue;
        float mean[VEC], mul[VEC], add[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 s = stats[(c + e) / a.L];
            mean[e] = s.x;
            mul[e] = w ? s.y * E::load(w + c + e) : s.y;
            add[e] = b ? E::load(b + c + e) : 0.f;
        }
        constexpr int U = 4;
        for (int64_t r = r0 + ty; r < r1; r += int64_t(TY) * U) {
            Piece<T, VEC> p[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * TY < r1) p[u].load(x + sample + (r + u * TY) * a.ld + c);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * TY < r1) {
                    float v[VEC];
                    p[u].get(v);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[e] = act_of<ACT>(fmaf(v[e] - mean[e], mul[e], add[e]));
                    Piece<T, VEC>::store(y + sample + (r + u * TY) * a.ld + c, v);
                }
        }
    }
}

// Pass 1 of the backward: chan[(sample chunks + chunk) 2 C + {0, C} + c] = the
// chunk's sums of dz xh (dw) and dz (db); part[(sample chunks + chunk) G + g] =
// the group's sums of w A and w Q.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock)
    gn_bwd_sums_kernel(const T* x, const T* dy, const T* w, const T* b, const float2* stats, float2* part, float* chan,
                       GnArgs a) {
    using E = Elem<T>;
    extern __shared__ float sm[];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int TX = a.tx, TY = kGnBlock / TX, tx = t % TX, ty = t / TX;
    const int W = TX * VEC;
    float* pa = sm;             // [TY][W] A, then the channel sums in row 0
    float* pq = pa + TY * W;    // [TY][W] Q
    float2* group = reinterpret_cast<float2*>(pq + TY * W);  // [G]
    const int64_t r0 = int64_t(blockIdx.y) * a.chunk_rows;
    const int64_t r1 = r0 + a.chunk_rows < a.S ? r0 + a.chunk_rows : a.S;
    const int64_t sample = int64_t(blockIdx.x) * a.S * a.ld;
    const int64_t slot = int64_t(blockIdx.x) * a.chunks + blockIdx.y;
    for (int g = t; g < a.G; g += kGnBlock) group[g] = make_float2(0.f, 0.f);

    for (int tile = 0; tile < a.tiles; ++tile) {
        const int c0 = tile * W, c = c0 + tx * VEC;
        float sa[VEC] = {}, sq[VEC] = {};
        if (ty < TY && c < a.C) {
            float mean[VEC], rstd[VEC], wc[VEC], bc[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 s = stats[int64_t(blockIdx.x) * a.G + (c + e) / a.L];
                mean[e] = s.x;
                rstd[e] = s.y;
                wc[e] = w ? E::load(w + c + e) : 1.f;
                bc[e] = b ? E::load(b + c + e) : 0.f;
            }
            constexpr int U = 2;
            for (int64_t r = r0 + ty; r < r1; r += int64_t(TY) * U) {
                Piece<T, VEC> p[U], q[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r + u * TY < r1) {
                        p[u].load_keep(x + sample + (r + u * TY) * a.ld + c);
                        q[u].load_keep(dy + sample + (r + u * TY) * a.ld + c);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r + u * TY < r1) {
                        float v[VEC], d[VEC];
                        p[u].get(v);
                        q[u].get(d);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float xh = (v[e] - mean[e]) * rstd[e];
                            const float dz = d[e] * act_grad<ACT>(fmaf(xh, wc[e], bc[e]));
                            sa[e] += dz;
                            sq[e] = fmaf(dz, xh, sq[e]);
                        }
                    }
            }
        }
        if (ty < TY) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                pa[ty * W + tx * VEC + e] = sa[e];
                pq[ty * W + tx * VEC + e] = sq[e];
            }
        }
        __syncthreads();
        const int cend = min(c0 + W, a.C);
        for (int i = t; i < cend - c0; i += kGnBlock) {
            float A = pa[i], Q = pq[i];
            for (int k = 1; k < TY; ++k) {
                A += pa[k * W + i];
                Q += pq[k * W + i];
            }
            chan[slot * 2 * a.C + c0 + i] = Q;
            chan[slot * 2 * a.C + a.C + c0 + i] = A;
            const float wc = w ? E::load(w + c0 + i) : 1.f;
            pa[i] = wc * A;
            pq[i] = wc * Q;
        }
        __syncthreads();
        for (int g = c0 / a.L + warp; g * a.L < cend; g += kGnBlock / 32) {
            const int ca = max(g * a.L, c0), cb = min((g + 1) * a.L, cend);
            float A = 0.f, Q = 0.f;
            for (int i = ca + lane; i < cb; i += 32) {
                A += pa[i - c0];
                Q += pq[i - c0];
            }
            for (int o = 16; o > 0; o >>= 1) {
                A += __shfl_xor_sync(0xffffffffu, A, o);
                Q += __shfl_xor_sync(0xffffffffu, Q, o);
            }
            if (lane == 0) group[g] = make_float2(group[g].x + A, group[g].y + Q);
        }
        __syncthreads();
    }
    for (int g = t; g < a.G; g += kGnBlock) part[slot * a.G + g] = group[g];
}

// Pass 2 of the backward.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock)
    gn_bwd_apply_kernel(const T* x, const T* dy, T* dx, const T* w, const T* b, const float2* stats,
                        const float2* part, GnArgs a) {
    using E = Elem<T>;
    extern __shared__ float2 means[];  // [G]: c1, c2
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int TX = a.tx, TY = kGnBlock / TX, tx = t % TX, ty = t / TX;
    const float m = float(a.S) * float(a.L);
    for (int g = warp; g < a.G; g += kGnBlock / 32) {
        float A = 0.f, Q = 0.f;
        for (int k = lane; k < a.chunks; k += 32) {
            const float2 q = part[(int64_t(blockIdx.x) * a.chunks + k) * a.G + g];
            A += q.x;
            Q += q.y;
        }
        for (int o = 16; o > 0; o >>= 1) {
            A += __shfl_xor_sync(0xffffffffu, A, o);
            Q += __shfl_xor_sync(0xffffffffu, Q, o);
        }
        if (lane == 0) means[g] = make_float2(A / m, Q / m);
    }
    __syncthreads();
    const int64_t r0 = int64_t(blockIdx.y) * a.rows;
    const int64_t r1 = r0 + a.rows < a.S ? r0 + a.rows : a.S;
    const int64_t sample = int64_t(blockIdx.x) * a.S * a.ld;
    if (ty >= TY) return;
    for (int tile = 0; tile < a.tiles; ++tile) {
        const int c = (tile * TX + tx) * VEC;
        if (c >= a.C) continue;
        float mean[VEC], rstd[VEC], wc[VEC], bc[VEC], c1[VEC], c2[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int g = (c + e) / a.L;
            const float2 s = stats[int64_t(blockIdx.x) * a.G + g];
            mean[e] = s.x;
            rstd[e] = s.y;
            c1[e] = means[g].x;
            c2[e] = means[g].y;
            wc[e] = w ? E::load(w + c + e) : 1.f;
            bc[e] = b ? E::load(b + c + e) : 0.f;
        }
        constexpr int U = 2;
        for (int64_t r = r0 + ty; r < r1; r += int64_t(TY) * U) {
            Piece<T, VEC> p[U], q[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * TY < r1) {
                    p[u].load(x + sample + (r + u * TY) * a.ld + c);
                    q[u].load(dy + sample + (r + u * TY) * a.ld + c);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * TY < r1) {
                    float v[VEC], d[VEC];
                    p[u].get(v);
                    q[u].get(d);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float xh = (v[e] - mean[e]) * rstd[e];
                        const float dz = d[e] * act_grad<ACT>(fmaf(xh, wc[e], bc[e]));
                        // the product rounded as the sums' terms are, so that a
                        // group of one element comes out as exactly 0
                        v[e] = rstd[e] * (__fmul_rn(dz, wc[e]) - c1[e] - xh * c2[e]);
                    }
                    Piece<T, VEC>::store(dx + sample + (r + u * TY) * a.ld + c, v);
                }
        }
    }
}

// ---- launchers -------------------------------------------------------------
// Channel vectors side by side: all of them where they fit the CTA, else equal tiles.
inline void gn_tiles(GnArgs& a, int vec) {
    const int nv = (a.C + vec - 1) / vec;
    a.tiles = (nv + kGnBlock - 1) / kGnBlock;
    a.tx = (nv + a.tiles - 1) / a.tiles;
}

template <typename T, int VEC, int ACT>
cudaError_t gn_forward_launch(const void* x, void* y, const void* w, const void* b, float* stats, void* ws, GnArgs a,
                              const LaunchCfg& cfg) {
    gn_tiles(a, VEC);
    const int ty = kGnBlock / a.tx;
    float2* part = static_cast<float2*>(ws);
    auto k1 = gn_stats_kernel<T, VEC>;
    auto k2 = gn_apply_kernel<T, VEC, ACT>;
    const size_t s1 = size_t(ty) * a.tx * VEC * 8 + size_t(a.G) * sizeof(Moments), s2 = size_t(a.G) * 8;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k1), s1, cfg);
    if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(k2), s2, cfg);
    if (e != cudaSuccess) return e;
    k1<<<dim3(unsigned(a.B), unsigned(a.chunks)), kGnBlock, s1, cfg.stream>>>(static_cast<const T*>(x), part, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k2<<<dim3(unsigned(a.B), unsigned((a.S + a.rows - 1) / a.rows)), kGnBlock, s2, cfg.stream>>>(
        static_cast<const T*>(x), static_cast<T*>(y), static_cast<const T*>(w), static_cast<const T*>(b), part,
        reinterpret_cast<float2*>(stats), a);
    return cudaGetLastError();
}

template <typename T, int VEC, int ACT>
cudaError_t gn_backward_launch(const void* x, const void* dy, const void* w, const void* b, const float* stats,
                               void* dx, float* dw, float* db, void* ws, GnArgs a, const LaunchCfg& cfg) {
    gn_tiles(a, VEC);
    const int ty = kGnBlock / a.tx;
    float* chan = static_cast<float*>(ws);
    const size_t slots = size_t(a.B) * a.chunks;
    float2* part = reinterpret_cast<float2*>(chan + slots * 2 * a.C);
    auto k1 = gn_bwd_sums_kernel<T, VEC, ACT>;
    auto k2 = gn_bwd_apply_kernel<T, VEC, ACT>;
    const size_t s1 = size_t(ty) * a.tx * VEC * 8 + size_t(a.G) * 8, s2 = size_t(a.G) * 8;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k1), s1, cfg);
    if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(k2), s2, cfg);
    if (e != cudaSuccess) return e;
    const T *xp = static_cast<const T*>(x), *dyp = static_cast<const T*>(dy);
    const T *wp = static_cast<const T*>(w), *bp = static_cast<const T*>(b);
    const float2* st = reinterpret_cast<const float2*>(stats);
    k1<<<dim3(unsigned(a.B), unsigned(a.chunks)), kGnBlock, s1, cfg.stream>>>(xp, dyp, wp, bp, st, part, chan, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k2<<<dim3(unsigned(a.B), unsigned((a.S + a.rows - 1) / a.rows)), kGnBlock, s2, cfg.stream>>>(
        xp, dyp, static_cast<T*>(dx), wp, bp, st, part, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const unsigned cg = unsigned((a.C + 31) / 32);
    column_partials_kernel<<<cg, dim3(32, 32), 0, cfg.stream>>>(chan, int(slots), 2 * int64_t(a.C), a.C, dw);
    column_partials_kernel<<<cg, dim3(32, 32), 0, cfg.stream>>>(chan + a.C, int(slots), 2 * int64_t(a.C), a.C, db);
    return cudaGetLastError();
}

template <typename T>
GnForwardLaunch gn_forward_table(bool vec, int act) {
    constexpr int V = Elem<T>::kVec;
    static const GnForwardLaunch t[2][4] = {
        {gn_forward_launch<T, 1, 0>, gn_forward_launch<T, 1, 1>, gn_forward_launch<T, 1, 2>, gn_forward_launch<T, 1, 3>},
        {gn_forward_launch<T, V, 0>, gn_forward_launch<T, V, 1>, gn_forward_launch<T, V, 2>, gn_forward_launch<T, V, 3>}};
    return t[vec][act];
}

template <typename T>
GnBackwardLaunch gn_backward_table(bool vec, int act) {
    constexpr int V = Elem<T>::kVec;
    static const GnBackwardLaunch t[2][4] = {{gn_backward_launch<T, 1, 0>, gn_backward_launch<T, 1, 1>,
                                              gn_backward_launch<T, 1, 2>, gn_backward_launch<T, 1, 3>},
                                             {gn_backward_launch<T, V, 0>, gn_backward_launch<T, V, 1>,
                                              gn_backward_launch<T, V, 2>, gn_backward_launch<T, V, 3>}};
    return t[vec][act];
}

}  // namespace rowops
