// Group norm with an activation on channels-last data: B samples of S positions
// of C channels (position stride ld), G groups of L = C / G channels. Over the m =
// S L elements of a sample's group, mean and biased variance;
//   xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  y = act(xh w + b)
// Backward, with dz = dy act'(xh w + b) and per sample and channel
// A_c = sum_s dz, Q_c = sum_s dz xh:
//   dx = rstd (dz w - c1 - xh c2),  c1 = sum_{c in group} w_c A_c / m, c2 = sum w_c Q_c / m
//   dw_c = sum over the samples of Q_c,  db_c = sum over the samples of A_c
//
// Bound by memory traffic. This file: the parts that both forms share, and the
// two-pass form for samples too large for the shared memory of a cluster. Its
// first pass leaves the groups' sums of each chunk of a sample's positions, its
// second adds up the chunks of its sample and writes the result, reading the
// tensors again, from L2: batches of samples of at most 64 MB go through both
// passes before the next one starts.
//
// A thread keeps one vector of channels over the positions of its chunk, so a
// channel's parameters and sums live in registers and a group may hold any
// number of channels, straddling vectors. The variance is never a difference of
// large sums: a thread sums x - k and (x - k)^2 about its own first value k, and
// (count, mean, sum of squares about the mean) are merged from there on, each
// merge taking the squares of the means' differences. Arithmetic on packed pairs.
#pragma once

#include <type_traits>

#include <cooperative_groups.h>

#include "activations.cuh"
#include "column_partials.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace rowops {

namespace cg = cooperative_groups;

// (count, mean, sum of squares about the mean) of two sets as those of their union
struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ Moments merge(Moments a, Moments b) {
    if (b.n == 0.f) return a;
    if (a.n == 0.f) return b;
    const float n = a.n + b.n, d = b.mean - a.mean, f = b.n * rcp_approx(n);
    return Moments{n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * (a.n * f)};
}

// A vector of VEC channels as P pairs (one element: the second half is 0).
template <typename T, int VEC>
struct Vec {
    using E = Elem<T>;
    using Word = std::conditional_t<VEC == 1, T, uint4>;
    static constexpr int P = VEC == 1 ? 1 : VEC / 2;
    __device__ __forceinline__ static Word load(const T* p) {
        if constexpr (VEC == 1) return *p;
        else return *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ static void get(const Word& w, float2 (&v)[P]) {
        if constexpr (VEC == 1) {
            v[0] = make_float2(E::load(&w), 0.f);
        } else {
            float f[VEC];
            E::unpack(w, f);
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] = make_float2(f[2 * k], f[2 * k + 1]);
        }
    }
    __device__ __forceinline__ static Word pack(const float2 (&v)[P]) {
        if constexpr (VEC == 1) {
            Word w;
            E::store(&w, v[0].x);
            return w;
        } else {
            float f[VEC];
#pragma unroll
            for (int k = 0; k < P; ++k) f[2 * k] = v[k].x, f[2 * k + 1] = v[k].y;
            return E::pack(f);
        }
    }
    __device__ __forceinline__ static void put(T* p, const float2 (&v)[P]) {
        if constexpr (VEC == 1) E::store(p, v[0].x);
        else st_stream16(p, pack(v));
    }
    __device__ __forceinline__ static void keep(Word* p, const float2 (&v)[P]) { *p = pack(v); }  // shared memory
};

// per-channel values of a thread's vector as pairs
template <int VEC, int P, typename F>
__device__ __forceinline__ void each_channel(float2 (&v)[P], F f) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
        v[k].x = f(VEC == 1 ? 0 : 2 * k);
        v[k].y = VEC == 1 ? 0.f : f(2 * k + 1);
    }
}

// The groups of the VEC channels from c on (L may be any number).
template <int VEC>
struct Groups {
    int g[VEC];
    __device__ __forceinline__ Groups(int c, const GnArgs& a) {
        // (c + 1/2) / L is at least 1 / (2 L) from a whole number, and c < 8192
        int k = int((float(c) + 0.5f) * a.inv_L), left = a.L - (c - k * a.L);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            g[e] = k;
            if (--left == 0) {
                left = a.L;
                ++k;
            }
        }
    }
};

// w or b of the VEC channels from c on, `dflt` where there is none
template <typename T, int VEC, int P>
__device__ __forceinline__ void load_affine(const T* p, int c, float dflt, float2 (&v)[P]) {
    using V = Vec<T, VEC>;
    if (!p) each_channel<VEC>(v, [&](int) { return dflt; });
    else if (VEC > 1 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) V::get(V::load(p + c), v);
    else each_channel<VEC>(v, [&](int e) { return Elem<T>::load(p + c + e); });
}

// Sums of x - k and (x - k)^2 about a thread's first value k, and what they say.
template <int P>
struct Shifted {
    float2 k[P], s1[P], s2[P];  // k: negated
    __device__ __forceinline__ void start(const float2 (&v)[P]) {
#pragma unroll
        for (int j = 0; j < P; ++j) k[j] = make_float2(-v[j].x, -v[j].y);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < P; ++j) k[j] = s1[j] = s2[j] = f2(0.f);
    }
    __device__ __forceinline__ void add(const float2 (&v)[P]) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float2 d = f2_add(v[j], k[j]);
            s1[j] = f2_add(s1[j], d);
            s2[j] = f2_fma(d, d, s2[j]);
        }
    }
    // the means and the squares about them of n positions, per channel
    template <int VEC>
    __device__ __forceinline__ void leave(int n, float* mean, float* m2) const {
        const float inv = n ? 1.f / float(n) : 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float s = e & 1 ? s1[e / 2].y : s1[e / 2].x, d = s * inv;
            const float q = fmaf(-s, d, e & 1 ? s2[e / 2].y : s2[e / 2].x);
            mean[e] = d - (e & 1 ? k[e / 2].y : k[e / 2].x);
            m2[e] = q < 0.f ? 0.f : q;  // a NaN stays
        }
    }
};

// One warp: the moments of a group from its threads' means and squares, at
// [row][column], `width` columns of W from c0, rows 0 .. ty; row r stands for
// ceil((rows - r) / ty) positions. The mean first, then the squares about it. The
// divisions are done once for groups of one width.
struct GroupMoments {
    int W, live, each, more, dr, dc, r0, k0, width;
    __device__ __forceinline__ GroupMoments(int W_, int width_, int ty, int rows) : W(W_), width(width_) {
        const int lane = threadIdx.x & 31;
        live = (rows < ty ? rows : ty) * width;  // entries with a position
        each = rows / ty, more = rows - each * ty;  // row r: each + (r < more)
        dr = 32 / width, dc = 32 - dr * width;      // a step of 32 entries
        r0 = lane / width, k0 = lane - r0 * width;
    }
    template <typename F>
    __device__ __forceinline__ void entries(int c0, F f) const {
        int r = r0, k = k0;
        for (int i = threadIdx.x & 31; i < live; i += 32) {
            f(float(each + (r < more)), r * W + c0 + k);
            r += dr;
            k += dc;
            if (k >= width) {
                k -= width;
                ++r;
            }
        }
    }
    __device__ __forceinline__ Moments of(const float* pm, const float* pq, int c0) const {
        const float ref = pm[c0];
        float n = 0.f, s = 0.f, q = 0.f;
        entries(c0, [&](float m, int at) {
            n += m;
            s = fmaf(m, pm[at] - ref, s);
        });
        for (int o = 16; o > 0; o >>= 1) {
            n += __shfl_xor_sync(0xffffffffu, n, o);
            s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        const float off = n > 0.f ? s * (1.f / n) : 0.f;
        entries(c0, [&](float m, int at) {
            const float d = (pm[at] - ref) - off;
            q += fmaf(m * d, d, pq[at]);
        });
        for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
        return Moments{n, ref + off, q};
    }
};

// The CTA's sums over the ty rows of red[ty][W], left in row 0; several threads
// a column where there are enough. Ends with a barrier.
template <int BLOCK>
__device__ __forceinline__ void column_sums(float2* red, int W, int ty) {
    const int parts = max(1, min(ty, BLOCK / W));
    const int per = (ty + parts - 1) / parts;
    for (int i = threadIdx.x; i < W * parts; i += BLOCK) {
        const int p = i / W, c = i - p * W, r1 = min((p + 1) * per, ty);
        float2 s = f2(0.f);
        for (int r = p * per; r < r1; ++r) s = f2_add(s, red[r * W + c]);
        if (p * per < ty) red[p * per * W + c] = s;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < W; c += BLOCK) {
        float2 s = red[c];
        for (int p = 1; p < parts && p * per < ty; ++p) s = f2_add(s, red[p * per * W + c]);
        red[c] = s;
    }
    __syncthreads();
}

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// a value where CTA `rank` of the cluster keeps it
template <typename V>
__device__ __forceinline__ V* in_cta(const cg::cluster_group& cl, V* p, int rank, int cluster) {
    return cluster > 1 ? cl.map_shared_rank(p, rank) : p;
}

// ---- two passes -------------------------------------------------------------
// f(u, word of each pointer) for n positions a stride apart, U of them in flight.
template <typename T, int VEC, int U, int N, typename F>
__device__ __forceinline__ void walk(const T* const (&p0)[N], int64_t step, int n, F f) {
    using V = Vec<T, VEC>;
    const T* p[N];
#pragma unroll
    for (int k = 0; k < N; ++k) p[k] = p0[k];
    auto batch = [&](int live) {
        typename V::Word w[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < live)
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    w[u][k] = V::load(p[k]);
                    p[k] += step;
                }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < live) f(w[u]);
    };
    for (; n >= U; n -= U) batch(U);
    if (n > 0) batch(n);
}

// What a CTA of the two-pass kernels works on; blockIdx.x: the batch's sample.
struct GnChunk {
    int tx, ty, n;   // n: the thread's positions
    int rows;        // the CTA's
    int64_t first;   // element offset of the thread's first position, channel 0
    int64_t step;    // between its positions
    __device__ __forceinline__ GnChunk(const GnArgs& a, int block, unsigned chunk, int64_t chunk_rows) {
        const int TY = block / a.tx;
        ty = int(threadIdx.x) / a.tx;
        tx = int(threadIdx.x) - ty * a.tx;
        const int64_t r0 = chunk * chunk_rows, left = a.S - r0;
        rows = int(left < chunk_rows ? (left > 0 ? left : 0) : chunk_rows);
        n = ty < TY && rows > ty ? (rows - ty + TY - 1) / TY : 0;
        first = ((a.b0 + blockIdx.x) * a.S + r0 + ty) * a.ld;
        step = int64_t(TY) * a.ld;
    }
};

// Pass 1 of the forward: part[(sample chunks + chunk) G + g] = (mean, sum of squares
// about it) of the chunk's positions. One CTA of 1024 threads for each SM: the
// fewer CTAs, the fewer sums a CTA of pass 2 has to read.
template <typename T, int VEC>
__global__ void __launch_bounds__(kGnWide) gn_stats_kernel(const T* x, float2* part, GnArgs a) {
    using V = Vec<T, VEC>;
    constexpr int P = V::P, U = VEC == 1 ? 4 : 8;
    extern __shared__ __align__(16) float sm[];
    grid_wait();
    grid_go();
    const int t = threadIdx.x, warp = t >> 5, TY = kGnWide / a.tx;
    const GnChunk k(a, kGnWide, blockIdx.y, a.chunk_rows);
    const int W = a.tx * VEC;                                  // channels of a tile
    float* pm = sm;                                            // [TY][W] means
    float* pq = pm + TY * W;                                   // [TY][W] squares
    Moments* group = reinterpret_cast<Moments*>(pq + TY * W);  // [G]
    for (int g = t; g < a.G; g += kGnWide) group[g] = Moments{0.f, 0.f, 0.f};

    for (int tile = 0; tile < a.tiles; ++tile) {
        const int c0 = tile * W, c = c0 + k.tx * VEC;
        Shifted<P> s;
        s.clear();
        if (k.n > 0 && c < a.C) {
            const T* const from[1] = {x + k.first + c};
            bool first = true;
            walk<T, VEC, U>(from, k.step, k.n, [&](const typename V::Word (&wd)[1]) {
                float2 v[P];
                V::get(wd[0], v);
                if (first) s.start(v);
                first = false;
                s.add(v);
            });
        }
        if (k.ty < TY) s.template leave<VEC>(c < a.C ? k.n : 0, pm + k.ty * W + k.tx * VEC, pq + k.ty * W + k.tx * VEC);
        __syncthreads();
        // a warp per group of the tile; those that the tile cuts on their own
        const int cend = min(c0 + W, a.C);
        const GroupMoments whole(W, a.L, TY, k.rows);
        for (int g = c0 / a.L + warp; g * a.L < cend; g += kGnWide / 32) {
            const int ca = max(g * a.L, c0), cb = min((g + 1) * a.L, cend);
            const Moments m = cb - ca == a.L ? whole.of(pm, pq, ca - c0)
                                             : GroupMoments(W, cb - ca, TY, k.rows).of(pm, pq, ca - c0);
            if ((t & 31) == 0) group[g] = merge(group[g], m);
        }
        __syncthreads();
    }
    float2* out = part + (int64_t(blockIdx.x) * a.chunks + blockIdx.y) * a.G;
    for (int g = t; g < a.G; g += kGnWide) out[g] = make_float2(group[g].mean, group[g].m2);
}

// Pass 2 of the forward.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock, 3)
    gn_apply_kernel(const T* x, T* y, const T* w, const T* b, const float2* part, float2* stats_out, GnArgs a) {
    using V = Vec<T, VEC>;
    constexpr int P = V::P, U = 4;
    extern __shared__ float2 stats[];  // [G]
    __shared__ Moments red[kGnBlock];
    const int t = threadIdx.x, TY = kGnBlock / a.tx;
    grid_wait();
    grid_go();
    {  // the sample's moments, Y threads a group
        int X = 1;
        while (X < a.G && X < kGnBlock) X <<= 1;
        const int px = t & (X - 1), py = t / X, Y = kGnBlock / X;
        const float2* p = part + int64_t(blockIdx.x) * a.chunks * a.G;
        for (int g0 = 0; g0 < a.G; g0 += X) {
            const int g = g0 + px;
            Moments m{0.f, 0.f, 0.f};
            if (g < a.G)
#pragma unroll 4
                for (int k = py; k < a.chunks; k += Y) {
                    const float2 q = p[k * a.G + g];
                    const int64_t left = a.S - k * a.chunk_rows;
                    m = merge(m, Moments{float(left < a.chunk_rows ? left : a.chunk_rows) * float(a.L), q.x, q.y});
                }
            red[t] = m;
            __syncthreads();
            if (py == 0 && g < a.G) {
                for (int i = 1; i < Y; ++i) m = merge(m, red[i * X + px]);
                stats[g] = make_float2(m.mean, 1.f / sqrtf(m.m2 / m.n + a.eps));
                if (stats_out && blockIdx.y == 0) stats_out[(a.b0 + blockIdx.x) * a.G + g] = stats[g];
            }
            __syncthreads();
        }
    }
    // the positions that pass 1 read last first: they are the likeliest in L2
    const GnChunk k(a, kGnBlock, gridDim.y - 1 - blockIdx.y, a.rows);
    if (k.n == 0) return;
    for (int tile = 0; tile < a.tiles; ++tile) {
        const int c = (tile * a.tx + k.tx) * VEC;
        if (c >= a.C) continue;
        const Groups<VEC> g(c, a);
        float2 mean[P], mul[P], add[P];
        load_affine<T, VEC>(w, c, 1.f, mul);
        load_affine<T, VEC>(b, c, 0.f, add);
        each_channel<VEC>(mean, [&](int e) { return -stats[g.g[e]].x; });
        float2 rstd[P];
        each_channel<VEC>(rstd, [&](int e) { return stats[g.g[e]].y; });
#pragma unroll
        for (int j = 0; j < P; ++j) mul[j] = f2_mul(mul[j], rstd[j]);
        const T* const from[1] = {x + k.first + c};
        T* py = y + k.first + c;
        walk<T, VEC, U>(from, k.step, k.n, [&](const typename V::Word (&wd)[1]) {
            float2 v[P];
            V::get(wd[0], v);
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] = act_of2<ACT>(f2_fma(f2_add(v[j], mean[j]), mul[j], add[j]));
            V::put(py, v);
            py += k.step;
        });
    }
}

// A thread's channels in the backward pass. xc = x - mean; z = xc (rstd w) + b; dz =
// dy act'(z). The sums are of dz and dz xc (times rstd at the end, dz xh).
//   bf16: dx = dz (rstd w) - rstd c1 - xc (rstd^2 c2), two fused operations
//   fp32: dx = rstd ((dz w - c1) - xc (rstd c2)) with dz w rounded as in the sum that
//         c1 comes from, so that a group of one element gets exactly 0 (single
//         operations: a packed product and sum came out as one fused operation)
// The backward pass is bound by instructions in bf16 and by traffic in fp32.
template <typename T, int VEC, int ACT>
struct GnSlope {
    using V = Vec<T, VEC>;
    using Word = typename V::Word;
    static constexpr int P = V::P;
    static constexpr bool kSingle = sizeof(T) == 4;
    float2 mean[P], rstd[P], rw[P], b[P];  // mean negated
    float2 w[kSingle ? P : 1], c1[P], c2[P];
    // c: the channel within the block of groups that `stats` starts at, cb: in all
    __device__ __forceinline__ void load(const T* pw, const T* pb, const float2* stats, int c, int cb,
                                         const GnArgs& a) {
        const Groups<VEC> g(c, a);
        each_channel<VEC>(mean, [&](int e) { return -stats[g.g[e]].x; });
        each_channel<VEC>(rstd, [&](int e) { return stats[g.g[e]].y; });
        load_affine<T, VEC>(pw, cb, 1.f, rw);
        load_affine<T, VEC>(pb, cb, 0.f, b);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if constexpr (kSingle) w[j] = rw[j];
            rw[j] = f2_mul(rw[j], rstd[j]);
        }
    }
    // the group means -c1, -c2
    __device__ __forceinline__ void means(const float2* gs, int c, const GnArgs& a) {
        const Groups<VEC> g(c, a);
        each_channel<VEC>(c1, [&](int e) { return gs[g.g[e]].x; });
        each_channel<VEC>(c2, [&](int e) { return gs[g.g[e]].y; });
#pragma unroll
        for (int j = 0; j < P; ++j) {
            c2[j] = f2_mul(c2[j], rstd[j]);
            if constexpr (!kSingle) {
                c1[j] = f2_mul(c1[j], rstd[j]);
                c2[j] = f2_mul(c2[j], rstd[j]);
            }
        }
    }
    __device__ __forceinline__ void slope(const Word& wx, const Word& wd, float2 (&xc)[P], float2 (&dz)[P]) const {
        V::get(wx, xc);
        V::get(wd, dz);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            xc[j] = f2_add(xc[j], mean[j]);
            dz[j] = f2_mul(dz[j], act_grad2<ACT>(f2_fma(xc[j], rw[j], b[j])));
        }
    }
    __device__ __forceinline__ void add(const Word& wx, const Word& wd, float2 (&sa)[P], float2 (&sq)[P]) const {
        float2 xc[P], dz[P];
        slope(wx, wd, xc, dz);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            sa[j] = f2_add(sa[j], dz[j]);
            sq[j] = f2_fma(dz[j], xc[j], sq[j]);
        }
    }
    // (A, Q) of each channel
    __device__ __forceinline__ void leave(const float2 (&sa)[P], const float2 (&sq)[P], float2* r) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            r[e] = e & 1 ? make_float2(sa[e / 2].y, sq[e / 2].y * rstd[e / 2].y)
                         : make_float2(sa[e / 2].x, sq[e / 2].x * rstd[e / 2].x);
    }
    __device__ __forceinline__ void of(const Word& wx, const Word& wd, float2 (&v)[P]) const {
        float2 xc[P], dz[P];
        slope(wx, wd, xc, dz);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if constexpr (kSingle) {
                const float2 t = make_float2(__fadd_rn(__fmul_rn(dz[j].x, w[j].x), c1[j].x),
                                             __fadd_rn(__fmul_rn(dz[j].y, w[j].y), c1[j].y));
                v[j] = f2_mul(rstd[j], f2_fma(xc[j], c2[j], t));
            } else {
                v[j] = f2_fma(xc[j], c2[j], f2_fma(dz[j], rw[j], c1[j]));
            }
        }
    }
};

// Pass 1 of the backward, for each chunk of a sample ("slot"): chan[slot 2 C + {0,
// C} + c] = the sums of dz xh (dw) and dz (db); part[slot G + g] = the group's sums
// of w A and w Q. One CTA of 512 threads for each SM.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnWideBwd)
    gn_bwd_sums_kernel(const T* x, const T* dy, const T* w, const T* b, const float2* stats, float2* part, float* chan,
                       GnArgs a) {
    using E = Elem<T>;
    using V = Vec<T, VEC>;
    constexpr int P = V::P, U = 2;
    extern __shared__ __align__(16) float2 sm2[];
    grid_wait();
    grid_go();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, TY = kGnWideBwd / a.tx;
    const GnChunk k(a, kGnWideBwd, blockIdx.y, a.chunk_rows);
    const int W = a.tx * VEC;
    float2* red = sm2;             // [TY][W] A, Q
    float2* group = red + TY * W;  // [G]
    const int64_t slot = (a.b0 + blockIdx.x) * a.chunks + blockIdx.y;
    for (int g = t; g < a.G; g += kGnWideBwd) group[g] = f2(0.f);

    for (int tile = 0; tile < a.tiles; ++tile) {
        const int c0 = tile * W, c = c0 + k.tx * VEC;
        GnSlope<T, VEC, ACT> slope;
        float2 sa[P], sq[P];
#pragma unroll
        for (int j = 0; j < P; ++j) sa[j] = sq[j] = slope.rstd[j] = f2(0.f);
        if (k.n > 0 && c < a.C) {
            slope.load(w, b, stats + (a.b0 + blockIdx.x) * a.G, c, c, a);
            const T* const from[2] = {x + k.first + c, dy + k.first + c};
            walk<T, VEC, U>(from, k.step, k.n,
                            [&](const typename V::Word (&wd)[2]) { slope.add(wd[0], wd[1], sa, sq); });
        }
        if (k.ty < TY) slope.leave(sa, sq, red + k.ty * W + k.tx * VEC);
        __syncthreads();
        column_sums<kGnWideBwd>(red, W, TY);
        const int cend = min(c0 + W, a.C);
        for (int i = t; i < cend - c0; i += kGnWideBwd) {
            const float2 s = red[i];
            chan[slot * 2 * a.C + c0 + i] = s.y;
            chan[slot * 2 * a.C + a.C + c0 + i] = s.x;
            const float wc = w ? E::load(w + c0 + i) : 1.f;
            red[i] = make_float2(wc * s.x, wc * s.y);
        }
        __syncthreads();
        for (int g = c0 / a.L + warp; g * a.L < cend; g += kGnWideBwd / 32) {
            const int ca = max(g * a.L, c0), cb = min((g + 1) * a.L, cend);
            float2 s = f2(0.f);
            for (int i = ca + lane; i < cb; i += 32) s = f2_add(s, red[i - c0]);
            for (int o = 16; o > 0; o >>= 1) {
                s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
                s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
            }
            if (lane == 0) group[g] = f2_add(group[g], s);
        }
        __syncthreads();
    }
    for (int g = t; g < a.G; g += kGnWideBwd) part[slot * a.G + g] = group[g];
}

// Pass 2 of the backward.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock, 2)
    gn_bwd_apply_kernel(const T* x, const T* dy, T* dx, const T* w, const T* b, const float2* stats,
                        const float2* part, GnArgs a) {
    using E = Elem<T>;
    using V = Vec<T, VEC>;
    constexpr int P = V::P, U = 2;
    extern __shared__ float2 means[];  // [G]: -c1, -c2
    __shared__ float2 red[kGnBlock];
    const int t = threadIdx.x, TY = kGnBlock / a.tx;
    grid_wait();
    grid_go();
    {
        int X = 1;
        while (X < a.G && X < kGnBlock) X <<= 1;
        const int px = t & (X - 1), py = t / X, Y = kGnBlock / X;
        const float2* p = part + (a.b0 + blockIdx.x) * a.chunks * a.G;
        const float m = float(a.S) * float(a.L);
        for (int g0 = 0; g0 < a.G; g0 += X) {
            const int g = g0 + px;
            float2 s = f2(0.f);
            if (g < a.G)
#pragma unroll 8
                for (int k = py; k < a.chunks; k += Y) s = f2_add(s, p[k * a.G + g]);
            red[t] = s;
            __syncthreads();
            if (py == 0 && g < a.G) {
                for (int i = 1; i < Y; ++i) s = f2_add(s, red[i * X + px]);
                means[g] = make_float2(-s.x / m, -s.y / m);
            }
            __syncthreads();
        }
    }
    const GnChunk k(a, kGnBlock, gridDim.y - 1 - blockIdx.y, a.rows);
    if (k.n == 0) return;
    for (int tile = 0; tile < a.tiles; ++tile) {
        const int c = (tile * a.tx + k.tx) * VEC;
        if (c >= a.C) continue;
        GnSlope<T, VEC, ACT> slope;
        slope.load(w, b, stats + (a.b0 + blockIdx.x) * a.G, c, c, a);
        slope.means(means, c, a);
        const T* const from[2] = {x + k.first + c, dy + k.first + c};
        T* po = dx + k.first + c;
        walk<T, VEC, U>(from, k.step, k.n, [&](const typename V::Word (&wd)[2]) {
            float2 v[P];
            slope.of(wd[0], wd[1], v);
            V::put(po, v);
            po += k.step;
        });
    }
}

// dw, db from P rows of their partial sums [2][C].
inline cudaError_t gn_reduce_channels(const float* chan, int64_t P, int C, float* dw, float* db,
                                      const LaunchCfg& cfg) {
    return reduce_partials(chan, P, 2 * int64_t(C), C, dw, db, cfg);
}

// ---- launchers -------------------------------------------------------------
// Channel vectors side by side: all of them where they fit the CTA, else equal
// tiles (the same ones in both passes).
inline void gn_tiles(GnArgs& a, int vec) {
    const int nv = (a.C + vec - 1) / vec;
    a.tiles = (nv + kGnBlock - 1) / kGnBlock;
    a.tx = (nv + a.tiles - 1) / a.tiles;
}

// A launch that may start while the one before it drains: every kernel here waits
// for that one before it touches memory.
inline cudaError_t gn_launch(const void* kern, dim3 grid, int block, size_t smem, const LaunchCfg& cfg, void** args) {
    cudaError_t e = allow_smem(kern, smem, cfg);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3(unsigned(block));
    lc.dynamicSmemBytes = smem;
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelExC(&lc, kern, args);
}

template <typename T, int VEC, int ACT>
cudaError_t gn_forward_two_pass(const void* x, void* y, const void* w, const void* b, float* stats, void* ws, GnArgs a,
                                const LaunchCfg& cfg) {
    gn_tiles(a, VEC);
    const size_t s1 = size_t(kGnWide / a.tx) * a.tx * VEC * 8 + size_t(a.G) * sizeof(Moments);
    for (a.b0 = 0; a.b0 < a.B; a.b0 += a.batch) {
        const unsigned n = unsigned(std::min<int64_t>(a.batch, a.B - a.b0));
        float2* part = static_cast<float2*>(ws) + a.b0 * a.chunks * a.G;
        void* a1[] = {&x, &part, &a};
        void* a2[] = {&x, &y, &w, &b, &part, &stats, &a};
        cudaError_t e = gn_launch(reinterpret_cast<const void*>(gn_stats_kernel<T, VEC>), dim3(n, unsigned(a.chunks)),
                                  kGnWide, s1, cfg, a1);
        if (e == cudaSuccess)
            e = gn_launch(reinterpret_cast<const void*>(gn_apply_kernel<T, VEC, ACT>),
                          dim3(n, unsigned((a.S + a.rows - 1) / a.rows)), kGnBlock, size_t(a.G) * 8, cfg, a2);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int VEC, int ACT>
cudaError_t gn_backward_two_pass(const void* x, const void* dy, const void* w, const void* b, const float* stats,
                                 void* dx, float* dw, float* db, void* ws, GnArgs a, const LaunchCfg& cfg) {
    gn_tiles(a, VEC);
    const size_t s1 = 8 * (size_t(kGnWideBwd / a.tx) * a.tx * VEC + a.G);
    float* chan = static_cast<float*>(ws);
    const int64_t slots = int64_t(a.B) * a.chunks;
    float2* part = reinterpret_cast<float2*>(chan + slots * 2 * a.C);
    for (a.b0 = 0; a.b0 < a.B; a.b0 += a.batch) {
        const unsigned n = unsigned(std::min<int64_t>(a.batch, a.B - a.b0));
        void* a1[] = {&x, &dy, &w, &b, &stats, &part, &chan, &a};
        void* a2[] = {&x, &dy, &dx, &w, &b, &stats, &part, &a};
        cudaError_t e = gn_launch(reinterpret_cast<const void*>(gn_bwd_sums_kernel<T, VEC, ACT>),
                                  dim3(n, unsigned(a.chunks)), kGnWideBwd, s1, cfg, a1);
        if (e == cudaSuccess)
            e = gn_launch(reinterpret_cast<const void*>(gn_bwd_apply_kernel<T, VEC, ACT>),
                          dim3(n, unsigned((a.S + a.rows - 1) / a.rows)), kGnBlock, size_t(a.G) * 8, cfg, a2);
        if (e != cudaSuccess) return e;
    }
    return gn_reduce_channels(chan, slots, a.C, dw, db, cfg);
}

}  // namespace rowops
