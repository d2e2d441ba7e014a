// Group norm with an activation on channels-last data: B samples of S positions
// of C channels (position stride ld), G groups of L = C / G channels. Over the m =
// S L elements of a sample's group, mean and biased variance;
//   xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps);  y = act(xh w + b)
// Backward, with dz = dy act'(xh w + b) and per sample and channel
// A_c = sum_s dz, Q_c = sum_s dz xh:
//   dx = rstd (dz w - c1 - xh c2),  c1 = sum_{c in group} w_c A_c / m, c2 = sum w_c Q_c / m
//   dw_c = sum over the samples of Q_c,  db_c = sum over the samples of A_c
//
// Bound by memory traffic. This file: what both forms share; groupnorm_fused.cuh
// holds a sample's groups in shared memory between the passes, and
// groupnorm_stream.cuh reads them again from L2 where they are too large.
//
// A thread keeps one vector of channels over the positions of its chunk, so a
// channel's parameters and sums live in registers and a group may hold any
// number of channels, straddling vectors. The variance is never a difference of
// large sums: a thread sums x - k and (x - k)^2 about its own first value k, and
// (count, mean, sum of squares about the mean) are merged from there on, each
// merge taking the squares of the means' differences. All these means are kept less
// one value of the group, its first channel at the sample's first position, which is
// within sqrt(m) spreads of the mean as it is one of the m values: rounded as they are,
// means of 10^6 spreads would lose the variance's fourth digit. The value is added
// back where the results are made. Arithmetic on packed pairs.
#pragma once

#include <type_traits>

#include <cooperative_groups.h>

#include "activations.cuh"
#include "column_partials.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace rowops {

namespace cg = cooperative_groups;

// A vector of VEC channels as P pairs: 16 bytes, or two elements, or one (whose
// pair's second half is 0).
template <typename T, int VEC>
struct Vec {
    using E = Elem<T>;
    static constexpr bool kWhole = VEC * sizeof(T) == 16;
    static_assert(kWhole || VEC <= 2, "16 bytes, or one or two elements");
    using Two = std::conditional_t<sizeof(T) == 4, uint2, uint32_t>;
    using Word = std::conditional_t<kWhole, uint4, std::conditional_t<VEC == 1, T, Two>>;
    static constexpr int P = VEC == 1 ? 1 : VEC / 2;
    __device__ __forceinline__ static Word load(const T* p) { return *reinterpret_cast<const Word*>(p); }
    __device__ __forceinline__ static void get(const Word& w, float2 (&v)[P]) {
        if constexpr (kWhole) {
            float f[VEC];
            E::unpack(w, f);
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] = make_float2(f[2 * k], f[2 * k + 1]);
        } else if constexpr (VEC == 1) {
            v[0] = make_float2(E::load(&w), 0.f);
        } else if constexpr (sizeof(T) == 4) {
            v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        } else {
            v[0] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        }
    }
    __device__ __forceinline__ static Word pack(const float2 (&v)[P]) {
        if constexpr (kWhole) {
            float f[VEC];
#pragma unroll
            for (int k = 0; k < P; ++k) f[2 * k] = v[k].x, f[2 * k + 1] = v[k].y;
            return E::pack(f);
        } else if constexpr (VEC == 1) {
            Word w;
            E::store(&w, v[0].x);
            return w;
        } else if constexpr (sizeof(T) == 4) {
            return make_uint2(__float_as_uint(v[0].x), __float_as_uint(v[0].y));
        } else {
            return pack_bf16x2(v[0].x, v[0].y);
        }
    }
    __device__ __forceinline__ static void put(T* p, const float2 (&v)[P]) {
        if constexpr (kWhole) st_stream16(p, pack(v));
        else *reinterpret_cast<Word*>(p) = pack(v);
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
    else if (VEC > 1 && reinterpret_cast<uintptr_t>(p) % sizeof(typename V::Word) == 0) V::get(V::load(p + c), v);
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
    // the means, less their groups' refs, and the squares about them of n positions, per
    // channel; k and ref are values, whose difference is exact where they are close
    template <int VEC>
    __device__ __forceinline__ void leave(int n, const Groups<VEC>& g, const float* refs, float* mean,
                                          float* m2) const {
        const float inv = n ? 1.f / float(n) : 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float s = e & 1 ? s1[e / 2].y : s1[e / 2].x, d = s * inv;
            const float q = fmaf(-s, d, e & 1 ? s2[e / 2].y : s2[e / 2].x);
            mean[e] = d - ((e & 1 ? k[e / 2].y : k[e / 2].x) + refs[g.g[e]]);
            m2[e] = q < 0.f ? 0.f : q;  // a NaN stays
        }
    }
};

// Sums over `lanes` consecutive lanes (a power of two).
__device__ __forceinline__ float2 lanes_sum(float2 s, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    }
    return s;
}

// f(item, lane of its team, live) for n items shared out to teams of lanes, the whole
// CTA in step (f holds shuffles); items at or past n are not live.
template <typename F>
__device__ __forceinline__ void by_teams(int n, int team_log2, F f) {
    for (int i0 = 0; i0 < n << team_log2; i0 += kGnBlock) {
        const int i = i0 + int(threadIdx.x), item = i >> team_log2;
        f(item < n ? item : 0, i & ((1 << team_log2) - 1), item < n);
    }
}

// Sets of equal size n as one, given s = (sum of d, sum of squares about the
// sets' means + n d^2) over the sets, d their means less `ref`, the mean of one
// of them: so no more than the number of sets cancels. per: 1 / number of sets.
__device__ __forceinline__ float2 joined(float ref, float2 s, float n, float per) {
    const float off = s.x * per, q = fmaf(-n * s.x, off, s.y);
    return make_float2(ref + off, q < 0.f ? 0.f : q);  // a NaN stays
}

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// a value where CTA `rank` of the cluster keeps it
template <typename V>
__device__ __forceinline__ V* in_cta(const cg::cluster_group& cl, V* p, int rank, int cluster) {
    return cluster > 1 ? cl.map_shared_rank(p, rank) : p;
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
    // the group means (-c1, -c2) = of(group)
    template <typename F>
    __device__ __forceinline__ void means(F of, int c, const GnArgs& a) {
        const Groups<VEC> g(c, a);
        each_channel<VEC>(c1, [&](int e) { return of(g.g[e]).x; });
        each_channel<VEC>(c2, [&](int e) { return of(g.g[e]).y; });
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

// dw, db from P rows of their partial sums [2][C].
inline cudaError_t gn_reduce_channels(const float* chan, int64_t P, int C, float* dw, float* db,
                                      const LaunchCfg& cfg) {
    return reduce_partials(chan, P, 2 * int64_t(C), C, dw, db, cfg);
}

}  // namespace rowops
