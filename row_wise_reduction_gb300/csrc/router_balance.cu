// Balance loss of a router, and its gradient. For T rows of logits over E
// experts and the K experts chosen for each row, over the n rows that take part:
//   p = softmax(logits);  c_e = choices of expert e;  P_e = sum_t p_te
//   loss = coef E / (n^2 K) sum_e c_e P_e
//   dlogits_te = dloss coef E / (n^2 K) p_te (c_e - sum_j c_j p_tj)
// Both passes are bound by the logits' traffic (read once; read and written
// once). A team of TL lanes holds a row, NV vectors a lane, so the max, the sum
// and the dot product are a lane's own work plus a butterfly over the team; a
// lane keeps its columns over all rows, so P_e is added up in registers.
//
// Forward: the CTAs of a cluster add up their P_e and c_e through distributed
// shared memory and leave one partial row per cluster; a second kernel adds
// those in a fixed order and forms the loss. A problem that one cluster takes
// finishes in the first kernel.
#include <type_traits>

#include <cooperative_groups.h>

#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace cg = cooperative_groups;

namespace rowops {
namespace {

constexpr int kBlock = 256;
constexpr int kCluster = 8;

// A lane's NV vectors of VEC elements (vector v holds columns VEC (TL v + tl) ..)
// of a row; columns past E come out as -inf.
template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_row(const T* row, int E_, int tl, int TL, float (&v)[NV][VEC]) {
    using E = Elem<T>;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = VEC * (TL * j + tl);
        if constexpr (VEC == 1) {
            v[j][0] = c < E_ ? E::load(row + c) : -INFINITY;
        } else if (c < E_) {
            E::unpack(ld_stream16(row + c), v[j]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[j][e] = -INFINITY;
        }
    }
}

__device__ __forceinline__ float team_max(float v, int TL) {
    for (int o = TL / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float team_sum(float v, int TL) {
    for (int o = TL / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// v = exp(v - max) of the row, returns 1 / its sum (0 for a row of -inf alone;
// a NaN in the row makes the sum NaN)
template <int VEC, int NV>
__device__ __forceinline__ float row_exp(float (&v)[NV][VEC], int TL) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) m = fmaxf(m, v[j][e]);
    m = team_max(m, TL);
    if (m == -INFINITY) m = 0.f;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            v[j][e] = ex2_approx((v[j][e] - m) * kLog2eF);
            s += v[j][e];
        }
    s = team_sum(s, TL);
    return s == 0.f ? 0.f : 1.f / s;
}

__device__ __forceinline__ void finish_loss(const float* P, const int* c, int E, int K, float coef, float* loss,
                                            int64_t* counts, double* red) {
    // P, c: E sums and E + 1 counts; every thread of the CTA
    double t = 0.0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        t += double(c[e]) * double(P[e]);
        counts[e] = c[e];
    }
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < int(blockDim.x >> 5); ++w) s += red[w];
        const double n = double(c[E]);
        *loss = c[E] == 0 ? 0.f : float(s * double(coef) * E / (n * n * K));
        counts[E] = c[E];
    }
}

template <typename T, typename I, int VEC, int NV>
__global__ void __launch_bounds__(kBlock)
    balance_kernel(const T* logits, const I* experts, const uint8_t* mask, int64_t rows, int E, int K, int64_t ld,
                   int tl_log2, float coef, float* loss, int64_t* counts, float* part_p, int* part_c, bool last) {
    extern __shared__ float sm[];
    __shared__ double red[kBlock / 32];
    float* P = sm;                                          // [kBlock / 32][E], row 0 the CTA's
    int* cnt = reinterpret_cast<int*>(sm + kBlock / 32 * E);  // [E + 1]
    float* Ps = reinterpret_cast<float*>(cnt + E + 1);      // [E] and [E + 1]: the cluster's, in rank 0
    int* cs = reinterpret_cast<int*>(Ps + E);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int TL = 1 << tl_log2, tl = lane & (TL - 1), sub = lane >> tl_log2, SR = 32 >> tl_log2;
    for (int i = threadIdx.x; i <= E; i += kBlock) cnt[i] = 0;
    __syncthreads();

    float acc[NV][VEC] = {};
    int n = 0;
    const int64_t step = int64_t(gridDim.x) * (kBlock / 32) * SR;
    for (int64_t rb = (int64_t(blockIdx.x) * (kBlock / 32) + warp) * SR; rb < rows; rb += step) {
        const int64_t row = rb + sub;
        const bool live = row < rows && (!mask || mask[row]);
        float v[NV][VEC];
        if (live) {
            load_row<T, VEC, NV>(logits + row * ld, E, tl, TL, v);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] = -INFINITY;
        }
        if (live)
            for (int k = tl; k < K; k += TL) {
                const I e = experts[row * K + k];
                if (e >= 0 && e < E) atomicAdd(&cnt[int(e)], 1);
            }
        const float inv = row_exp<VEC, NV>(v, TL);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[j][e] = fmaf(v[j][e], inv, acc[j][e]);
        if (live && tl == 0) ++n;
    }
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0 && n) atomicAdd(&cnt[E], n);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            for (int o = TL; o < 32; o <<= 1) acc[j][e] += __shfl_xor_sync(0xffffffffu, acc[j][e], o);
            const int c = VEC * (TL * j + tl) + e;
            if (sub == 0 && c < E) P[warp * E + c] = acc[j][e];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < E; c += kBlock) {
        float s = P[c];
        for (int w = 1; w < kBlock / 32; ++w) s += P[w * E + c];
        P[c] = s;
    }
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    // every CTA adds up its share of the columns over the cluster's CTAs, in
    // order of rank, and leaves the sums in rank 0
    const int R = int(cl.num_blocks()), rank = int(cl.block_rank());
    for (int c = rank * kBlock + int(threadIdx.x); c <= E; c += R * kBlock) {
        float s = 0.f;
        int k = 0;
        for (int q = 0; q < R; ++q) {
            if (c < E) s += cl.map_shared_rank(P, q)[c];
            k += cl.map_shared_rank(cnt, q)[c];
        }
        if (last) {
            if (c < E) cl.map_shared_rank(Ps, 0)[c] = s;
            cl.map_shared_rank(cs, 0)[c] = k;
        } else {
            const int64_t g = blockIdx.x / R;
            if (c < E) part_p[g * E + c] = s;
            part_c[g * (E + 1) + c] = k;
        }
    }
    cl.sync();
    if (last && rank == 0) finish_loss(Ps, cs, E, K, coef, loss, counts, red);
}

// The clusters' partial rows, added up in order, and the loss: one CTA.
__global__ void __launch_bounds__(1024)
    balance_finish_kernel(const float* part_p, const int* part_c, int G, int E, int K, float coef, float* loss,
                          int64_t* counts) {
    extern __shared__ float sm[];
    __shared__ double red[32];
    // 1024 / X threads share a column (X the smallest power of two >= E + 1, at most 1024)
    int X = 1;
    while (X < E + 1 && X < 1024) X <<= 1;
    const int x = threadIdx.x & (X - 1), y = threadIdx.x / X, Y = 1024 / X;
    float* P = sm;                               // [E]
    int* c = reinterpret_cast<int*>(P + E);      // [E + 1]
    float* tp = reinterpret_cast<float*>(c + E + 1);  // [1024]
    int* tc = reinterpret_cast<int*>(tp + 1024);
    for (int c0 = 0; c0 <= E; c0 += X) {
        const int e = c0 + x;
        float s = 0.f;
        int k = 0;
        if (e <= E)
            for (int g = y; g < G; g += Y) {
                if (e < E) s += part_p[int64_t(g) * E + e];
                k += part_c[int64_t(g) * (E + 1) + e];
            }
        tp[threadIdx.x] = s;
        tc[threadIdx.x] = k;
        __syncthreads();
        if (y == 0 && e <= E) {
            for (int q = 1; q < Y; ++q) {
                s += tp[q * X + x];
                k += tc[q * X + x];
            }
            if (e < E) P[e] = s;
            c[e] = k;
        }
        __syncthreads();
    }
    finish_loss(P, c, E, K, coef, loss, counts, red);
}

// dlogits of every row; the counts enter as c_e minus their mean, which the
// gradient does not see (sum_j p_j = 1) and which keeps the difference exact
// where the counts are nearly even.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kBlock)
    balance_backward_kernel(const T* logits, const int64_t* counts, const float* dloss, const uint8_t* mask,
                            T* dlogits, int64_t rows, int E_, int K, int64_t ld, int tl_log2, float coef) {
    using E = Elem<T>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int TL = 1 << tl_log2, tl = lane & (TL - 1), sub = lane >> tl_log2, SR = 32 >> tl_log2;
    // f_e = dloss coef E / (n^2 K) (c_e - mean c)
    float f[NV][VEC];
    {
        int64_t own = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = VEC * (TL * j + tl) + e;
                if (c < E_) own += counts[c];
            }
        for (int o = TL / 2; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
        const double n = double(counts[E_]), mean = double(own) / E_;
        const double k = n > 0.0 ? double(*dloss) * double(coef) * E_ / (n * n * K) : 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = VEC * (TL * j + tl) + e;
                f[j][e] = c < E_ ? float((double(counts[c]) - mean) * k) : 0.f;
            }
    }
    const int64_t step = int64_t(gridDim.x) * (kBlock / 32) * SR;
    for (int64_t rb = (int64_t(blockIdx.x) * (kBlock / 32) + warp) * SR; rb < rows; rb += step) {
        const int64_t row = rb + sub;
        const bool in = row < rows, live = in && (!mask || mask[row]);
        float v[NV][VEC];
        if (live) {
            load_row<T, VEC, NV>(logits + row * ld, E_, tl, TL, v);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] = -INFINITY;
        }
        const float inv = row_exp<VEC, NV>(v, TL);
        float d = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) d = fmaf(v[j][e], f[j][e], d);
        d = team_sum(d, TL) * inv;
        if (in) {
            T* out = dlogits + row * ld;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = VEC * (TL * j + tl);
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = live ? v[j][e] * inv * (f[j][e] - d) : 0.f;
                if (c < E_) {
                    if constexpr (VEC == 1) E::store(out + c, o[0]);
                    else st_stream16(out + c, E::pack(o));
                }
            }
        }
    }
}

struct Shape {
    int nv, tl_log2;  // vectors of a lane (a power of two), lanes of a team
};

// About 16 (vectors) or 4 (single elements) elements a lane: the wider the
// lane's share, the fewer shuffles a row takes; a team's vector access covers at
// least a 32-byte sector.
Shape choose(int E, int vec) {
    const int nvec = (E + vec - 1) / vec, per = vec == 1 ? 4 : 16 / vec;
    int l = vec == 1 ? 0 : 1;
    while (l < 5 && (per << l) < nvec) ++l;
    int nv = 1;
    while ((nv << l) < nvec) nv <<= 1;
    return Shape{nv, l};
}

size_t balance_smem(int E) { return size_t(4) * (size_t(kBlock / 32) * E + 2 * (E + 1) + E); }

template <typename T, typename I, int VEC, int NV>
cudaError_t launch_fwd(const void* logits, const void* experts, const uint8_t* mask, int64_t rows, int E, int K,
                       int64_t ld, int tl_log2, float coef, float* loss, int64_t* counts, void* ws,
                       const LaunchCfg& cfg) {
    auto kern = balance_kernel<T, I, VEC, NV>;
    const size_t smem = balance_smem(E);
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, cfg);
    if (e != cudaSuccess) return e;
    const int64_t rows_per_cta = int64_t(kBlock / 32) * (32 >> tl_log2);
    const int64_t items = (rows + rows_per_cta - 1) / rows_per_cta;
    const int64_t bytes = rows * E * int64_t(sizeof(T));
    int grid, cl;
    if (bytes <= kBalanceOneCluster) {
        cl = items >= kCluster ? kCluster : (items >= 4 ? 4 : (items >= 2 ? 2 : 1));
        grid = cl;
    } else {
        cl = kCluster;
        grid = grid_for(reinterpret_cast<const void*>(kern), kBlock, smem, items, cfg);
        grid = (grid + cl - 1) / cl * cl;
        if (grid > kBalanceMaxClusters * cl) grid = kBalanceMaxClusters * cl;
    }
    const int G = grid / cl;
    float* part_p = static_cast<float*>(ws);
    int* part_c = reinterpret_cast<int*>(part_p + size_t(G) * E);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(unsigned(grid));
    lc.blockDim = dim3(kBlock);
    lc.dynamicSmemBytes = smem;
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cl);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    e = cudaLaunchKernelEx(&lc, kern, static_cast<const T*>(logits), static_cast<const I*>(experts), mask, rows, E, K,
                           ld, tl_log2, coef, loss, counts, part_p, part_c, G == 1);
    if (e != cudaSuccess || G == 1) return e;
    const size_t fs = size_t(4) * (2 * size_t(E) + 1 + 2048);
    balance_finish_kernel<<<1, 1024, fs, cfg.stream>>>(part_p, part_c, G, E, K, coef, loss, counts);
    return cudaGetLastError();
}

template <typename T, int VEC, int NV>
cudaError_t launch_bwd(const void* logits, const int64_t* counts, const float* dloss, const uint8_t* mask,
                       void* dlogits, int64_t rows, int E, int K, int64_t ld, int tl_log2, float coef,
                       const LaunchCfg& cfg) {
    auto kern = balance_backward_kernel<T, VEC, NV>;
    const int64_t rows_per_cta = int64_t(kBlock / 32) * (32 >> tl_log2);
    const int grid = grid_for(reinterpret_cast<const void*>(kern), kBlock, 0, (rows + rows_per_cta - 1) / rows_per_cta,
                              cfg);
    kern<<<grid, kBlock, 0, cfg.stream>>>(static_cast<const T*>(logits), counts, dloss, mask,
                                          static_cast<T*>(dlogits), rows, E, K, ld, tl_log2, coef);
    return cudaGetLastError();
}

// NV of the vector forms reach kBalanceMaxExperts / (32 VEC), of the element form
// kBalanceMaxExperts / 32
template <typename T, int VEC, typename F>
cudaError_t by_nv(int nv, F f) {
    static_assert(kBalanceMaxExperts == 1024, "");
    switch (nv) {
        case 1: return f(std::integral_constant<int, 1>());
        case 2: return f(std::integral_constant<int, 2>());
        case 4: return f(std::integral_constant<int, 4>());
        case 8:
            if constexpr (8 * VEC <= 32) return f(std::integral_constant<int, 8>());
            break;
        case 16:
            if constexpr (16 * VEC <= 32) return f(std::integral_constant<int, 16>());
            break;
        case 32:
            if constexpr (32 * VEC <= 32) return f(std::integral_constant<int, 32>());
            break;
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t balance(const void* logits, const void* experts, bool wide, const uint8_t* mask, int64_t rows, int E,
                    int K, int64_t ld, float coef, float* loss, int64_t* counts, void* ws, bool vec,
                    const LaunchCfg& cfg) {
    auto run = [&](auto V) {
        constexpr int VEC = decltype(V)::value;
        const Shape s = choose(E, VEC);
        return by_nv<T, VEC>(s.nv, [&](auto NV) {
            return wide ? launch_fwd<T, int64_t, VEC, decltype(NV)::value>(logits, experts, mask, rows, E, K, ld,
                                                                           s.tl_log2, coef, loss, counts, ws, cfg)
                        : launch_fwd<T, int32_t, VEC, decltype(NV)::value>(logits, experts, mask, rows, E, K, ld,
                                                                           s.tl_log2, coef, loss, counts, ws, cfg);
        });
    };
    return vec ? run(std::integral_constant<int, Elem<T>::kVec>()) : run(std::integral_constant<int, 1>());
}

template <typename T>
cudaError_t balance_backward(const void* logits, const int64_t* counts, const float* dloss, const uint8_t* mask,
                             void* dlogits, int64_t rows, int E, int K, int64_t ld, float coef, bool vec,
                             const LaunchCfg& cfg) {
    auto run = [&](auto V) {
        constexpr int VEC = decltype(V)::value;
        const Shape s = choose(E, VEC);
        return by_nv<T, VEC>(s.nv, [&](auto NV) {
            return launch_bwd<T, VEC, decltype(NV)::value>(logits, counts, dloss, mask, dlogits, rows, E, K, ld,
                                                           s.tl_log2, coef, cfg);
        });
    };
    return vec ? run(std::integral_constant<int, Elem<T>::kVec>()) : run(std::integral_constant<int, 1>());
}

}  // namespace

BalanceLaunch balance_f32() { return balance<float>; }
BalanceLaunch balance_bf16() { return balance<bf16_t>; }
BalanceBackwardLaunch balance_backward_f32() { return balance_backward<float>; }
BalanceBackwardLaunch balance_backward_bf16() { return balance_backward<bf16_t>; }

}  // namespace rowops
