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
//
// fp32 131072 x 256, 8 choices: 31 us (4.6 TB/s with the choices), of which the second
// kernel's launch and latency are about 4; its gradient 47 us (5.7 TB/s). With 256 experts
// a CTA has 85 KB of shared memory, so two share an SM, and of clusters of eight 36 fit:
// 288 CTAs, 24% of an SM's warps, where the gradient, with the same shuffles a row and no
// cluster, has 456 and 34%. 64 x 8: 4.1 to 4.8
// and 3.4 us, a launch's latency. bf16 131072 x 60, rows that are no whole vectors: 16
// and 13 us by pairs, 21 and 16 by single elements.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>

#include "async_ring.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace cg = cooperative_groups;

namespace rowops {
namespace {

constexpr int kBlock = 256;
constexpr int kCluster = 8;

// A lane's share of a row: NV vectors of VEC elements, vector j holding columns
// VEC (TL j + tl) .. (16 bytes, a pair of bf16, or one element). FULL: every lane's
// vectors lie within the row. Values are kept
// as pairs for the packed arithmetic (a lone element with a -inf).
template <typename T, int VEC, int NV, bool FULL>
struct Row {
    using E = Elem<T>;
    static constexpr bool kWhole = VEC * sizeof(T) == 16;
    static_assert(kWhole || VEC == 1 || VEC * sizeof(T) == 4, "");
    using Word = std::conditional_t<kWhole, uint4, std::conditional_t<VEC == 1, T, uint32_t>>;
    static constexpr int N = NV * VEC, P = N == 1 ? 1 : N / 2;
    Word w[NV];
    __device__ __forceinline__ static int column(int j, int tl, int TL) { return VEC * (TL * j + tl); }
    // as fp32; columns past E as -inf
    __device__ __forceinline__ void get(int E_, int tl, int TL, float2 (&v)[P]) const {
        float f[N == 1 ? 2 : N];
        if constexpr (N == 1) f[1] = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (kWhole) {
                E::unpack(w[j], f + j * VEC);
            } else if constexpr (VEC == 1) {
                f[j] = E::load(&w[j]);
            } else {
                f[2 * j] = __uint_as_float(w[j] << 16);
                f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
            if constexpr (!FULL) {
                const bool in = column(j, tl, TL) < E_;
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[j * VEC + e] = in ? f[j * VEC + e] : -INFINITY;
            }
        }
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = make_float2(f[2 * k], f[2 * k + 1]);
    }
    __device__ __forceinline__ static void put(T* row, const float2 (&v)[P], int E_, int tl, int TL) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = column(j, tl, TL);
            if (!FULL && c >= E_) continue;
            if constexpr (VEC == 1) {
                E::store(row + c, j & 1 ? v[j / 2].y : v[j / 2].x);
            } else if constexpr (VEC == 2) {
                *reinterpret_cast<uint32_t*>(row + c) = pack_bf16x2(v[j].x, v[j].y);
            } else {
                float f[VEC];
#pragma unroll
                for (int e = 0; e < VEC; e += 2) f[e] = v[(j * VEC + e) / 2].x, f[e + 1] = v[(j * VEC + e) / 2].y;
                st_stream16(row + c, E::pack(f));
            }
        }
    }
    // f(value, column) for the lane's columns
    template <typename V, typename F>
    __device__ __forceinline__ static void each(V (&v)[P], int E_, int tl, int TL, F f) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = column(i / VEC, tl, TL) + i % VEC;
            if (FULL || c < E_) f(i & 1 ? v[i / 2].y : v[i / 2].x, c);
        }
    }
};

// A warp's rows one after the other, `step` apart, kDepth of them on their way: through
// a ring of copies, or (single bf16) one row ahead in registers. With one row ahead in
// either form the kernels waited for memory two thirds of the time.
constexpr int kDepth = 4;

template <typename T, typename I, int VEC, int NV, bool FULL>
struct Rows {
    using R = Row<T, VEC, NV, FULL>;
    using Word = typename R::Word;
    static constexpr bool kRing = sizeof(Word) >= 4;
    Ring<kDepth, NV, kBlock, Word> ring;
    I* choices;  // [kDepth][threads], this thread's
    int64_t rows, step, ahead, ld;
    const T* from;
    const I* choice;
    int E, K, tl, TL;
    R next;
    I next_choice = -1;
    // choice: NULL where the choices are not wanted
    __device__ __forceinline__ Rows(void* smem, const T* logits, const I* experts, int64_t first, int64_t step_,
                                    int64_t rows_, int E_, int K_, int64_t ld_, int tl_, int TL_)
        : ring(static_cast<Word*>(smem)),
          choices(reinterpret_cast<I*>(static_cast<Word*>(smem) + kDepth * NV * kBlock) + threadIdx.x),
          rows(rows_), step(step_), ahead(first), ld(ld_), from(logits + first * ld_),
          choice(experts ? experts + first * K_ : nullptr), E(E_), K(K_), tl(tl_), TL(TL_) {
#pragma unroll
        for (int d = 0; d < (kRing ? kDepth - 1 : 1); ++d) ask();
    }
    __device__ __forceinline__ void ask() {
        const bool there = ahead < rows;
        if constexpr (kRing) {
            if (there) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (FULL || R::column(j, tl, TL) < E) ring.ask(j, from + R::column(j, tl, TL));
                if (choice && tl < K) copy_async<sizeof(I)>(choices + ring.in * kBlock, choice + tl);
            }
            ring.asked();
        } else if (there) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (R::column(j, tl, TL) < E) next.w[j] = from[R::column(j, tl, TL)];
            if (choice && tl < K) next_choice = choice[tl];
        }
        ahead += step;
        from += step * ld;
        if (choice) choice += step * K;
    }
    // the oldest row and the lane's first choice of it; asks for one more
    __device__ __forceinline__ void take(float2 (&v)[R::P], I& first) {
        if constexpr (kRing) {
            ask();
            ring.wait();
            R r;
#pragma unroll
            for (int j = 0; j < NV; ++j) r.w[j] = ring.get(j);
            first = choices[ring.out * kBlock];
            ring.done();
            r.get(E, tl, TL, v);
        } else {
            next.get(E, tl, TL, v);
            first = next_choice;
            ask();
        }
    }
};
template <typename T, typename I, int VEC, int NV>
constexpr size_t rows_smem() {
    constexpr size_t word = VEC * sizeof(T);
    return word < 4 ? 0 : size_t(kDepth) * kBlock * (NV * word + sizeof(I));
}

__device__ __forceinline__ float team_max(float v, int TL) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < TL) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float team_sum(float v, int TL) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < TL) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// v = exp(v - max) of the row, returns 1 / its sum (0 for a row of -inf alone;
// a NaN in the row makes the sum NaN). The maximum is taken off before the product
// with log2(e), which would overflow for logits at the type's lowest value.
template <int P>
__device__ __forceinline__ float row_exp(float2 (&v)[P], int TL) {
    float m = fmaxf(v[0].x, v[0].y);
#pragma unroll
    for (int k = 1; k < P; ++k) m = fmaxf(m, fmaxf(v[k].x, v[k].y));
    m = team_max(m, TL);
    if (m == -INFINITY) m = 0.f;
    float2 s = f2(0.f);
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const float2 t = f2_mul(f2_add(v[k], f2(-m)), f2(kLog2eF));
        v[k] = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        s = f2_add(s, v[k]);
    }
    const float d = team_sum(s.x + s.y, TL);
    return d == 0.f ? 0.f : rcp_approx(d);
}

// P, c: E sums and E + 1 counts; every thread of the CTA. The terms are positive
// and added as a tree, in fp32 (an SM has two lanes for fp64).
__device__ __forceinline__ void finish_loss(const float* P, const int* c, int E, int K, float coef, float* loss,
                                            int64_t* counts, float* red) {
    float t = 0.f;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        t = fmaf(float(c[e]), P[e], t);
        counts[e] = c[e];
    }
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int warps = int(blockDim.x >> 5);
        float s = threadIdx.x < warps ? red[threadIdx.x] : 0.f;
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            const float n = float(c[E]);
            *loss = c[E] == 0 ? 0.f : s / n * (coef * float(E) / (n * float(K)));
            counts[E] = c[E];
        }
    }
}

// (Registers for three CTAs an SM; in fp32 the shared memory leaves two from some 100
// experts on.)
template <typename T, typename I, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(kBlock, NV * VEC <= 16 ? 3 : 1)
    balance_kernel(const T* logits, const I* experts, const uint8_t* mask, int64_t rows, int E, int K, int64_t ld,
                   int tl_log2, float coef, float* loss, int64_t* counts, float* part_p, int* part_c, bool last) {
    using R = Row<T, VEC, NV, FULL>;
    extern __shared__ __align__(16) unsigned char sm[];  // the rows on their way, then:
    __shared__ float red[kBlock / 32];
    float* P = reinterpret_cast<float*>(sm + rows_smem<T, I, VEC, NV>());  // [kBlock / 32][E], row 0 the CTA's
    int* cnt = reinterpret_cast<int*>(P + kBlock / 32 * E);  // [E + 1]
    float* Ps = reinterpret_cast<float*>(cnt + E + 1);      // [E] and [E + 1]: the cluster's, in rank 0
    int* cs = reinterpret_cast<int*>(Ps + E);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int TL = 1 << tl_log2, tl = lane & (TL - 1), sub = lane >> tl_log2, SR = 32 >> tl_log2;
    let_next_start();
    for (int i = threadIdx.x; i <= E; i += kBlock) cnt[i] = 0;
    __syncthreads();

    float2 acc[R::P] = {};
    int n = 0;
    const int64_t step = int64_t(gridDim.x) * (kBlock / 32) * SR;
    const int64_t r0 = (int64_t(blockIdx.x) * (kBlock / 32) + warp) * SR;
    Rows<T, I, VEC, NV, FULL> in(sm, logits, experts, r0 + sub, step, rows, E, K, ld, tl, TL);
    bool taken = r0 + sub < rows && (!mask || mask[r0 + sub]);
    for (int64_t rb = r0; rb < rows; rb += step) {
        const int64_t row = rb + sub;
        const bool live = taken;
        taken = row + step < rows && (!mask || mask[row + step]);
        float2 v[R::P];
        I first;
        in.take(v, first);
        if (live && tl < K) {
            if (first >= 0 && first < E) atomicAdd(&cnt[int(first)], 1);
            for (int k = tl + TL; k < K; k += TL) {
                const I e = experts[row * K + k];
                if (e >= 0 && e < E) atomicAdd(&cnt[int(e)], 1);
            }
        }
        const float inv = row_exp(v, TL);
        if (live) {
#pragma unroll
            for (int k = 0; k < R::P; ++k) acc[k] = f2_fma(v[k], f2(inv), acc[k]);
            if (tl == 0) ++n;
        }
    }
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0 && n) atomicAdd(&cnt[E], n);
#pragma unroll
    for (int k = 0; k < R::P; ++k)
        for (int o = TL; o < 32; o <<= 1) {
            acc[k].x += __shfl_xor_sync(0xffffffffu, acc[k].x, o);
            acc[k].y += __shfl_xor_sync(0xffffffffu, acc[k].y, o);
        }
    if (sub == 0) R::each(acc, E, tl, TL, [&](float s, int c) { P[warp * E + c] = s; });
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
    const int blocks = int(cl.num_blocks()), rank = int(cl.block_rank());
    for (int c = rank * kBlock + int(threadIdx.x); c <= E; c += blocks * kBlock) {
        float s = 0.f;
        int k = 0;
        for (int q = 0; q < blocks; ++q) {
            if (c < E) s += cl.map_shared_rank(P, q)[c];
            k += cl.map_shared_rank(cnt, q)[c];
        }
        if (last) {
            if (c < E) cl.map_shared_rank(Ps, 0)[c] = s;
            cl.map_shared_rank(cs, 0)[c] = k;
        } else {
            const int64_t g = blockIdx.x / blocks;
            if (c < E) part_p[g * E + c] = s;
            part_c[g * (E + 1) + c] = k;
        }
    }
    cl.sync();
    if (last && rank == 0) finish_loss(Ps, cs, E, K, coef, loss, counts, red);
}

// The clusters' partial rows, added up in order, and the loss: one CTA. 1024 / X
// threads share a column (X the smallest power of two >= E).
__global__ void __launch_bounds__(1024)
    balance_finish_kernel(const float* part_p, const int* part_c, int G, int E, int K, float coef, float* loss,
                          int64_t* counts) {
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float red[32];
    __shared__ float tp[1024];
    __shared__ int tc[1024];
    int X = 1;
    while (X < E) X <<= 1;
    const int t = threadIdx.x, e = t & (X - 1), y = t / X, Y = 1024 / X;
    float* P = reinterpret_cast<float*>(sm);  // [E]
    int* c = reinterpret_cast<int*>(P + E);  // [E + 1]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.f;
    int k = 0, took[kBalanceMaxClusters / 32];  // the rows that take part
    if (t < 32)
#pragma unroll
        for (int u = 0; u < kBalanceMaxClusters / 32; ++u) {
            const int g = t + 32 * u;
            took[u] = g < G ? part_c[int64_t(g) * (E + 1) + E] : 0;
        }
    if (e < E) {
        constexpr int U = 16;  // partial rows on their way
        for (int g0 = y; g0 < G; g0 += U * Y) {
            float p[U];
            int n[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = g0 + u * Y;
                p[u] = g < G ? part_p[int64_t(g) * E + e] : 0.f;
                n[u] = g < G ? part_c[int64_t(g) * (E + 1) + e] : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s += p[u];
                k += n[u];
            }
        }
    }
    tp[t] = s;
    tc[t] = k;
    if (t < 32) {
        int n = 0;
#pragma unroll
        for (int u = 0; u < kBalanceMaxClusters / 32; ++u) n += took[u];
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if (t == 0) c[E] = n;
    }
    __syncthreads();
    if (y == 0 && e < E) {
        for (int q = 1; q < Y; ++q) {
            s += tp[q * X + e];
            k += tc[q * X + e];
        }
        P[e] = s;
        c[e] = k;
    }
    __syncthreads();
    finish_loss(P, c, E, K, coef, loss, counts, red);
}

// dlogits of every row; the counts enter as c_e minus their mean, which the
// gradient does not see (sum_j p_j = 1) and which keeps the difference exact
// where the counts are nearly even.
template <typename T, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(kBlock, NV * VEC <= 16 ? 3 : 1)
    balance_backward_kernel(const T* logits, const int64_t* counts, const float* dloss, const uint8_t* mask,
                            T* dlogits, int64_t rows, int E, int K, int64_t ld, int tl_log2, float coef) {
    using R = Row<T, VEC, NV, FULL>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int TL = 1 << tl_log2, tl = lane & (TL - 1), sub = lane >> tl_log2, SR = 32 >> tl_log2;
    extern __shared__ __align__(16) unsigned char sm[];
    const int64_t step = int64_t(gridDim.x) * (kBlock / 32) * SR;
    const int64_t r0 = (int64_t(blockIdx.x) * (kBlock / 32) + warp) * SR;
    Rows<T, int32_t, VEC, NV, FULL> in(sm, logits, nullptr, r0 + sub, step, rows, E, K, ld, tl, TL);
    T* out = dlogits + (r0 + sub) * ld;
    bool taken = r0 + sub < rows && (!mask || mask[r0 + sub]);
    // f_e = dloss coef / (n^2 K) (E c_e - sum c), the difference in whole numbers
    float2 f[R::P] = {};
    {
        int64_t all = 0;
        R::each(f, E, tl, TL, [&](float, int c) { all += counts[c]; });
        for (int o = TL / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        const float n = float(counts[E]), k = n > 0.f ? *dloss / n * (coef / (n * float(K))) : 0.f;
        R::each(f, E, tl, TL, [&](float& v, int c) { v = float(counts[c] * E - all) * k; });
    }
    for (int64_t rb = r0; rb < rows; rb += step, out += step * ld) {
        const int64_t row = rb + sub;
        const bool live = taken;
        taken = row + step < rows && (!mask || mask[row + step]);
        float2 v[R::P];
        int32_t none;
        in.take(v, none);
        const float inv = row_exp(v, TL);
        float2 dot = f2(0.f);
#pragma unroll
        for (int k = 0; k < R::P; ++k) dot = f2_fma(v[k], f[k], dot);
        const float d = team_sum(dot.x + dot.y, TL) * inv;
        if (row < rows) {
#pragma unroll
            for (int k = 0; k < R::P; ++k)
                v[k] = live ? f2_mul(f2_mul(v[k], f2(inv)), f2_add(f[k], f2(-d))) : f2(0.f);
            R::put(out, v, E, tl, TL);
        }
    }
}

struct Shape {
    int nv, tl_log2;  // vectors of a lane (a power of two), lanes of a team
};

// About 16 elements a lane, in vectors, or 4 words: the wider the lane's share, the
// fewer shuffles a row takes; a team's access covers a 32-byte sector.
Shape choose(int E, int vec, bool whole) {
    const int nvec = (E + vec - 1) / vec, per = whole ? 16 / vec : 4;
    int l = whole ? 1 : 0;
    while (l < 5 && (per << l) < nvec) ++l;
    int nv = 1;
    while ((nv << l) < nvec) nv <<= 1;
    return Shape{nv, l};
}

size_t balance_smem(int E) { return size_t(4) * (size_t(kBlock / 32) * E + 2 * (E + 1) + E); }

template <typename T, typename I, int VEC, int NV, bool FULL>
cudaError_t launch_fwd(const void* logits, const void* experts, const uint8_t* mask, int64_t rows, int E, int K,
                       int64_t ld, int tl_log2, float coef, float* loss, int64_t* counts, void* ws,
                       const LaunchCfg& cfg) {
    auto kern = balance_kernel<T, I, VEC, NV, FULL>;
    const size_t smem = balance_smem(E) + rows_smem<T, I, VEC, NV>();
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
        // one wave: with a few clusters more than fit (then 57 where 51 did) the kernel took
        // nearly twice the time
        int n = clusters_on_device(reinterpret_cast<const void*>(kern), kBlock, smem, cl, cfg);
        if (n > kBalanceMaxClusters) n = kBalanceMaxClusters;
        grid = int(std::min<int64_t>((items + cl - 1) / cl, n)) * cl;
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
    cudaLaunchConfig_t fc = {};
    fc.gridDim = dim3(1);
    fc.blockDim = dim3(1024);
    fc.dynamicSmemBytes = size_t(4) * (2 * size_t(E) + 1);
    fc.stream = cfg.stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    fc.attrs = attr;
    fc.numAttrs = 1;
    return cudaLaunchKernelEx(&fc, balance_finish_kernel, static_cast<const float*>(part_p),
                              static_cast<const int*>(part_c), G, E, K, coef, loss, counts);
}

template <typename T, int VEC, int NV, bool FULL>
cudaError_t launch_bwd(const void* logits, const int64_t* counts, const float* dloss, const uint8_t* mask,
                       void* dlogits, int64_t rows, int E, int K, int64_t ld, int tl_log2, float coef,
                       const LaunchCfg& cfg) {
    auto kern = balance_backward_kernel<T, VEC, NV, FULL>;
    const int64_t rows_per_cta = int64_t(kBlock / 32) * (32 >> tl_log2);
    const size_t smem = rows_smem<T, int32_t, VEC, NV>();
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, cfg);
    if (e != cudaSuccess) return e;
    const int grid = grid_for(reinterpret_cast<const void*>(kern), kBlock, smem,
                              (rows + rows_per_cta - 1) / rows_per_cta, cfg);
    kern<<<grid, kBlock, smem, cfg.stream>>>(static_cast<const T*>(logits), counts, dloss, mask,
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

// f(VEC, NV, FULL) of a shape; full rows have instantiations of their own with vectors.
// vec: elements of the widest access; a pair of fp32 goes as two.
template <typename T, typename F>
cudaError_t by_shape(int E, int vec, F f, Shape* shape) {
    constexpr int V = Elem<T>::kVec, PAIR = sizeof(T) == 2 ? 2 : 1;
    vec = vec == V ? V : (vec >= PAIR ? PAIR : 1);
    const Shape s = choose(E, vec, vec == V);
    *shape = s;
    using Yes = std::true_type;
    using No = std::false_type;
    using Vec = std::integral_constant<int, V>;
    if (vec == 1) return by_nv<T, 1>(s.nv, [&](auto nv) { return f(std::integral_constant<int, 1>(), nv, No()); });
    if (vec == PAIR)
        return by_nv<T, PAIR>(s.nv, [&](auto nv) { return f(std::integral_constant<int, PAIR>(), nv, No()); });
    if ((V * s.nv) << s.tl_log2 == E) return by_nv<T, V>(s.nv, [&](auto nv) { return f(Vec(), nv, Yes()); });
    return by_nv<T, V>(s.nv, [&](auto nv) { return f(Vec(), nv, No()); });
}

template <typename T>
cudaError_t balance(const void* logits, const void* experts, bool wide, const uint8_t* mask, int64_t rows, int E,
                    int K, int64_t ld, float coef, float* loss, int64_t* counts, void* ws, int vec,
                    const LaunchCfg& cfg) {
    Shape s;
    return by_shape<T>(
        E, vec,
        [&](auto v, auto nv, auto full) {
            constexpr int VEC = decltype(v)::value, NV = decltype(nv)::value;
            constexpr bool FULL = decltype(full)::value;
            return wide ? launch_fwd<T, int64_t, VEC, NV, FULL>(logits, experts, mask, rows, E, K, ld, s.tl_log2, coef,
                                                                loss, counts, ws, cfg)
                        : launch_fwd<T, int32_t, VEC, NV, FULL>(logits, experts, mask, rows, E, K, ld, s.tl_log2, coef,
                                                                loss, counts, ws, cfg);
        },
        &s);
}

template <typename T>
cudaError_t balance_backward(const void* logits, const int64_t* counts, const float* dloss, const uint8_t* mask,
                             void* dlogits, int64_t rows, int E, int K, int64_t ld, float coef, int vec,
                             const LaunchCfg& cfg) {
    Shape s;
    return by_shape<T>(
        E, vec,
        [&](auto v, auto nv, auto full) {
            return launch_bwd<T, decltype(v)::value, decltype(nv)::value, decltype(full)::value>(
                logits, counts, dloss, mask, dlogits, rows, E, K, ld, s.tl_log2, coef, cfg);
        },
        &s);
}

}  // namespace

BalanceLaunch balance_f32() { return balance<float>; }
BalanceLaunch balance_bf16() { return balance<bf16_t>; }
BalanceBackwardLaunch balance_backward_f32() { return balance_backward<float>; }
BalanceBackwardLaunch balance_backward_bf16() { return balance_backward<bf16_t>; }

}  // namespace rowops
