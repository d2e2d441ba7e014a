// Sampling: one token a row of logits, cut by top-k, top-p and min-p, drawn with a
// given uniform number. With m the row's largest logit and T its temperature
//   w_j = exp((x_j - m) / T)
// and the columns ordered by value, the largest first, equal ones by index, what is
// kept is the shortest of the prefixes that the cuts allow:
//   top-k   the first k;                              min-p   those with w_j >= min_p;
//   top-p   the fewest (one at least) of top-k's whose sum reaches top_p times top-k's sum.
// The token is the first column, by index, at which the running sum of the kept
// w exceeds u times their sum.
//
// A cut or a draw lies next to a border in some row, where sums in 32 bits, or in
// another order, give another token. So weights are fixed-point numbers of 44
// fractional bits (right to 2^-29 of their value), whose 64-bit sums are exact and
// the same in any order, and a cut is an exact pair: a place in the order of the
// values, as the distance `kd` of a logit's ordered bits from the maximum's, and how
// many of the equal ones, by index, still belong.
//
// A row is held in the shared memory of a cluster of CTAs, each with a share of its
// columns, and every sweep is over that copy. The k-th value, and the value at which
// a mass is reached, are found digit by digit: a histogram of 8 bits of kd (counts, or
// counts and masses) over what agrees with the digits so far, added up over the
// cluster through distributed shared memory.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>

#include "async_ring.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace cg = cooperative_groups;

namespace rowops {
namespace {

constexpr int kBlock = 512, kWarps = kBlock / 32;
constexpr int kCluster = 8;  // the most CTAs of a row
constexpr int kBins = 256;
constexpr int kFraction = 44;
constexpr uint64_t kOne = uint64_t(1) << kFraction;

// 2^(j / 16) in fixed point
struct Roots {
    uint64_t v[16];
};

// A row's weights: 2^-((m - x) c), c = log2(e) / T in two parts.
struct Weights {
    float m, c_hi, c_lo;
    const uint64_t* roots;
    // (m - x) c = zi / 16 - f with |f| <= 1/32 and 2^f - 1 by its series, whose terms
    // past the fifth are below 2^-36. The difference and the product carry their errors
    // along: what is lost is f's own rounding and the series', about 2^-29.
    __device__ __forceinline__ uint64_t operator()(float x) const {
        if (x == m) return kOne;
        const float d = m - x, bb = d - m, dl = (m - (d - bb)) - (x + bb);
        const float t = -d * c_hi;
        if (!(t > -62.f) || x == -INFINITY) return 0;
        const float tl = -(fmaf(d, c_hi, t) + fmaf(d, c_lo, dl * c_hi));
        const float r = fmaf(t, 16.f, 12582912.f);
        const int z = __float_as_int(r) - 0x4b400000;
        const float f = fmaf(r - 12582912.f, -0.0625f, t) + tl;
        const float g = f * fmaf(f, fmaf(f, fmaf(f, fmaf(f, 1.3333558e-3f, 9.6181291e-3f), 5.5504109e-2f), 0.24022651f),
                                 0.69314718f);
        const uint64_t root = roots[z & 15];
        const int64_t w = int64_t(root) + ((int64_t(int32_t(root >> 14)) * __float2int_rn(g * 0x1p35f)) >> 21);
        const int s = -(z >> 4);
        return (uint64_t(w) + ((uint64_t(1) << s) >> 1)) >> s;
    }
};

// bits in the order of the values; -0 is 0
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// What the CTAs of a cluster tell one another.
struct Told {
    float top;
    int first;             // greedy: its first column at the maximum
    uint64_t mass;         // of what lies strictly before the cut
    uint32_t ties;         // at the cut
};

struct Shared {
    uint64_t roots[16];
    uint64_t mass[2][kBins];
    uint32_t count[2][kBins];
    uint64_t warp_mass[kWarps];
    uint32_t warp_count[kWarps];
    float warp_top[kWarps];
    Told own;               // read by the others
    Told all[kCluster];     // written by the others
    // one thread's answers for the CTA
    uint64_t target, before, total;
    uint32_t bin, found;
    float c_hi, c_lo;
    uint32_t kd_min_p;
};

template <typename T>
struct Digits {
    static constexpr int kKey = std::is_same_v<T, float> ? 32 : 16;
};

// A cut: what lies before kd, and the first `ties` at it.
struct Cut {
    uint32_t kd, ties;
};
__device__ __forceinline__ Cut shorter(Cut a, Cut b) {
    return a.kd != b.kd ? (a.kd < b.kd ? a : b) : Cut{a.kd, a.ties < b.ties ? a.ties : b.ties};
}

template <typename T>
struct Row {
    using E = Elem<T>;
    static constexpr int kDrop = 32 - Digits<T>::kKey;
    Shared& sh;
    const T* x;  // this CTA's columns, -inf behind them up to a whole vector
    int n, C, rank;
    uint32_t top_key;
    Weights w;

    __device__ __forceinline__ uint32_t kd(float v) const { return (top_key >> kDrop) - (ordered(v) >> kDrop); }

    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int k = threadIdx.x; k * E::kVec < n; k += kBlock) {
            float v[E::kVec];
            E::unpack(reinterpret_cast<const uint4*>(x)[k], v);
#pragma unroll
            for (int e = 0; e < E::kVec; ++e) f(v[e]);
        }
    }

    // The cut at which the counts reach `k` (MASS false), or the masses reach p times
    // their sum over what `within` keeps. `flip`: which histogram the next level takes;
    // both are zero here and when it returns.
    template <bool MASS>
    __device__ Cut find(cg::cluster_group& cluster, uint32_t k, double p, Cut within, int& flip) {
        uint32_t prefix = 0;
        uint64_t before = 0, target = k;
        for (int shift = Digits<T>::kKey - 8; shift >= 0; shift -= 8, flip ^= 1) {
            each([&](float v) {
                const uint32_t at = kd(v);
                if (shift + 8 < Digits<T>::kKey && (at >> (shift + 8)) != prefix) return;
                if constexpr (MASS) {
                    if (at >= within.kd) return;
                    const uint64_t mass = w(v);
                    if (mass) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[flip][(at >> shift) & 255]), mass);
                } else {
                    atomicAdd(&sh.count[flip][(at >> shift) & 255], 1u);
                }
            });
            cluster.sync();
            // a thread has a bin: its sum over the cluster, then the running sum over the bins
            uint64_t mine = 0, run;
            if (threadIdx.x < kBins) {
                for (int r = 0; r < C; ++r) {
                    const Shared* o = cluster.map_shared_rank(&sh, r);
                    mine += MASS ? o->mass[flip][threadIdx.x] : o->count[flip][threadIdx.x];
                }
                if constexpr (MASS) {  // those equal to the k-th value that are among the first k
                    const bool agrees = shift + 8 == Digits<T>::kKey || (within.kd >> (shift + 8)) == prefix;
                    if (within.ties && agrees && ((within.kd >> shift) & 255) == threadIdx.x)
                        mine += uint64_t(within.ties) * w(value_at(within.kd));
                }
                sh.mass[flip ^ 1][threadIdx.x] = 0;
                sh.count[flip ^ 1][threadIdx.x] = 0;
            }
            run = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t other = __shfl_up_sync(0xffffffffu, run, o);
                if ((threadIdx.x & 31) >= o) run += other;
            }
            const int warp = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 31) sh.warp_mass[warp] = run;
            __syncthreads();
            uint64_t total = 0;
#pragma unroll
            for (int i = 0; i < kBins / 32; ++i) {
                if (i < warp) run += sh.warp_mass[i];
                total += sh.warp_mass[i];
            }
            if (MASS && shift + 8 == Digits<T>::kKey) target = uint64_t(ceil(p * double(total)));
            if (threadIdx.x < kBins && before + run >= target && before + run - mine < target) {
                sh.bin = threadIdx.x;
                sh.before = before + run - mine;
            }
            __syncthreads();
            prefix = prefix << 8 | sh.bin;
            before = sh.before;
        }
        // both histograms are zero for the next search: the last level's is read until all have been here
        cluster.sync();
        if (threadIdx.x < kBins) sh.mass[flip ^ 1][threadIdx.x] = 0, sh.count[flip ^ 1][threadIdx.x] = 0;
        __syncthreads();
        uint64_t ties = target - before;
        if constexpr (MASS) {
            const uint64_t one = w(value_at(prefix));
            ties = one ? (ties + one - 1) / one : 1;
            if (prefix == within.kd && ties > within.ties) ties = within.ties;
        }
        return Cut{prefix, uint32_t(ties < 0xffffffffu ? ties : 0xffffffffu)};
    }

    __device__ __forceinline__ float value_at(uint32_t at) const {
        uint32_t key = ((top_key >> kDrop) - at) << kDrop;
        if (kDrop && !(key & 0x80000000u)) key |= 0xffffu;  // a negative bf16's lower bits of order are ones
        return value_of(key);
    }
};

template <typename T>
__global__ void __launch_bounds__(kBlock) sample_kernel(const __grid_constant__ SampleArgs a, const __grid_constant__ Roots roots,
                                                        int share) {
    using E = Elem<T>;
    __shared__ Shared sh;
    extern __shared__ uint4 held[];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank()), lane = threadIdx.x & 31,
              warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / C;
    const int lo = rank * share, n = a.N - lo < share ? (a.N > lo ? a.N - lo : 0) : share;
    T* x = reinterpret_cast<T*>(held);
    {
        const T* from = static_cast<const T*>(a.logits) + row * a.ld + lo;
        const int whole = (reinterpret_cast<uintptr_t>(from) & 15) == 0 ? n / E::kVec : 0;
        for (int k = threadIdx.x; k < whole; k += kBlock) copy_async<16>(x + k * E::kVec, from + k * E::kVec);
        for (int c = whole * E::kVec + threadIdx.x; c < n; c += kBlock) x[c] = from[c];
        for (int c = n + threadIdx.x; c < (n + E::kVec - 1) / E::kVec * E::kVec; c += kBlock) E::store(x + c, -INFINITY);
        if (threadIdx.x < kBins)
            for (int i = 0; i < 2; ++i) sh.mass[i][threadIdx.x] = 0, sh.count[i][threadIdx.x] = 0;
        if (threadIdx.x < 16) sh.roots[threadIdx.x] = roots.v[threadIdx.x];
        asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
        __syncthreads();
    }
    Row<T> r{sh, x, n, C, rank, 0, {}};

    // the maximum, NaN where there is one
    float top = -INFINITY;
    r.each([&](float v) { top = max_nan(top, v); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.warp_top[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kWarps; ++i) top = max_nan(top, sh.warp_top[i]);
        sh.own.top = top;
    }
    cluster.sync();
    top = -INFINITY;
    for (int i = 0; i < C; ++i) top = max_nan(top, cluster.map_shared_rank(&sh, i)->own.top);
    top += 0.f;
    const bool none = !(top > -INFINITY);  // a NaN, or nothing to draw from
    const float temperature = a.temperature ? a.temperature[row] : a.temperature_all;
    const bool greedy = !(temperature > 0.f);
    r.top_key = ordered(top);

    if (none || greedy) {
        int first = 0x7fffffff;
        if (!none)
            for (int c = threadIdx.x; c < n; c += kBlock)
                if (E::load(x + c) == top) {
                    first = lo + c;
                    break;
                }
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) sh.warp_count[warp] = uint32_t(first);
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kWarps; ++i) first = min(first, int(sh.warp_count[i]));
            cluster.map_shared_rank(&sh, 0)->all[rank].first = first;
        }
        cluster.sync();
        if (rank == 0 && threadIdx.x == 0) {
            for (int i = 0; i < C; ++i) first = min(first, sh.all[i].first);
            a.token[row] = none ? -1 : first;
            if (a.logprob) a.logprob[row] = none ? NAN : 0.f;
        }
        return;
    }

    // the row's numbers in 64 bits, once
    const float min_p = a.min_p ? a.min_p[row] : a.min_p_all, top_p = a.top_p ? a.top_p[row] : a.top_p_all;
    const int top_k = a.top_k ? a.top_k[row] : a.top_k_all;
    if (threadIdx.x == 0) {
        const double c = 1.4426950408889634 / double(temperature);
        sh.c_hi = float(c);
        sh.c_lo = float(c - double(sh.c_hi));
        // the smallest value that min-p keeps: (x - m) / T >= ln(min_p)
        sh.kd_min_p = 0xffffffffu;
        if (min_p > 0.f) {
            const double least = double(top) + double(temperature) * log(double(min_p < 1.f ? min_p : 1.f));
            const float up = least > -3.4028234e38 ? __double2float_ru(least) : -INFINITY;
            uint32_t key = ordered(up);
            if (Row<T>::kDrop && (key & 0x80000000u)) key += 0xffffu;  // the next bf16 (below zero: cut off, it is that)
            sh.kd_min_p = (r.top_key >> Row<T>::kDrop) - (key >> Row<T>::kDrop);
        }
    }
    __syncthreads();
    r.w = Weights{top, sh.c_hi, sh.c_lo, sh.roots};
    Cut cut{sh.kd_min_p, 0xffffffffu};
    int flip = 0;
    Cut within{0xffffffffu, 0u};
    if (top_k > 0 && top_k < a.N) {
        within = r.template find<false>(cluster, uint32_t(top_k), 0., within, flip);
        cut = shorter(cut, within);
    }
    if (top_p < 1.f) cut = shorter(cut, r.template find<true>(cluster, 0u, top_p > 0.f ? double(top_p) : 1e-300, within, flip));

    // what is kept, warp by warp in the order of the columns
    const int part = ((n + kWarps - 1) / kWarps + 31) / 32 * 32, c0 = warp * part, c1 = min(n, c0 + part);
    uint64_t mass = 0;
    uint32_t ties = 0;
    for (int c = c0 + lane; c < c1; c += 32) {
        const float v = E::load(x + c);
        const uint32_t at = r.kd(v);
        if (at < cut.kd) mass += r.w(v);
        ties += at == cut.kd;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) sh.warp_mass[warp] = mass, sh.warp_count[warp] = ties;
    __syncthreads();
    if (threadIdx.x < C) {
        Told t = {};
        for (int i = 0; i < kWarps; ++i) t.mass += sh.warp_mass[i], t.ties += sh.warp_count[i];
        Told* to = &cluster.map_shared_rank(&sh, threadIdx.x)->all[rank];
        to->mass = t.mass;
        to->ties = t.ties;
    }
    cluster.sync();
    const uint64_t one = cut.kd == 0xffffffffu ? 0 : r.w(r.value_at(cut.kd));
    uint64_t sum = 0;
    uint32_t tied = 0;  // of all CTAs
    for (int i = 0; i < C; ++i) {
        sum += sh.all[i].mass;
        tied += sh.all[i].ties;
    }
    sum += uint64_t(min(tied, cut.ties)) * one;
    const float u = a.u[row];
    uint64_t draw = u > 0.f ? uint64_t(double(u) * double(sum)) : 0;
    if (draw >= sum) draw = sum - 1;  // u of 1 and above: the last one kept
    // the CTA, then the warp, then the lane in whose part the running sum exceeds the draw
    uint32_t left = cut.ties;  // ties that still belong
    bool here = false;
    for (int i = 0; i <= rank; ++i) {
        const uint32_t t = min(sh.all[i].ties, left);
        const uint64_t m = sh.all[i].mass + t * one;
        here = draw < m;
        if (i == rank || here) {
            here = here && i == rank;
            break;
        }
        draw -= m;
        left -= t;
    }
    if (!here) return;
    for (int i = 0; i <= warp; ++i) {
        const uint32_t t = min(sh.warp_count[i], left);
        const uint64_t m = sh.warp_mass[i] + t * one;
        here = draw < m;
        if (i == warp || here) {
            here = here && i == warp;
            break;
        }
        draw -= m;
        left -= t;
    }
    if (!here) return;
    for (int c = c0; c < c1; c += 32) {
        const float v = c + lane < c1 ? E::load(x + c + lane) : -INFINITY;
        const uint32_t at = r.kd(v);
        const uint32_t tie = __ballot_sync(0xffffffffu, c + lane < c1 && at == cut.kd);
        const bool in = at < cut.kd || (at == cut.kd && uint32_t(__popc(tie & ((1u << lane) - 1))) < left);
        uint64_t run = c + lane < c1 && in ? r.w(v) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t other = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += other;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, run > draw);
        if (past) {
            if (lane == __ffs(past) - 1) {
                a.token[row] = lo + c + lane;
                if (a.logprob)
                    a.logprob[row] = float((v == top ? 0. : (double(v) - double(top)) / double(temperature)) -
                                           log(double(sum) * 0x1p-44));
            }
            return;
        }
        draw -= __shfl_sync(0xffffffffu, run, 31);
        left -= min(left, uint32_t(__popc(tie)));
    }
}

template <typename T>
cudaError_t launch(const SampleArgs& a, const LaunchCfg& cfg) {
    static const Roots roots = [] {
        Roots t;
        for (int j = 0; j < 16; ++j) t.v[j] = uint64_t(std::llrint(std::exp2(j / 16.0) * double(kOne)));
        return t;
    }();
    constexpr int V = Elem<T>::kVec;
    int C = 1;
    while (C < kCluster && (a.N + C - 1) / C * int(sizeof(T)) > 64 * 1024) C *= 2;
    const int share = ((a.N + C - 1) / C + V - 1) / V * V;
    const size_t smem = size_t(share) * sizeof(T);
    auto k = sample_kernel<T>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem, cfg);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(unsigned(a.M * C));
    lc.blockDim = dim3(kBlock);
    lc.dynamicSmemBytes = smem;
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, k, a, roots, share);
}

}  // namespace

SampleLaunch sample_f32() { return launch<float>; }
SampleLaunch sample_bf16() { return launch<bf16_t>; }

}  // namespace rowops
