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
// fractional bits (right to 2^-29 of their value and 2^-45, half of the last bit: what is below that
// of the maximum's weight is 0 and not drawn), whose 64-bit sums are exact and
// the same in any order, and a cut is an exact pair: a place in the order of the
// values, as the distance `kd` of a logit's ordered bits from the maximum's, and how
// many of the equal ones, by index, still belong.
//
// A row is held in the shared memory of a cluster of CTAs, each with a share of its
// columns, and every sweep is over that copy. One histogram of the values' upper 16
// bits (every value of bf16 a bin of its own) says in which bin the k-th value lies,
// and in which a mass is reached; the bins are counted by the CTAs and added up
// through distributed shared memory. Of bf16 the counts are enough: a bin's mass is its count
// times its value's weight, so weights are computed by the bin and not by the element, and the CTAs'
// own masses follow from their own counts. fp32 values differ within a bin: masses are
// added up beside the counts (in three words of 16 bits and more, each a native 32-bit
// atomic; 64-bit ones in shared memory took fifteen times as long), and the cut's bin is searched: its elements are compared
// with one another if they are few, else digit by digit (61 x 50021, cuts by row and half of the rows greedy, 37 us, by digits always 46).
//
// Bound, for many rows, by shared memory: an atomic an element into the histogram and a look-up an element in the
// CTA that has the draw, banks in conflict (bf16 256 x 131072 with top-p: 110 us, 9.9 of them the reading of
// the logits; 512 rows without cuts 170; fp32 61 x 50021 with every cut in every row 56). For few, by its steps one after
// another, up to eight exchanges within the row's cluster, and the fetching of their instructions (bf16 1 x 32000
// with every cut: 16.5 us on the device). Compact code with the steps as functions is slower in both: 20.5 and 120 us.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>

#include "async_ring.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace cg = cooperative_groups;

namespace rowops {
namespace {

// 512 threads a CTA and shares of 64 KB at most: 110 us for 256 rows of 131072 bf16 with top-p, 170 for 512 without
// cuts; an earlier form of it took 112 and 175, with 256 threads
// and 32 KB 125 and 188, with 512 threads and 32 KB 172 and 236 (twice the CTAs in a row's exchanges).
constexpr int kBlock = 512, kWarps = kBlock / 32;
constexpr int kCluster = 8;  // the most CTAs of a row
constexpr int kDigit = 256;  // bins of a digit
// The histogram: 13 binades of 128 bins below the largest magnitude, for either sign, and one
// bin for what is nearer to zero.
constexpr int kHalf = 13 * 128, kBins = 2 * kHalf + 1, kBinsHeld = (kBins + 1 + 31) / 32 * 32;
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
    // along: what is lost is f's own rounding and the series', about 2^-29 of the weight, and its last bit.
    __device__ __forceinline__ uint64_t operator()(float x) const {
        const float d = m - x, bb = d - m, dl = (m - (d - bb)) - (x + bb);
        float t = -d * c_hi;
        const bool some = t > -62.f;  // (false for a NaN, which -inf times a c of 0 gives)
        t = some ? t : 0.f;
        const float tl = -(fmaf(d, c_hi, t) + fmaf(d, c_lo, dl * c_hi));
        const float r = fmaf(t, 16.f, 12582912.f);
        const int z = __float_as_int(r) - 0x4b400000;
        const float f = fmaf(r - 12582912.f, -0.0625f, t) + tl;
        const float g = f * fmaf(f, fmaf(f, fmaf(f, fmaf(f, 1.3333558e-3f, 9.6181291e-3f), 5.5504109e-2f), 0.24022651f),
                                 0.69314718f);
        const uint64_t root = roots[z & 15];
        const int64_t w = int64_t(root) + ((int64_t(int32_t(root >> 14)) * __float2int_rn(g * 0x1p35f)) >> 21);
        const int s = some ? -(z >> 4) : 0;
        const uint64_t rounded = (uint64_t(w) + ((uint64_t(1) << s) >> 1)) >> s;
        return x == m ? kOne : some ? rounded : 0;  // (no branches: the weights of a vector overlap)
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

// two bf16 at a time; the maximum NaN where there is one
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// What the CTAs of a cluster tell one another.
struct Told {
    float top, low;
    int first;       // greedy: its first column at the maximum
    uint64_t mass;   // of its part of the bins; of what it holds before the cut
    uint32_t count;  // of its part of the bins; of what it holds at the cut
};
// The bin in which a count or a mass is reached, and what lies before it.
struct Found {
    uint32_t bin, count;
    uint64_t mass;
};

struct Shared {
    uint64_t roots[16];
    union {
        uint64_t mass[2][kDigit];  // digits: masses, or counts
        struct {                   // or the elements of a cut's bin, by their distance from its largest key
            uint32_t list[2][kDigit];  // top-k's, top-p's: read by the others
            uint64_t mass[kDigit];     // of the elements of all CTAs
        } few;
    };
    uint32_t listed[2];
    uint64_t mass_before;
    uint64_t warp_mass[kWarps];
    uint32_t warp_count[kWarps];
    float warp_top[kWarps], warp_low[kWarps];
    Told own;             // read by the others
    uint64_t near_zero;   // bf16: the mass of the bin for it, read by the others
    Told all[kCluster], kept[kCluster];  // written by the others
    Found found[2];       // by whoever has the bin
    uint64_t before;
    uint32_t bin;
    float c_hi, c_lo;
    double min_p_below;   // T ln(min_p)
    uint32_t kd_min_p;
};

// A cut: what lies before kd in the order of the values, and the first `ties` at it.
struct Cut {
    uint32_t kd, ties;
};
constexpr uint32_t kNone = 0xffffffffu;
__device__ __forceinline__ Cut shorter(Cut a, Cut b) {
    return a.kd != b.kd ? (a.kd < b.kd ? a : b) : Cut{a.kd, a.ties < b.ties ? a.ties : b.ties};
}

// All of the row's threads: what one has written in its CTA's shared memory, or in another's, is there.
__device__ __forceinline__ void meet(cg::cluster_group& cluster) {
    if (cluster.num_blocks() > 1) cluster.sync();
    else __syncthreads();
}

// Sums over the CTA's threads, or what lies before a thread; every thread calls them.
__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += red[i];
    return v;
}
template <typename N>
__device__ __forceinline__ N block_before(N v, N* red, N* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    N run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N other = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += other;
    }
    __syncthreads();
    if (lane == 31) red[warp] = run;
    __syncthreads();
    N all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) run += red[i];
        all += red[i];
    }
    *total = all;
    return run - v;
}

// 32-bit words of the histogram: counts, and three of every bin's mass, or one and a half of its weight
template <typename T>
constexpr int kHeldWords = std::is_same_v<T, float> ? 4 * kBinsHeld : kBinsHeld / 2 * 5;

template <typename T>
struct Row {
    using E = Elem<T>;
    static constexpr bool kF32 = std::is_same_v<T, float>;
    static constexpr int kKey = kF32 ? 32 : 16, kDrop = 32 - kKey;
    Shared& sh;
    uint32_t* counts;  // [kBinsHeld], and, fp32, three words of each bin's mass
    uint64_t* part_masses;  // [bins / C], and their counts
    uint32_t* part_counts;
    const T* x;        // this CTA's columns, -inf behind them up to a whole vector
    int n, C, rank;
    uint32_t top_key;
    Weights w;
    int most, least;   // upper 15 bits of the magnitudes that have bins: from `least` (1 at least) to `most`
    int half, bins;    // bins of a sign; of the histogram

    __device__ __forceinline__ uint32_t key(float v) const { return ordered(v) >> kDrop; }
    __device__ __forceinline__ uint32_t kd(float v) const { return (top_key >> kDrop) - key(v); }
    __device__ __forceinline__ float value_at(uint32_t at) const {
        uint32_t k = ((top_key >> kDrop) - at) << kDrop;
        if (kDrop && !(k & 0x80000000u)) k |= 0xffffu;  // a negative bf16's lower bits of order are ones
        return value_of(k);
    }

    __device__ __forceinline__ void choose_bins(float low) {
        // (a magnitude's upper 15 bits)
        const uint32_t t = __float_as_uint(w.m) >> 16 & 0x7fffu, l = __float_as_uint(low) >> 16 & 0x7fffu;
        most = int(t > l ? t : l);
        least = most - kHalf + 1 > 1 ? most - kHalf + 1 : 1;
        if (most < 1) most = 1;
        half = most - least + 1;
        bins = 2 * half + 1;
    }
    // the bin of a value by the upper 16 bits of its order; bins and more: below all of them
    __device__ __forceinline__ uint32_t bin_of(uint32_t key16) const {
        const int up = int(key16) - 0x8000, down = 0x7fff - int(key16);
        return up >= least ? uint32_t(most - up) : down >= least ? uint32_t(half + 1 + down - least) : uint32_t(half);
    }
    // the largest such 16 bits in a bin
    __device__ __forceinline__ uint32_t bin_top(uint32_t bin) const {
        return bin < uint32_t(half)   ? 0x8000u + most - bin
               : bin > uint32_t(half) ? 0x7fffu - least - (bin - half - 1)
                                      : 0x8000u + least - 1;
    }
    __device__ __forceinline__ bool near_zero(uint32_t bin) const { return bin == uint32_t(half); }
    // whether a bin's elements are equal
    __device__ __forceinline__ bool single(uint32_t bin) const { return !kF32 && !near_zero(bin); }
    __device__ __forceinline__ uint32_t bin_kd(uint32_t bin) const { return (top_key >> 16) - bin_top(bin); }  // bf16

    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int k = threadIdx.x; k * E::kVec < n; k += kBlock) {
            float v[E::kVec];
            E::unpack(reinterpret_cast<const uint4*>(x)[k], v);
#pragma unroll
            for (int e = 0; e < E::kVec; ++e) f(v[e]);
        }
    }

    // This CTA's histogram. bf16: counts, and the mass near zero; fp32: what is asked for.
    __device__ __forceinline__ void count(bool masses) {
        if constexpr (kF32) {
            for (int k = threadIdx.x; k * E::kVec < n; k += kBlock) {
                float v[E::kVec];
                E::unpack(reinterpret_cast<const uint4*>(x)[k], v);
                uint32_t bin[E::kVec];
#pragma unroll
                for (int e = 0; e < E::kVec; ++e) bin[e] = bin_of(ordered(v[e]) >> 16);
                if (masses) {
                    uint64_t m[E::kVec];
#pragma unroll
                    for (int e = 0; e < E::kVec; ++e) m[e] = w(v[e]);
#pragma unroll
                    for (int e = 0; e < E::kVec; ++e) {
                        if (bin[e] >= uint32_t(bins) || m[e] == 0) continue;
                        atomicAdd(counts + kBinsHeld + bin[e], uint32_t(m[e]) & 0xffffu);
                        atomicAdd(counts + 2 * kBinsHeld + bin[e], uint32_t(m[e] >> 16) & 0xffffu);
                        if (m[e] >> 32) atomicAdd(counts + 3 * kBinsHeld + bin[e], uint32_t(m[e] >> 32));
                        atomicAdd(counts + bin[e], 1u);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < E::kVec; ++e)
                        if (bin[e] < uint32_t(bins)) atomicAdd(counts + bin[e], 1u);
                }
            }
        } else {
            uint64_t near = 0;
            for (int k = threadIdx.x; k * E::kVec < n; k += kBlock) {
                const uint4 u = reinterpret_cast<const uint4*>(x)[k];
                const uint32_t four[4] = {u.x, u.y, u.z, u.w};
                bool any = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int bin = held_bin(e & 1 ? four[e / 2] >> 16 : four[e / 2] & 0xffffu);
                    any = any || bin == half;
                    atomicAdd(counts + bin, 1u);
                }
                if (any)  // few: more than 13 binades below the largest
#pragma unroll 1
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t b = x[k * 8 + e].bits;
                        if (held_bin(b) == half) near += w(__uint_as_float(b << 16));
                    }
            }
            near = block_sum(near, sh.warp_mass);
            if (threadIdx.x == 0) sh.near_zero = near;
        }
    }
    // the bin of a bf16; the one behind all others for what is below them
    __device__ __forceinline__ int held_bin(uint32_t b) const {
        const int up = min(most - int(b), half), down = min(max(int(b) - 0x8000 + half + 1 - least, half), bins);
        return b & 0x8000u ? down : up;
    }

    // bf16: the weights of the bins that this CTA has something in, and of those of its part, 16 upper bits
    // apart from the lower ones; near zero 0.
    __device__ __forceinline__ uint64_t weight(int bin) const {
        const uint16_t* upper = reinterpret_cast<const uint16_t*>(counts + 2 * kBinsHeld);
        return uint64_t(upper[bin]) << 32 | counts[kBinsHeld + bin];
    }
    __device__ __forceinline__ void tabulate() const {
        uint16_t* upper = reinterpret_cast<uint16_t*>(counts + 2 * kBinsHeld);
        const int part = part_bins(), first = rank * part, end = first + part;
#pragma unroll 2
        for (int b = threadIdx.x; b <= bins; b += kBlock) {
            const bool used = b < bins && b != half && (counts[b] || (b >= first && b < end));
            const uint64_t one = used ? w(value_at(bin_kd(b))) : 0;
            counts[kBinsHeld + b] = uint32_t(one);
            upper[b] = uint16_t(one >> 32);
        }
        __syncthreads();
    }

    // The counts and masses of this CTA's part of the bins, over the cluster, in shared
    // memory; a thread's share of them, their sums and what lies before them in the whole order.
    struct Share {
        int first, end;  // of the part
        uint32_t count, count_before;
        uint64_t mass, mass_before;
    };
    __device__ __forceinline__ int part_bins() const { return (bins + C - 1) / C; }
    __device__ __forceinline__ void gather(cg::cluster_group& cluster, bool masses, Share& s) const {
        const int part = part_bins(), each = (part + kBlock - 1) / kBlock;
        constexpr int U = 2;  // bins on their way
        for (int i0 = threadIdx.x; i0 < part; i0 += U * kBlock) {
            uint32_t c[U] = {};
            uint64_t m[U] = {};
#pragma unroll
            for (int r = 0; r < kCluster; ++r)
                if (r < C) {
                    const uint32_t* o = cluster.map_shared_rank(counts, r);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int i = i0 + u * kBlock, bin = rank * part + i;
                        if (i < part && bin < bins) {
                            c[u] += o[bin];
                            if (kF32 && masses)
                                m[u] += o[kBinsHeld + bin] + (uint64_t(o[2 * kBinsHeld + bin]) << 16) +
                                        (uint64_t(o[3 * kBinsHeld + bin]) << 32);
                        }
                    }
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kBlock, bin = rank * part + i;
                if (i >= part) break;
                if (!kF32 && bin < bins) {
                    m[u] = c[u] * weight(bin);
                    if (near_zero(bin))
                        for (int r = 0; r < C; ++r) m[u] += cluster.map_shared_rank(&sh, r)->near_zero;
                }
                part_counts[i] = c[u];
                part_masses[i] = m[u];
            }
        }
        __syncthreads();
        s.first = min(int(threadIdx.x) * each, part);
        s.end = min(s.first + each, part);
        s.count = 0, s.mass = 0;
        for (int i = s.first; i < s.end; ++i) {
            s.count += part_counts[i];
            s.mass += part_masses[i];
        }
    }

    // The thread in whose share the running count (or mass) reaches `goal` tells every CTA.
    template <bool MASS>
    __device__ __forceinline__ void tell(cg::cluster_group& cluster, const Share& s, uint64_t goal) const {
        uint64_t run = MASS ? s.mass_before : s.count_before;
        if (run >= goal || run + (MASS ? s.mass : s.count) < goal) return;
        Found f{uint32_t(rank * part_bins()), s.count_before, s.mass_before};
        int i = s.first;
        for (;; ++i) {
            run += MASS ? part_masses[i] : part_counts[i];
            if (run >= goal || i + 1 >= s.end) break;
            f.count += part_counts[i];
            f.mass += part_masses[i];
        }
        f.bin += uint32_t(i);
        for (int r = 0; r < C; ++r) cluster.map_shared_rank(&sh, r)->found[MASS] = f;
    }

    // The cut in a bin whose elements differ, where the counts (or the masses, of what
    // `within` keeps) reach `goal`, `before` of it in the bins before; *mass becomes the mass of the bin's elements before
    // the cut. Of at most kDigit elements: each CTA lists its own, and every CTA compares each with all, a thread
    // each. Of more: digit by digit (the mass by a sweep, if `want`).
    template <bool MASS>
    __device__ Cut find(cg::cluster_group& cluster, uint32_t bin, uint64_t goal, uint64_t before, Cut within, int& flip,
                        bool want, uint64_t* mass) {
        const uint32_t top = kF32 ? bin_top(bin) << 16 | 0xffffu : bin_top(bin);
        const uint32_t width = near_zero(bin) ? (2u * least << (16 - kDrop)) - 1 : 0xffffu;
        const uint32_t from = (top_key >> kDrop) - top;  // kd of the bin's largest key (mod 2^32: it may be past the maximum's)
        each([&](float v) {
            const uint32_t at = top - key(v);
            if (at > width || (MASS && from + at >= within.kd)) return;
            const uint32_t i = atomicAdd(&sh.listed[MASS], 1u);
            if (i < kDigit) sh.few.list[MASS][i] = at;
        });
        meet(cluster);
        const int i = threadIdx.x;
        uint32_t n = 0, at = 0;
        bool mine = false;
        uint32_t here[kCluster];
#pragma unroll
        for (int r = 0; r < kCluster; ++r) here[r] = r < C ? cluster.map_shared_rank(&sh, r)->listed[MASS] : 0;
        int of = 0;
        uint32_t place = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
            if (uint32_t(i) - n < here[r] && i < kDigit) of = r, place = uint32_t(i) - n, mine = true;
            n += here[r];
        }
        if (mine) at = cluster.map_shared_rank(&sh, of)->few.list[MASS][place % kDigit];
        // those equal to the k-th value that are among the first k: one more element, of their mass
        const uint32_t tie = within.kd - from;
        const bool ties = MASS && within.ties && tie <= width;
        if (n + ties > kDigit) {
            meet(cluster);  // the lists' place becomes the digits'
            if (i < kDigit) sh.mass[0][i] = sh.mass[1][i] = 0;
            __syncthreads();
            const Cut cut = find_digits<MASS>(cluster, bin, goal, before, within, flip);
            if (want) *mass = mass_in(cluster, bin, cut.kd);
            return cut;
        }
        uint32_t* all = sh.few.list[!MASS];
        if (mine) {
            all[i] = at;
            sh.few.mass[i] = w(value_at(from + at));
        } else if (ties && uint32_t(i) == n) {
            at = all[i] = tie;
            sh.few.mass[i] = uint64_t(within.ties) * w(value_at(within.kd));
        }
        n += ties;
        __syncthreads();
        if (uint32_t(i) < n) {
            uint64_t less = 0, equal = 0, mass_less = 0;
            for (uint32_t j = 0; j < n; ++j) {
                const uint32_t other = all[j];
                const uint64_t m = sh.few.mass[j], one = MASS ? m : 1;
                less += other < at ? one : 0;
                equal += other == at ? one : 0;
                if constexpr (!MASS) mass_less += other < at ? m : 0;
            }
            if (before + less < goal && before + less + equal >= goal) {  // (equal ones tell the same)
                sh.bin = at;
                sh.before = before + less;
                sh.mass_before = mass_less;
            }
        }
        __syncthreads();
        if (want) *mass = sh.mass_before;
        return reach<MASS>(from + sh.bin, goal - sh.before, within);
    }
    // The same, of any number of elements, digit by digit of the distance from the bin's largest key. `flip`: which
    // digit's bins are next; both sets are zero here and when it returns.
    template <bool MASS>
    __device__ Cut find_digits(cg::cluster_group& cluster, uint32_t bin, uint64_t goal, uint64_t before, Cut within,
                               int& flip) {
        const uint32_t top = kF32 ? bin_top(bin) << 16 | 0xffffu : bin_top(bin);
        const uint32_t width = near_zero(bin) ? (2u * least << (16 - kDrop)) - 1 : 0xffffu;
        const uint32_t from = (top_key >> kDrop) - top;  // kd of the bin's largest key (mod 2^32: it may be past the maximum's)
        uint32_t prefix = 0;
        const int bits = near_zero(bin) ? kKey : 16;
        for (int shift = bits - 8; shift >= 0; shift -= 8, flip ^= 1) {
            each([&](float v) {
                const uint32_t at = top - key(v);
                if (at > width || (shift + 8 < bits && (at >> (shift + 8)) != prefix)) return;
                const uint32_t d = at >> shift & 255u;
                if constexpr (MASS) {
                    if (from + at >= within.kd) return;
                    const uint64_t mass = w(v);
                    if (mass) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[flip][d]), mass);
                } else {
                    atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[flip][d]), 1ull);
                }
            });
            meet(cluster);
            // a thread has a digit: its sum over the cluster, then what lies before it
            uint64_t mine = 0;
            if (threadIdx.x < kDigit) {
                for (int r = 0; r < C; ++r) mine += cluster.map_shared_rank(&sh, r)->mass[flip][threadIdx.x];
                if constexpr (MASS) {  // those equal to the k-th value that are among the first k
                    const uint32_t at = within.kd - from;
                    if (within.ties && at <= width && (shift + 8 == bits || (at >> (shift + 8)) == prefix) &&
                        (at >> shift & 255u) == threadIdx.x)
                        mine += uint64_t(within.ties) * w(value_at(within.kd));
                }
                sh.mass[flip ^ 1][threadIdx.x] = 0;
            }
            uint64_t total;
            const uint64_t run = before + block_before(mine, sh.warp_mass, &total);
            if (threadIdx.x < kDigit && run < goal && run + mine >= goal) {
                sh.bin = threadIdx.x;
                sh.before = run;
            }
            __syncthreads();
            prefix = prefix << 8 | sh.bin;
            before = sh.before;
        }
        // the last digit's bins are read until all have been here
        meet(cluster);
        if (threadIdx.x < kDigit) sh.mass[flip ^ 1][threadIdx.x] = 0;
        __syncthreads();
        return reach<MASS>(from + prefix, goal - before, within);
    }

    // the cut at kd of which `rest` is still wanted
    template <bool MASS>
    __device__ __forceinline__ Cut reach(uint32_t at, uint64_t rest, Cut within) const {
        if constexpr (MASS) {
            const uint64_t one = w(value_at(at));
            rest = one ? (rest + one - 1) / one : 1;
            if (at == within.kd && rest > within.ties) rest = within.ties;
        }
        return Cut{at, uint32_t(rest < kNone ? rest : kNone)};
    }

    // the cluster's mass of what lies in `bin` before kd
    __device__ uint64_t mass_in(cg::cluster_group& cluster, uint32_t bin, uint32_t at) {
        uint64_t mass = 0;
        each([&](float v) {
            if (bin_of(ordered(v) >> 16) == bin && kd(v) < at) mass += w(v);
        });
        mass = block_sum(mass, sh.warp_mass);
        if (int(threadIdx.x) < C) cluster.map_shared_rank(&sh, threadIdx.x)->kept[rank].mass = mass;
        meet(cluster);
        mass = 0;
        for (int r = 0; r < C; ++r) mass += sh.kept[r].mass;
        meet(cluster);  // (written again by the final sums)
        return mass;
    }

    // The sums of what a warp's columns [c0, c1), whole vectors but for the row's end, hold before
    // the cut, and their ties at it. table: the cut's bin, if that settles it; else -1.
    __device__ __forceinline__ void warp_sums(int c0, int c1, Cut cut, int table, uint64_t* mass, uint32_t* ties) const {
        uint64_t m = 0;
        uint32_t t = 0;
        const float at_cut = cut.kd == kNone ? -INFINITY : value_at(cut.kd);
        for (int c = c0 + (threadIdx.x & 31) * E::kVec; c < c1; c += 32 * E::kVec) {
            const uint4 u = *reinterpret_cast<const uint4*>(x + c);
            if (!kF32 && table >= 0) {
                const uint32_t four[4] = {u.x, u.y, u.z, u.w};
                bool any = false;
#pragma unroll
                for (int e = 0; e < E::kVec; ++e) {
                    const int bin = held_bin(e & 1 ? four[e / 2] >> 16 : four[e / 2] & 0xffffu);
                    if (bin < table) m += weight(bin);
                    t += bin == table;
                    any = any || bin == half;
                }
                if (any && table > half)
#pragma unroll 1
                    for (int e = 0; e < E::kVec; ++e)
                        if (held_bin(read_bits(c + e)) == half) m += w(E::load(x + c + e));
                continue;
            }
            float v[E::kVec];
            E::unpack(u, v);
            float most_here = v[0];
#pragma unroll
            for (int e = 1; e < E::kVec; ++e) most_here = fmaxf(most_here, v[e]);
            if (most_here < at_cut) continue;
            if constexpr (kF32) {
#pragma unroll
                for (int e = 0; e < E::kVec; ++e) {
                    const uint32_t at = kd(v[e]);
                    if (at < cut.kd) m += w(v[e]);
                    t += at == cut.kd;
                }
            } else {
#pragma unroll 1
                for (int e = 0; e < E::kVec; ++e) {
                    const float one = E::load(x + c + e);
                    const uint32_t at = kd(one);
                    if (at < cut.kd) m += w(one);
                    t += at == cut.kd;
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        *mass = m;
        *ties = __reduce_add_sync(0xffffffffu, t);
    }
    __device__ __forceinline__ uint32_t read_bits(int c) const {
        if constexpr (kF32) return 0;
        else return x[c].bits;
    }
};

// part * v, rounded down, or up: exact, where 64-bit floating point would do, at two
// instructions a cycle and SM, what the CTA's every thread needs. part: not negative, at most 1 (above: as 1).
__device__ __forceinline__ uint64_t part_of(float part, uint64_t v, bool up) {
    if (part >= 1.f) return v;
    const uint32_t b = __float_as_uint(part), e = b >> 23;
    const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b;  // part = m 2^-(150 - e)
    const int s = 150 - int(e ? e : 1);                      // at least 24
    uint64_t lo = v * m, hi = __umul64hi(v, m);
    if (up) {  // (a part of 2^-128 and less is more than nothing)
        if (s >= 128) return m != 0;
        const uint64_t one = s >= 64 ? ~uint64_t(0) : (uint64_t(1) << s) - 1;
        lo += one;
        hi += (lo < one) + (s > 64 ? (uint64_t(1) << (s - 64)) - 1 : 0);
    }
    return s >= 128 ? 0 : s >= 64 ? hi >> (s - 64) : (hi << (64 - s)) | (lo >> s);
}

// Of at most 32 parts in order, lane i's with a mass before the cut and ties at it, that in which the
// running sum exceeds *draw; *draw and *left (the ties that still belong) become what they are at
// its begin. Every lane of the warp calls it.
__device__ __forceinline__ int which(uint64_t mass, uint32_t ties, int parts, uint64_t one, uint64_t* draw,
                                     uint32_t* left) {
    const int lane = threadIdx.x & 31;
    if (lane >= parts) mass = 0, ties = 0;
    uint32_t run_ties = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t other = __shfl_up_sync(0xffffffffu, run_ties, o);
        if (lane >= o) run_ties += other;
    }
    const uint32_t kept = min(run_ties, *left), before = min(run_ties - ties, *left);
    mass += (kept - before) * one;
    uint64_t run = mass;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t other = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += other;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, run > *draw);
    const int i = past ? __ffs(past) - 1 : parts - 1;
    *draw -= __shfl_sync(0xffffffffu, run - mass, i);
    *left -= __shfl_sync(0xffffffffu, before, i);
    return i;
}

template <typename T>
__global__ void __launch_bounds__(kBlock, 2) sample_kernel(const __grid_constant__ SampleArgs a,
                                                        const __grid_constant__ Roots roots, int share, bool held) {
    using E = Elem<T>;
    using R = Row<T>;
    __shared__ Shared sh;
    extern __shared__ uint4 dynamic[];
    uint32_t* counts = reinterpret_cast<uint32_t*>(dynamic);
    uint64_t* part_masses = reinterpret_cast<uint64_t*>(counts + (held ? kHeldWords<T> : 0));
    const int part_room = held ? kBinsHeld / int(cg::this_cluster().num_blocks()) : 0;
    uint32_t* part_counts = reinterpret_cast<uint32_t*>(part_masses + part_room);
    T* x = reinterpret_cast<T*>(part_counts + part_room);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank()), lane = threadIdx.x & 31,
              warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / C;
    const int lo = rank * share, n = a.N - lo < share ? (a.N > lo ? a.N - lo : 0) : share;
    const float given = a.temperature ? a.temperature[row] : a.temperature_all;
    const float temperature = given > 0.f ? fmaxf(given, 0x1p-126f) : given;  // (log2(e) / T is finite)
    const float min_p = a.min_p ? a.min_p[row] : a.min_p_all, top_p = a.top_p ? a.top_p[row] : a.top_p_all;
    const int top_k = a.top_k ? a.top_k[row] : a.top_k_all;
    {
        const T* from = static_cast<const T*>(a.logits) + row * a.ld + lo;
        const int whole = (reinterpret_cast<uintptr_t>(from) & 15) == 0 ? n / E::kVec : 0;
        for (int k = threadIdx.x; k < whole; k += kBlock) copy_async<16>(x + k * E::kVec, from + k * E::kVec);
        for (int c = whole * E::kVec + threadIdx.x; c < n; c += kBlock) x[c] = from[c];
        for (int c = n + threadIdx.x; c < (n + E::kVec - 1) / E::kVec * E::kVec; c += kBlock) E::store(x + c, -INFINITY);
        if (threadIdx.x < 2) sh.listed[threadIdx.x] = 0;
        if (held)
            for (int i = threadIdx.x; i < (R::kF32 ? 4 : 1) * kBinsHeld; i += kBlock) counts[i] = 0;
        if (threadIdx.x < 16) sh.roots[threadIdx.x] = roots.v[threadIdx.x];
        asm volatile("cp.async.commit_group;" ::: "memory");
        // what of the row's numbers needs 64 bits, by a thread each while the copies are on their way
        if (threadIdx.x == 32) {
            const double c = 1.4426950408889634 / double(temperature);
            sh.c_hi = float(c);
            sh.c_lo = float(c - double(sh.c_hi));
        }
        if (threadIdx.x == 64 && min_p > 0.f)
            sh.min_p_below = double(temperature) * log(double(min_p < 1.f ? min_p : 1.f));
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
    }
    R r{sh, counts, part_masses, part_counts, x, n, C, rank, 0, {}, 0, 0, 0, 0};

    // the maximum, NaN where there is one, and the minimum
    float top = -INFINITY, low = INFINITY;
    if constexpr (R::kF32) {
        r.each([&](float v) {
            top = max_nan(top, v);
            low = fminf(low, v);
        });
    } else {
        uint32_t t2 = 0xff80ff80u, l2 = 0x7f807f80u;  // two at a time
        for (int k = threadIdx.x; k * 8 < n; k += kBlock) {
            const uint4 u = reinterpret_cast<const uint4*>(x)[k];
            t2 = max2_nan(t2, max2_nan(max2_nan(u.x, u.y), max2_nan(u.z, u.w)));
            l2 = min2(l2, min2(min2(u.x, u.y), min2(u.z, u.w)));
        }
        top = max_nan(__uint_as_float(t2 << 16), __uint_as_float(t2 & 0xffff0000u));
        low = fminf(__uint_as_float(l2 << 16), __uint_as_float(l2 & 0xffff0000u));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    if (lane == 0) sh.warp_top[warp] = top, sh.warp_low[warp] = low;
    __syncthreads();
    if (warp == 0) {
        top = sh.warp_top[lane % kWarps], low = sh.warp_low[lane % kWarps];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
        }
        if (lane == 0) sh.own.top = top, sh.own.low = low;
    }
    meet(cluster);
    {
        const Told& o = cluster.map_shared_rank(&sh, min(lane, C - 1))->own;
        top = o.top, low = o.low;
#pragma unroll
        for (int d = kCluster / 2; d > 0; d >>= 1) {
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
        }
        top = __shfl_sync(0xffffffffu, top, 0), low = __shfl_sync(0xffffffffu, low, 0);
    }
    top += 0.f;
    const bool none = !(top > -INFINITY);  // a NaN, or nothing to draw from
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
        meet(cluster);
        if (rank == 0 && threadIdx.x == 0) {
            for (int i = 0; i < C; ++i) first = min(first, sh.all[i].first);
            a.token[row] = none ? -1 : first;
            if (a.logprob) a.logprob[row] = none ? NAN : 0.f;
        }
        return;
    }

    if (threadIdx.x == 0) {
        // the smallest value that min-p keeps: (x - m) / T >= ln(min_p)
        sh.kd_min_p = kNone;
        if (min_p > 0.f) {
            const double least = double(top) + sh.min_p_below;
            const float up = least > -3.4028234e38 ? __double2float_ru(least) : -INFINITY;
            uint32_t key = ordered(up);
            if (R::kDrop && (key & 0x80000000u)) key += 0xffffu;  // the next bf16 (below zero: cut off, it is that)
            sh.kd_min_p = (r.top_key >> R::kDrop) - (key >> R::kDrop);
        }
    }
    __syncthreads();
    r.w = Weights{top, sh.c_hi, sh.c_lo, sh.roots};
    r.choose_bins(fmaxf(low, top - 43.7f * temperature));  // below: weights of 0 (2^-63)
    const bool cut_k = top_k > 0 && top_k < a.N, cut_p = top_p < 1.f;
    Cut cut{sh.kd_min_p, kNone}, within{kNone, 0u};
    if (!R::kF32 || cut_k || cut_p) {
        r.count(cut_p);
        if constexpr (!R::kF32) r.tabulate();
    }
    if (cut_k || cut_p) {
        meet(cluster);
        int flip = 0;
        typename R::Share s;
        r.gather(cluster, cut_p, s);
        uint32_t counts_here;
        uint64_t masses_here;
        s.count_before = block_before(s.count, sh.warp_count, &counts_here);
        s.mass_before = block_before(s.mass, sh.warp_mass, &masses_here);
        if (int(threadIdx.x) < C) {
            Told* to = &cluster.map_shared_rank(&sh, threadIdx.x)->all[rank];
            to->count = counts_here;
            to->mass = masses_here;
        }
        meet(cluster);
        uint32_t count_all = 0;
        uint64_t mass_all = 0;
        for (int i = 0; i < C; ++i) {
            if (i < rank) s.count_before += sh.all[i].count, s.mass_before += sh.all[i].mass;
            count_all += sh.all[i].count;
            mass_all += sh.all[i].mass;
        }
        Found in{kNone, 0, 0};  // the bin of the k-th value
        if (cut_k && uint32_t(top_k) <= count_all) {  // (else the first k are all that have a weight)
            r.template tell<false>(cluster, s, uint64_t(top_k));
            meet(cluster);
            in = sh.found[0];
            if (r.single(in.bin)) {
                within = Cut{r.bin_kd(in.bin), uint32_t(top_k) - in.count};
                mass_all = in.mass;
            } else {
                uint64_t mass_before = 0;
                within = r.template find<false>(cluster, in.bin, uint64_t(top_k), in.count, within, flip, cut_p, &mass_before);
                if (cut_p) mass_all = in.mass + mass_before;
            }
            mass_all += uint64_t(within.ties) * r.w(r.value_at(within.kd));
            cut = shorter(cut, within);
        }
        if (cut_p) {
            const uint64_t goal = max(part_of(fmaxf(top_p, 0.f), mass_all, true), uint64_t(1));
            Found f = in;
            if (in.bin == kNone || goal <= in.mass) {
                r.template tell<true>(cluster, s, goal);
                meet(cluster);
                f = sh.found[1];
            }
            cut = shorter(cut, r.single(f.bin)
                                   ? r.template reach<true>(r.bin_kd(f.bin), goal - f.mass, within)
                                   : r.template find<true>(cluster, f.bin, goal, f.mass, within, flip, false, nullptr));
        }
    }

    // What this CTA holds before the cut and at it. bf16: by its own counts, unless the cut
    // lies near zero; else by the columns, warp by warp in their order.
    const int part = ((n + kWarps - 1) / kWarps + 32 * E::kVec - 1) / (32 * E::kVec) * (32 * E::kVec);
    const uint64_t one = cut.kd == kNone ? 0 : r.w(r.value_at(cut.kd));
    uint64_t mass = 0;
    uint32_t ties = 0;
    bool by_bins = false;
    int table = -1;
    if constexpr (!R::kF32) {
        uint32_t end = r.bins;  // the cut's bin
        if (cut.kd != kNone) end = min(end, r.bin_of((r.top_key >> 16) - cut.kd));
        by_bins = !r.near_zero(end);
        if (by_bins) {
            table = int(end);
            for (uint32_t b = threadIdx.x; b < end; b += kBlock) mass += counts[b] * r.weight(int(b));
            mass = block_sum(mass, sh.warp_mass);
            if (uint32_t(r.half) < end) mass += sh.near_zero;
            ties = end < uint32_t(r.bins) ? counts[end] : 0;
        }
    }
    auto by_warps = [&] {
        uint64_t m;
        uint32_t t;
        r.warp_sums(warp * part, min(n, (warp + 1) * part), cut, table, &m, &t);
        __syncthreads();
        if (lane == 0) sh.warp_mass[warp] = m, sh.warp_count[warp] = t;
        __syncthreads();
    };
    if (!by_bins) {
        by_warps();
        for (int i = 0; i < kWarps; ++i) mass += sh.warp_mass[i], ties += sh.warp_count[i];
    }
    if (int(threadIdx.x) < C) {
        Told* to = &cluster.map_shared_rank(&sh, threadIdx.x)->kept[rank];
        to->mass = mass;
        to->count = ties;
    }
    meet(cluster);
    uint64_t sum = 0;
    ties = 0;
    for (int i = 0; i < C; ++i) {
        sum += sh.kept[i].mass;
        ties += sh.kept[i].count;
    }
    sum += uint64_t(min(ties, cut.ties)) * one;
    const float u = a.u[row];
    uint64_t draw = u > 0.f ? part_of(u, sum, false) : 0;
    if (draw >= sum) draw = sum - 1;  // u of 1 and above: the last one kept
    // the CTA, the warp's columns, and the 32 columns in which the running sum exceeds the draw
    uint32_t left = cut.ties;
    const Told& mine = sh.kept[min(lane, kCluster - 1)];
    if (which(mine.mass, mine.count, C, one, &draw, &left) != rank) return;
    if (by_bins) by_warps();
    auto of_warps = [&] {
        const int i = min(lane, kWarps - 1);
        return which(sh.warp_mass[i], sh.warp_count[i], kWarps, one, &draw, &left);
    };
    int c0 = of_warps() * part;
    int c1 = min(n, c0 + part);
    if (part > 4 * 32) {  // every warp a sixteenth of them
        const int less = ((c1 - c0 + kWarps - 1) / kWarps + 31) / 32 * 32;  // (whole vectors)
        uint64_t m;
        uint32_t t;
        r.warp_sums(c0 + warp * less, min(c1, c0 + (warp + 1) * less), cut, table, &m, &t);
        __syncthreads();
        if (lane == 0) sh.warp_mass[warp] = m, sh.warp_count[warp] = t;
        __syncthreads();
        c0 += of_warps() * less;
        c1 = min(c1, c0 + less);
    }
    if (warp != 0) return;
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
                if (a.logprob)  // two terms of one sign; sum is at least one
                    a.logprob[row] = -((v == top ? 0.f : (top - v) / temperature) +
                                       log1pf(float(sum - kOne) * 0x1p-44f));
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
    // Shares of 64 KB at most; while the CTAs are fewer than two an SM, of at least 4096 columns.
    int C = 1;
    while (C < kCluster && ((a.N + C - 1) / C * int(sizeof(T)) > 64 * 1024 ||
                            (a.M * C * 2 <= 2 * cfg.num_sms && a.N >= 2 * C * 4096)))
        C *= 2;
    const int share = ((a.N + C - 1) / C + V - 1) / V * V;
    // fp32 rows without top-k and top-p need no histogram, whose room a second CTA of the SM can have
    const bool held = sizeof(T) == 2 || a.top_k || a.top_p || a.top_p_all < 1.f || (a.top_k_all > 0 && a.top_k_all < a.N);
    const size_t smem = size_t(share) * sizeof(T) + (held ? size_t(kHeldWords<T>) * 4 + size_t(kBinsHeld / C) * 12 : 0);
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
    return cudaLaunchKernelEx(&lc, k, a, roots, share, held);
}

}  // namespace

SampleLaunch sample_f32() { return launch<float>; }
SampleLaunch sample_bf16() { return launch<bf16_t>; }

}  // namespace rowops
