// RMSNorm (with the residual's addition) and its result in 8 bits with scales:
//   s = x + residual as the I/O type stores it;  y = s w / sqrt(mean(s^2) + eps)
//   scale = max(max|y| / 448, 2^-126) over a row or `group` columns;  q = e4m3(y / scale)
// y itself is never rounded nor stored: with inv = 1 / sqrt(...), max|y| = inv max|s w|,
// so the sum of squares and the largest magnitudes are one pass over the row and one
// reduction, and the quotients follow from the registers that hold s w (which has to stay in fp32: groups where it does
// not, done again as s inv w, would have cost the kernels registers, fp32 8192 x 8192 131 to 159 us). Bound by the
// traffic: x (and the residual, in and out) and one byte out. Measured: bf16 16384 x 8192 with
// residual, groups of 128, 149 us (139 at the rate of a copy); 256 x 8192 4.1 us; fp32 rows off a 16-byte
// boundary, 1501 x 4099 in groups of 64, 14.6 to 15.6 us for 4.6; bf16 16384 x 4097 with residual 156 (a scale a row) to 178
// (groups of 128) for 69: neither memory nor issue (50% of it) is the bound there, but chains of dependent steps in few
// warps (27% of an SM's), a word of 4 or 2 bytes at a time.
#pragma once

#include <algorithm>

#include "async_ring.cuh"
#include "e4m3.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace rowops {

// A row's vectors, of V = 16 bytes' columns each, move in pieces of 16 bytes, 4, or 2 (single bf16), by the
// rows' alignment; the rest of the work goes by vectors whatever the pieces.
template <int PIECE>
__device__ __forceinline__ uint4 load_vector(const void* p, int bytes) {
    if constexpr (PIECE == 16) return *static_cast<const uint4*>(p);
    uint32_t w[4] = {0, 0, 0, 0};
    if constexpr (PIECE == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * i < bytes) w[i] = static_cast<const uint32_t*>(p)[i];
    }
    if constexpr (PIECE == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (2 * i < bytes) w[i / 2] |= uint32_t(static_cast<const uint16_t*>(p)[i]) << (i % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int PIECE>
__device__ __forceinline__ void store_vector(void* p, const uint4& v, int bytes) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (PIECE == 16) st_stream16(p, v);
    if constexpr (PIECE == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * i < bytes) static_cast<uint32_t*>(p)[i] = w[i];
    }
    if constexpr (PIECE == 2) {
        char* c = static_cast<char*>(p);
        if (bytes < 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (2 * i < bytes) reinterpret_cast<uint16_t*>(c)[i] = uint16_t(w[i / 2] >> (i % 2 * 16));
        } else if (reinterpret_cast<uintptr_t>(p) & 2) {
            *reinterpret_cast<uint16_t*>(c) = uint16_t(w[0]);
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(c + 4 * i + 2) = w[i] >> 16 | w[i + 1] << 16;
            *reinterpret_cast<uint16_t*>(c + 14) = uint16_t(w[3] >> 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(c)[i] = w[i];
        }
    }
}

// the first n of N quotients as e4m3 bytes; whole: all of them, at an address aligned to N
template <int N>
__device__ __forceinline__ void store_e4m3(uint8_t* q, const float (&f)[N], bool whole, int n) {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const uint32_t two = to_e4m3x2(f[i], f[i + 1]);
        w[i / 4] = i % 4 ? w[i / 4] | two << 16 : two;
    }
    if (whole) {
        if constexpr (N == 4) asm volatile("st.global.cs.u32 [%0], %1;" ::"l"(q), "r"(w[0]) : "memory");
        if constexpr (N == 8) asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(q), "r"(w[0]), "r"(w[1]) : "memory");
    } else if (n < N || (reinterpret_cast<uintptr_t>(q) & 1)) {
        if (n == N) {  // one, pairs, one
            q[0] = uint8_t(w[0]);
#pragma unroll
            for (int i = 1; i < N - 1; i += 2)
                *reinterpret_cast<uint16_t*>(q + i) =
                    uint16_t(i % 4 == 1 ? w[i / 4] >> 8 : w[i / 4] >> 24 | w[i / 4 + 1 < N / 4 ? i / 4 + 1 : 0] << 8);
            q[N - 1] = uint8_t(w[N / 4 - 1] >> 24);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < n) q[i] = uint8_t(w[i / 4] >> (i % 4 * 8));
        }
    } else if (reinterpret_cast<uintptr_t>(q) & 2) {
#pragma unroll
        for (int i = 0; i < N; i += 2) *reinterpret_cast<uint16_t*>(q + i) = uint16_t(w[i / 4] >> (i % 4 * 8));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<uint32_t*>(q + i) = w[i / 4];
    }
}

enum QuantMode { kQuantRow, kQuantLanes, kQuantGroups };

// The most threads of a CTA. Four vectors a thread in small pieces: fewer, so that two CTAs share an SM's registers
// (fp32 1501 x 4099, 288 threads a row: 14.6 us instead of 18).
constexpr int kQuantThreads = 512;
__host__ __device__ constexpr int quant_threads(int piece, int vpt) { return piece < 16 && vpt == 4 ? 320 : kQuantThreads; }

// A row for every `tpr` threads, VPT vectors a thread; the vectors come through rings of copies,
// each thread's its own (single bf16 straight to the registers). The weights stay in registers, at eight vectors a thread
// they are read again for every row.
// kQuantLanes: a group is 2^lanes_log2 lanes of a warp. kQuantGroups:
// any multiple of 32 columns; the maxima of every 32 columns meet in shared memory, in one of three
// arrays: a row's is cleared two barriers before it is used again. `aligned`: q's rows start at multiples of V.
template <typename T, int PIECE, bool RES, int VPT, int D, QuantMode MODE>
__global__ void __launch_bounds__(quant_threads(PIECE, VPT), quant_threads(PIECE, VPT) < kQuantThreads ? 2 : 0)
    rms_quant_kernel(const __grid_constant__ QuantArgs a, int tpr, int lanes_log2, int groups, bool aligned) {
    using E = Elem<T>;
    constexpr int V = E::kVec, S = RES ? 2 : 1;
    constexpr bool kRing = PIECE >= 4, kKept = VPT <= 4;
    extern __shared__ uint4 dynamic[];
    __shared__ float2 red[2][kQuantThreads / 32];
    const int t = threadIdx.x % tpr, team = threadIdx.x / tpr, teams = blockDim.x / tpr, lane = threadIdx.x & 31,
              warp = threadIdx.x >> 5, w0 = team * (tpr / 32), warps = tpr / 32;
    unsigned* tops = reinterpret_cast<unsigned*>(dynamic) + team * 3 * groups;
    uint4* ring = dynamic + (MODE == kQuantGroups ? (teams * 3 * groups * 4 + 15) / 16 : 0) + threadIdx.x;
    const int64_t step = int64_t(gridDim.x) * teams;
    const int N = int(a.N), vectors = (N + V - 1) / V;
    auto meet = [&] {
        if (tpr > 32) asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(tpr) : "memory");
        else __syncwarp();
    };
    auto bytes = [&](int k) { return PIECE == 16 ? 16 : min(16, (N - k * V) * E::kBytes); };  // of vector k
    int64_t row = int64_t(blockIdx.x) * teams + team, asked = row;
    auto ask_vector = [&](int place, const void* tensor, int k) {
        const char* from = static_cast<const char*>(tensor) + (asked * a.ld + k * V) * E::kBytes;
        uint4* to = ring + place * blockDim.x;
        if constexpr (PIECE == 16) {
            copy_async<16>(to, from);
        } else if constexpr (PIECE == 4) {
            const int n = bytes(k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * i < n) copy_async<4>(reinterpret_cast<char*>(to) + 4 * i, from + 4 * i);
        }
    };
    auto ask = [&](int slot) {
        if constexpr (kRing) {
            if (asked < a.M) {
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (t + j * tpr < vectors) {
                        ask_vector(slot * VPT * S + j, a.x, t + j * tpr);
                        if constexpr (RES) ask_vector(slot * VPT * S + VPT + j, a.residual, t + j * tpr);
                    }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            asked += step;
        }
    };
    auto take_vector = [&](int place, const void* tensor, int64_t at, int k) {
        if constexpr (kRing) return ring[place * blockDim.x];
        else return load_vector<PIECE>(static_cast<const T*>(tensor) + at, bytes(k));
    };
    // What lies behind a row's end, which no copy reaches, counts as 0. (The braces matter: without them nvcc 13.0 drops
    // the loop behind the pragma together with this statement, where that is not instantiated.)
    if constexpr (PIECE == 4) {
        for (int i = 0; i < D * VPT * S; ++i) {
            const int k = t + i % VPT * tpr;
            if (k == vectors - 1)
                for (int e = bytes(k) / 4; e < 4; ++e) reinterpret_cast<uint32_t*>(ring + i * blockDim.x)[e] = 0;
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) ask(d);
    uint4 w[kKept ? VPT : 1];
    auto weights = [&](int k) {
        const float ones[V] = {1.f, 1.f, 1.f, 1.f};
        if constexpr (V == 8) {
            const uint32_t one = 0x3f803f80u;
            return a.w ? load_vector<PIECE>(static_cast<const T*>(a.w) + k * V, bytes(k)) : make_uint4(one, one, one, one);
        } else {
            return a.w ? load_vector<PIECE>(static_cast<const T*>(a.w) + k * V, bytes(k)) : E::pack(ones);
        }
    };
    if constexpr (kKept) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (t + j * tpr < vectors) w[j] = weights(t + j * tpr);
    }
    if constexpr (MODE == kQuantGroups) {
        for (int i = t; i < 3 * groups; i += tpr) tops[i] = 0;
        meet();
    }
    const float inv_n = 1.f / float(N);
    int slot = 0, third = 0;
    for (int turn = 0; row < a.M; row += step, turn ^= 1) {
        if constexpr (kRing) asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
        float2 p[VPT][V / 2];  // s w
        float2 sq = make_float2(0.f, 0.f);
        float sum, top[MODE == kQuantLanes ? VPT : 1] = {};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = t + j * tpr;
            float most = 0.f;
            if (k < vectors) {
                const int64_t at = row * a.ld + k * V;
                uint4 x = take_vector(slot * VPT * S + j, a.x, at, k);
                float s[V], ws[V];
                E::unpack(x, s);
                if constexpr (RES) {
                    const uint4 r4 = take_vector(slot * VPT * S + VPT + j, a.residual, at, k);
                    float r[V];
                    E::unpack(r4, r);
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float2 two = f2_add(make_float2(s[e], s[e + 1]), make_float2(r[e], r[e + 1]));
                        s[e] = two.x, s[e + 1] = two.y;
                    }
                    x = E::pack(s);
                    store_vector<PIECE>(static_cast<T*>(a.residual_out) + at, x, bytes(k));
                    E::unpack(x, s);
                }
                E::unpack(kKept ? w[kKept ? j : 0] : weights(k), ws);
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float2 two = make_float2(s[e], s[e + 1]);
                    sq = f2_fma(two, two, sq);
                    p[j][e / 2] = f2_mul(two, make_float2(ws[e], ws[e + 1]));
                    most = max_nan(most, max_nan(fabsf(p[j][e / 2].x), fabsf(p[j][e / 2].y)));
                }
            }
            if constexpr (MODE == kQuantRow) top[0] = max_nan(top[0], most);
            if constexpr (MODE == kQuantLanes) {
#pragma unroll
                for (int o = 0; o < 5; ++o)
                    if (o < lanes_log2) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 1 << o));
                top[j] = most;
            }
            if constexpr (MODE == kQuantGroups) {  // (bits of what is not negative are in order, a NaN's above all)
#pragma unroll
                for (int o = 1; o < 32 / V; o <<= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
                if (k < vectors && lane % (32 / V) == 0)
                    atomicMax(tops + third * groups + k * V / int(a.group), __float_as_uint(most));
            }
        }
        ask(slot);
        slot = slot + 1 == D ? 0 : slot + 1;
        sum = sq.x + sq.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if constexpr (MODE == kQuantRow) top[0] = max_nan(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
        }
        if (tpr > 32) {
            if (lane == 0) red[turn][warp] = make_float2(sum, top[0]);
            meet();
            sum = 0.f;
#pragma unroll 4
            for (int i = 0; i < warps; ++i) {
                const float2 o = red[turn][w0 + i];
                sum += o.x;
                if constexpr (MODE == kQuantRow) top[0] = max_nan(top[0], o.y);
            }
        } else {
            meet();
        }
        const float inv = rsqrtf(sum * inv_n + a.eps);
        if constexpr (MODE == kQuantGroups) {
            unsigned* clear = tops + (third == 0 ? 2 : third - 1) * groups;
            for (int i = t; i < groups; i += tpr) clear[i] = 0;
        }
        float scale = MODE == kQuantRow ? quant_scale(top[0] * inv) : 0.f;
        if (MODE == kQuantRow && t == 0) a.scales[row] = scale;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = t + j * tpr;
            if (k >= vectors) continue;
            if constexpr (MODE == kQuantLanes) {
                scale = quant_scale(top[j] * inv);
                if ((lane & ((1 << lanes_log2) - 1)) == 0) a.scales[row * groups + (k >> lanes_log2)] = scale;
            }
            if constexpr (MODE == kQuantGroups) {
                const int g = k * V / int(a.group);
                scale = quant_scale(__uint_as_float(tops[third * groups + g]) * inv);
                if (k * V - g * int(a.group) == 0) a.scales[row * groups + g] = scale;
            }
            const float f = rcp_approx(scale);
            float both = inv * f;
            if (both > 3.4e38f) {  // then one after the other
#pragma unroll
                for (int e = 0; e < V / 2; ++e) p[j][e] = f2_mul(p[j][e], f2(inv));
                both = f;
            }
            float y[V];
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float2 two = f2_mul(p[j][e / 2], f2(both));
                y[e] = two.x, y[e + 1] = two.y;
            }
            const int n = bytes(k) / E::kBytes;
            store_e4m3(static_cast<uint8_t*>(a.q) + row * a.ldq + k * V, y, PIECE == 16 || (aligned && n == V), n);
        }
        third = third == 2 ? 0 : third + 1;
    }
    if constexpr (kRing) asm volatile("cp.async.wait_all;" ::: "memory");
}

// One CTA per row, any length and layout: rows of more words than a CTA holds. Pass 1 forms s (writing residual_out)
// and the sum of squares; then a warp takes a group at a time, its largest
// magnitude and its quotients (the whole row is one group of the CTA).
constexpr int kLoopBlock = 512;

template <typename T, bool RES>
__global__ void __launch_bounds__(kLoopBlock) rms_quant_looped_kernel(const QuantArgs a) {
    using E = Elem<T>;
    __shared__ float red[2][2][kLoopBlock / 32];  // alternate per row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* w = static_cast<const T*>(a.w);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        const T* x = static_cast<const T*>(a.x) + row * a.ld;
        const T* src = RES ? static_cast<T*>(a.residual_out) + row * a.ld : x;
        uint8_t* q = static_cast<uint8_t*>(a.q) + row * a.ldq;
        float sum = 0.f, top = 0.f;
        for (int64_t c = threadIdx.x; c < a.N; c += kLoopBlock) {
            float s = E::load(x + c);
            if constexpr (RES) {
                s = E::round(s + E::load(static_cast<const T*>(a.residual) + row * a.ld + c));
                E::store(static_cast<T*>(a.residual_out) + row * a.ld + c, s);
            }
            sum = fmaf(s, s, sum);
            if (a.group == a.N) top = max_nan(top, fabsf(w ? s * E::load(w + c) : s));
        }
        sum = group_reduce<kLoopBlock>(sum, red[turn][0], OpSum());
        const float inv = rsqrtf(sum / float(a.N) + a.eps);
        if (a.group == a.N) {
            top = group_reduce<kLoopBlock>(top, red[turn][1], OpMaxNan());
            const float scale = quant_scale(top * inv);
            if (threadIdx.x == 0) a.scales[row] = scale;
            const float f = 1.f / scale;  // (apart from inv: the product of the two may overflow)
            for (int64_t c = threadIdx.x; c < a.N; c += kLoopBlock) {
                const float s = E::load(src + c);
                q[c] = to_e4m3(s * (w ? E::load(w + c) : 1.f) * inv * f);
            }
            continue;
        }
        const int64_t groups = (a.N + a.group - 1) / a.group;
        for (int64_t g = warp; g < groups; g += kLoopBlock / 32) {
            const int64_t c0 = g * a.group, c1 = c0 + a.group < a.N ? c0 + a.group : a.N;
            top = 0.f;
            for (int64_t c = c0 + lane; c < c1; c += 32)
                top = max_nan(top, fabsf(E::load(src + c) * (w ? E::load(w + c) : 1.f)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float scale = quant_scale(top * inv), f = 1.f / scale;
            if (lane == 0) a.scales[row * groups + g] = scale;
            for (int64_t c = c0 + lane; c < c1; c += 32)
                q[c] = to_e4m3(E::load(src + c) * (w ? E::load(w + c) : 1.f) * inv * f);
        }
    }
}

// Threads of a row and vectors of a thread. Many rows: four vectors a thread, so that a row's
// reduction costs few instructions a byte; eight where four would leave an SM's room for 512 threads (by their
// registers) to fewer than 416, or take more than 512 a row. At most one row an SM: as many threads as the row has
// vectors, up to 512, since one row's latency is what counts then.
// Steps of the ring: with a residual and CTAs of 256 threads one (while a row is worked on, the next comes into
// the place that it was read from): bf16 16384 x 8192 took 150 us, with two 158, with three 161. Where one
// CTA has the SM, or without a residual, two: fp32 8192 x 8192 131 us, with one 142; bf16 16384 x 4096
// without residual 36, with one 40.
struct QuantShape {
    int tpr, vpt, teams;
};
inline bool quant_shape(int64_t vectors, int64_t M, int piece, const LaunchCfg& cfg, QuantShape* s) {
    auto threads = [&](int vpt) { return ((vectors + vpt - 1) / vpt + 31) / 32 * 32; };
    int vpt = 4;
    const int64_t four = threads(4);
    if (piece == 16 ? four > 256 && (four > kQuantThreads || four < 416) : four > quant_threads(piece, 4)) vpt = 8;
    if (M <= cfg.num_sms)
        while (vpt > 1 && threads(vpt / 2) <= quant_threads(piece, vpt / 2)) vpt /= 2;
    const int64_t tpr = threads(vpt);
    if (tpr > kQuantThreads) return false;
    s->tpr = int(tpr);
    s->vpt = vpt;
    s->teams = int(std::max<int64_t>(1, 256 / tpr));
    return true;
}

template <typename T, int PIECE, bool RES, int VPT, int D, QuantMode MODE>
cudaError_t launch_quant(const QuantArgs& a, const QuantShape& s, int lanes_log2, int groups, const LaunchCfg& cfg) {
    auto k = rms_quant_kernel<T, PIECE, RES, VPT, D, MODE>;
    constexpr int V = Elem<T>::kVec;
    const int block = s.tpr * s.teams;
    const size_t tops = MODE == kQuantGroups ? (size_t(s.teams) * 3 * groups * 4 + 15) / 16 * 16 : 0;
    const size_t smem = tops + (PIECE >= 4 ? size_t(16) * VPT * (RES ? 2 : 1) * D * block : 0);
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem, cfg);
    if (e != cudaSuccess) return e;
    const int grid = grid_for(reinterpret_cast<const void*>(k), block, smem, (a.M + s.teams - 1) / s.teams, cfg);
    const bool aligned = reinterpret_cast<uintptr_t>(a.q) % V == 0 && a.ldq % V == 0;
    k<<<grid, block, smem, cfg.stream>>>(a, s.tpr, lanes_log2, groups, aligned);
    return cudaGetLastError();
}

template <typename T, int PIECE, bool RES, int VPT, int D>
cudaError_t launch_quant_mode(const QuantArgs& a, const QuantShape& s, const LaunchCfg& cfg) {
    const int groups = int((a.N + a.group - 1) / a.group);
    if (groups == 1) return launch_quant<T, PIECE, RES, VPT, D, kQuantRow>(a, s, 0, 1, cfg);
    for (int log2 = 2; log2 <= 5; ++log2)
        if (a.group == int64_t(Elem<T>::kVec) << log2)
            return launch_quant<T, PIECE, RES, VPT, D, kQuantLanes>(a, s, log2, groups, cfg);
    return launch_quant<T, PIECE, RES, VPT, D, kQuantGroups>(a, s, 0, groups, cfg);
}

template <typename T, int PIECE>
cudaError_t launch_quant_vectors(const QuantArgs& a, const QuantShape& s, const LaunchCfg& cfg) {
    if (a.residual) {
        if (s.vpt == 1) return launch_quant_mode<T, PIECE, true, 1, 1>(a, s, cfg);
        if (s.vpt == 2) return launch_quant_mode<T, PIECE, true, 2, 1>(a, s, cfg);
        if (s.vpt == 8) return launch_quant_mode<T, PIECE, true, 8, 1>(a, s, cfg);
        if (PIECE == 16 && s.tpr > 256) return launch_quant_mode<T, PIECE, true, 4, PIECE == 16 ? 2 : 1>(a, s, cfg);
        return launch_quant_mode<T, PIECE, true, 4, 1>(a, s, cfg);
    }
    constexpr int D = PIECE >= 4 ? 2 : 1;
    return s.vpt == 1   ? launch_quant_mode<T, PIECE, false, 1, D>(a, s, cfg)
           : s.vpt == 2 ? launch_quant_mode<T, PIECE, false, 2, D>(a, s, cfg)
           : s.vpt == 4 ? launch_quant_mode<T, PIECE, false, 4, D>(a, s, cfg)
                        : launch_quant_mode<T, PIECE, false, 8, D>(a, s, cfg);
}

// piece: bytes of the widest access that every row allows; 0: the looped kernel
template <typename T>
cudaError_t launch_rms_quant(const QuantArgs& a, int piece, const LaunchCfg& cfg) {
    QuantShape s;
    if (piece && a.N <= int64_t(kQuantThreads) * 8 * Elem<T>::kVec &&
        quant_shape((a.N + Elem<T>::kVec - 1) / Elem<T>::kVec, a.M, piece, cfg, &s)) {
        if (piece == 16) return launch_quant_vectors<T, 16>(a, s, cfg);
        if (piece == 4) return launch_quant_vectors<T, 4>(a, s, cfg);
        if constexpr (sizeof(T) == 2) return launch_quant_vectors<T, 2>(a, s, cfg);
    }
    const bool res = a.residual != nullptr;
    auto k = res ? rms_quant_looped_kernel<T, true> : rms_quant_looped_kernel<T, false>;
    const int grid = grid_for(reinterpret_cast<const void*>(k), kLoopBlock, 0, a.M, cfg);
    k<<<grid, kLoopBlock, 0, cfg.stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rowops
