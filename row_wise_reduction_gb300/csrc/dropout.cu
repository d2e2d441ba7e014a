// Bias + dropout + residual, and its backward with the bias's gradient:
//   y = r + keep (x + b) / (1 - p);    dx = keep dy / (1 - p), db = column sums of dx
// (the backward is the same kernel on dy without bias and residual). Whether
// an element is kept follows from 16 random bits of Philox4x32-10: element (row,
// col) takes half-word col mod 8 of the block with counter (col / 8, row,
// offset) and key seed, and is kept where they reach round(65536 p). The mask is
// a function of position alone: never stored, and the same for every layout,
// launch shape and type. Sixteen bits an element instead of 32 halve the
// generator's share of the instructions: ten rounds of four for eight elements.
//
// A team of TL lanes holds 8 TL consecutive columns of a row; lane l makes the
// block of columns 8 l .. 8 l + 7. Each lane moves the columns that coalesce best
// for the type and alignment (bf16: its own eight as one 16-byte vector; fp32: two
// 16-byte vectors; short rows at odd offsets: eight single elements, TL apart) and
// gets the decisions for those columns, a byte a block, from the lanes that made
// them. The lanes keep their columns over all rows of a chunk, so the bias is
// loaded once and column sums stay in registers until the chunk's end; they leave
// one partial row per chunk, added up by a second kernel in a fixed order.
//
// Bound by traffic, with the instructions not far behind (for a 16-byte vector of bf16
// 112 backward, 138 with bias and residual; the generator's 40 among them): rows come in through a ring of
// copies into shared memory, a slot for each thread alone, so that the rows in
// flight take no registers. With four rows in flight in registers the kernel held
// half as many warps and bf16 16384 x 8192 with column sums took 124.8 us. Now 88 us
// (6.1 TB/s); forward, with bias and residual, 120 us (6.7 TB/s). bf16 4001 x 4097 with
// column sums, rows at odd offsets: 23 us for a floor of 9.6 (p = 0 without column
// sums 13 us), bound by neither memory (15%) nor issue (45%): 17 x 63 CTAs leave a warp
// eight rows, of which the ring's start is five, and the shifted form takes 29
// instructions an element where the vector form takes 14.
#include <algorithm>

#include "async_ring.cuh"
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
    PhiloxKeys keys;       // of the seed
    uint64_t offset;
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

// What the lanes of a warp hold: pieces of PE elements, NP of them.
template <int PE>
struct Columns {
    static constexpr int NP = 8 / PE;
    int lane, warp, tl, sub, TL, SR, RY;  // SR, RY: rows of a warp and of the CTA at a time
    int64_t c0, r0, r1, col[NP];
    bool in[NP];
    __device__ __forceinline__ explicit Columns(const DropArgs& a) {
        lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        TL = 1 << a.tl_log2, tl = lane & (TL - 1), sub = lane >> a.tl_log2;
        const int WX = 1 << a.wx_log2, wx = warp & (WX - 1);
        SR = 32 >> a.tl_log2, RY = (kWarps >> a.wx_log2) * SR;
        c0 = (int64_t(blockIdx.x) * WX + wx) * 8 * TL;
        r0 = int64_t(blockIdx.y) * a.chunk_rows;
        r1 = r0 + a.chunk_rows < a.M ? r0 + a.chunk_rows : a.M;
        r0 += (warp >> a.wx_log2) * SR;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            col[j] = c0 + PE * (TL * j + tl);
            in[j] = col[j] < a.N;
        }
    }
    // the decisions for the elements of piece j, from the lane that made their block
    __device__ __forceinline__ uint32_t keep(uint32_t own, int j) const {
        if constexpr (PE == 8) return own;
        const int at = PE * (TL * j + tl);  // column within the team's
        return __shfl_sync(0xffffffffu, own, (lane & ~(TL - 1)) + (at >> 3)) >> (at & 7);
    }
    // the CTA's column sums: over the warp's teams, then over the warps of the same columns
    __device__ __forceinline__ void leave(float (&acc)[NP][PE], float* part, const DropArgs& a) const {
        __shared__ float red[kWarps][256];
        const int WX = 1 << a.wx_log2;
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int e = 0; e < PE; ++e) {
                for (int o = TL; o < 32; o <<= 1) acc[j][e] += __shfl_xor_sync(0xffffffffu, acc[j][e], o);
                if (sub == 0) red[warp][PE * (TL * j + tl) + e] = acc[j][e];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < WX * 8 * TL; i += kWarps * 32) {
            const int w = i >> (3 + a.tl_log2), c = i & (8 * TL - 1);
            float s = 0.f;
            for (int k = w; k < kWarps; k += WX) s += red[k][c];
            const int64_t at = int64_t(blockIdx.x) * WX * 8 * TL + i;
            if (at < a.N) part[int64_t(blockIdx.y) * a.N + at] = s;
        }
    }
};

struct Generator {
    const PhiloxKeys& keys;
    uint32_t lo, hi;  // the offset
    __device__ __forceinline__ Generator(const DropArgs& a, bool rng) : keys(a.keys) {
        uint64_t off = a.offset;
        if (rng && a.device_offset) off += *a.device_offset;
        lo = uint32_t(off);
        hi = uint32_t(off >> 32);
    }
    __device__ __forceinline__ uint4 words(uint32_t block, uint32_t row) const {
        return philox4x32_10(make_uint4(block, row, lo, hi), keys);
    }
};

// 16-byte vectors (16-byte aligned rows, N a multiple of the vector). RNG: p > 0.
// SUM: column sums of the results into `part`. RES: a residual.
template <typename T, bool RNG, bool SUM, bool RES>
__global__ void __launch_bounds__(kWarps * 32, Elem<T>::kBytes == 2 ? 4 : 3)
    dropout_kernel(const T* x, const T* r, const T* b, T* y, float* part,
                   const __grid_constant__ DropArgs a) {
    using E = Elem<T>;
    constexpr int PE = E::kVec, NP = 8 / PE, N = NP * (RES ? 2 : 1), D = N == 1 ? 6 : (N == 2 ? 4 : 3);
    extern __shared__ uint4 slots[];
    if constexpr (SUM) let_next_start();
    const Columns<PE> c(a);
    const Generator gen(a, RNG);
    Ring<D, N, kWarps * 32> ring(slots);
    float2 bias[SUM ? 1 : NP][PE / 2];  // the backward pass has none
    if constexpr (!SUM) {
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int e = 0; e < PE / 2; ++e)
                bias[j][e] = b && c.in[j]
                                 ? make_float2(E::load(b + c.col[j] + 2 * e), E::load(b + c.col[j] + 2 * e + 1))
                                 : f2(0.f);
    }
    float2 acc[NP][PE / 2] = {};
    // the lane's first piece of the row to ask for and of the row to write
    const int64_t at = (c.r0 + c.sub) * a.ld + c.col[0], step = c.RY * a.ld;
    const T *px = x + at, *pr = RES ? r + at : nullptr;
    T* py = y + at;
    int64_t ahead = c.r0 + c.sub;
    auto ask = [&] {
#pragma unroll
        for (int j = 0; j < NP; ++j)
            if (ahead < c.r1 && c.in[j]) {
                ring.ask(j, px + j * PE * c.TL);
                if constexpr (RES) ring.ask(NP + j, pr + j * PE * c.TL);
            }
        ring.asked();
        ahead += c.RY;
        px += step;
        if constexpr (RES) pr += step;
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) ask();
#pragma unroll 1
    for (int64_t rb = c.r0; rb < c.r1; rb += c.RY, py += step) {
        ask();
        const int64_t row = rb + c.sub;
        uint32_t own = 0xffu;
        uint4 w = make_uint4(0, 0, 0, 0);
        if constexpr (RNG) {
            w = gen.words(uint32_t(c.c0 >> 3) + c.tl, uint32_t(row));
            if constexpr (PE < 8) own = keep_bits(w, a.lim);
        }
        ring.wait();
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            uint32_t keep = own;
            if constexpr (RNG) keep = c.keep(own, j);
            if (row < c.r1 && c.in[j]) {
                float v[PE];
                E::unpack(ring.get(j), v);
#pragma unroll
                for (int e = 0; e < PE; e += 2) {
                    float2 t = make_float2(v[e], v[e + 1]);
                    if constexpr (!SUM) t = f2_add(t, bias[j][e / 2]);
                    t = f2_mul(t, f2(a.scale));
                    if constexpr (RNG) {
                        bool k0 = keep >> e & 1u, k1 = keep >> (e + 1) & 1u;
                        if constexpr (PE == 8) {  // the block's own words
                            k0 = words[e / 2] << 16 > a.lim;
                            k1 = words[e / 2] > a.lim;
                        }
                        t = make_float2(k0 ? t.x : 0.f, k1 ? t.y : 0.f);
                    }
                    if constexpr (SUM) acc[j][e / 2] = f2_add(acc[j][e / 2], t);
                    v[e] = t.x;
                    v[e + 1] = t.y;
                }
                if constexpr (RES) {
                    float q[PE];
                    E::unpack(ring.get(NP + j), q);
#pragma unroll
                    for (int e = 0; e < PE; e += 2) {
                        const float2 t = f2_add(make_float2(v[e], v[e + 1]), make_float2(q[e], q[e + 1]));
                        v[e] = t.x;
                        v[e + 1] = t.y;
                    }
                }
                st_stream16(py + j * PE * c.TL, E::pack(v));
            }
        }
        ring.done();
    }
    if constexpr (SUM) {
        float sums[NP][PE];
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int e = 0; e < PE; ++e) sums[j][e] = e & 1 ? acc[j][e / 2].y : acc[j][e / 2].x;
        c.leave(sums, part, a);
    }
}

// Single elements: any layout.
template <typename T, bool RNG, bool SUM, int U>
__global__ void __launch_bounds__(kWarps * 32)
    dropout_elements_kernel(const T* x, const T* r, const T* b, T* y, float* part,
                   const __grid_constant__ DropArgs a) {
    using E = Elem<T>;
    if constexpr (SUM) let_next_start();
    const Columns<1> c(a);
    const Generator gen(a, RNG);
    float bias[8], acc[8][1] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) bias[j] = b && c.in[j] ? E::load(b + c.col[j]) : 0.f;
    for (int64_t rb = c.r0; rb < c.r1; rb += int64_t(c.RY) * U) {
        float xs[U][8], rs[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = rb + c.sub + int64_t(u) * c.RY;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (row < c.r1 && c.in[j]) {
                    xs[u][j] = E::load(x + row * a.ld + c.col[j]);
                    if (r) rs[u][j] = E::load(r + row * a.ld + c.col[j]);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = rb + c.sub + int64_t(u) * c.RY;
            uint32_t own = 0xffu;
            if constexpr (RNG) own = keep_bits(gen.words(uint32_t(c.c0 >> 3) + c.tl, uint32_t(row)), a.lim);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t keep = own;
                if constexpr (RNG) keep = c.keep(own, j);
                if (row < c.r1 && c.in[j]) {
                    float v = keep & 1u ? (xs[u][j] + bias[j]) * a.scale : 0.f;
                    if constexpr (SUM) acc[j][0] += v;
                    if (r) v += rs[u][j];
                    E::store(y + row * a.ld + c.col[j], v);
                }
            }
        }
    }
    if constexpr (SUM) c.leave(acc, part, a);
}

// Rows that start at changing offsets from a 16-byte boundary (the same for every
// tensor): each warp takes rows 8 apart, which all start at one offset, so its lanes
// keep their columns. Lane l holds the aligned 16-byte vector v = 31 segment + l,
// columns head + V v .. of its rows, and makes the block of random bits that they
// begin in; where they run into the next block its bits come from lane l + 1, whose
// block that is (lane 31 has only that to do). What is left behind the last whole
// vector comes as a part of one; the elements before the first go one by one, a row
// ahead. Two rows of column sums for each
// chunk, one from even segments and one from odd: with their columns shifted from
// warp to warp, neighbours overlap.
constexpr int kSegVecs = 31;

template <typename T, bool RNG, bool SUM, bool RES>
__global__ void __launch_bounds__(kWarps * 32, 4)
    dropout_shifted_kernel(const T* x, const T* r, const T* b, T* y, float* part,
                   const __grid_constant__ DropArgs a) {
    using E = Elem<T>;
    constexpr int V = E::kVec, SPAN = kSegVecs * V;  // columns from one segment to the next
    constexpr int N = RES ? 2 : 1, D = RES ? 4 : 6;
    extern __shared__ uint4 slots[];
    if constexpr (SUM) let_next_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = int64_t(blockIdx.y) * a.chunk_rows + warp;
    const int64_t r1 = int64_t(blockIdx.y + 1) * a.chunk_rows < a.M ? int64_t(blockIdx.y + 1) * a.chunk_rows : a.M;
    const Generator gen(a, RNG);
    Ring<D, N, kWarps * 32> ring(slots);

    const RowGeom geo = row_geometry<T>(x + (r0 < a.M ? r0 : 0) * a.ld, a.N);
    const int64_t v = int64_t(blockIdx.x) * kSegVecs + lane, col = geo.head + V * v;
    const uint32_t block = uint32_t(col >> 3);
    const int at = int(col & 7);
    const bool whole = lane < kSegVecs && v < geo.nvec;
    const int tail = lane < kSegVecs && v == geo.nvec ? geo.tail : 0;
    const bool held = whole || tail;
    const unsigned bytes = whole ? 16u : unsigned(tail * E::kBytes);
    const bool head = blockIdx.x == 0 && lane < geo.head;  // the first segment's lanes, one element each
    float bias[V], head_bias = 0.f, head_acc = 0.f;
    float2 acc[V / 2] = {};
#pragma unroll
    for (int e = 0; e < V; ++e) bias[e] = b && (whole || e < tail) ? E::load(b + col + e) : 0.f;
    if (b && head) head_bias = E::load(b + lane);

    const int64_t at0 = r0 * a.ld + col, step = kWarps * a.ld;
    const T *px = x + at0, *pr = RES ? r + at0 : nullptr;
    T* py = y + at0;
    int64_t ahead = r0;
    auto ask = [&] {
        if (ahead < r1 && held) {
            ring.ask_part(0, px, bytes);
            if constexpr (RES) ring.ask_part(1, pr, bytes);
        }
        ring.asked();
        ahead += kWarps;
        px += step;
        if constexpr (RES) pr += step;
    };
    float head_x = 0.f, head_r = 0.f;
    auto ask_head = [&](int64_t row) {
        if (head && row < r1) {
            head_x = E::load(x + row * a.ld + lane);
            if constexpr (RES) head_r = E::load(r + row * a.ld + lane);
        }
    };
    const bool any_head = blockIdx.x == 0 && geo.head > 0;  // the warp's
#pragma unroll
    for (int d = 0; d < D - 1; ++d) ask();
    ask_head(r0);
#pragma unroll 1
    for (int64_t row = r0; row < r1; row += kWarps, py += step) {
        ask();
        uint32_t own = 0xffu, keep = 0xffu;
        if constexpr (RNG) {
            own = keep_bits(gen.words(block, uint32_t(row)), a.lim);
            keep = (own | __shfl_down_sync(0xffffffffu, own, 1) << 8) >> at;
        }
        ring.wait();
        if (held) {
            float o[V];
            E::unpack(ring.get(0), o);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                float2 t = make_float2(o[e], o[e + 1]);
                if constexpr (!SUM) t = f2_add(t, make_float2(bias[e], bias[e + 1]));
                t = f2_mul(t, f2(a.scale));
                if constexpr (RNG) t = make_float2(keep >> e & 1u ? t.x : 0.f, keep >> (e + 1) & 1u ? t.y : 0.f);
                o[e] = t.x;
                o[e + 1] = t.y;
                if constexpr (SUM) acc[e / 2] = f2_add(acc[e / 2], t);
            }
            if constexpr (RES) {
                float q[V];
                E::unpack(ring.get(1), q);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] += q[e];
            }
            if (whole) {
                st_stream16(py, E::pack(o));
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e < tail) E::store(py + e, o[e]);
            }
        }
        if (any_head) {
            if constexpr (RNG) own = __shfl_sync(0xffffffffu, own, 0);  // the head's block
            if (head) {
                float h = own >> lane & 1u ? (head_x + head_bias) * a.scale : 0.f;
                if constexpr (SUM) head_acc += h;
                if constexpr (RES) h += head_r;
                E::store(y + row * a.ld + lane, h);
            }
            ask_head(row + kWarps);
        }
        ring.done();
    }

    if constexpr (SUM) {
        // each warp's, columns from SPAN segment on; then over the warps in order
        __shared__ float reds[kWarps][SPAN + V];
        float* red = reds[warp];
        for (int i = lane; i < SPAN + V; i += 32) red[i] = 0.f;
        __syncwarp();
        if (r0 < r1) {
            float* at0 = red + geo.head + V * lane;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (whole || e < tail) at0[e] = e & 1 ? acc[e / 2].y : acc[e / 2].x;
            if (head) red[lane] = head_acc;
        }
        __syncthreads();
        auto sum = [&](int i) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += reds[w][i];
            return s;
        };
        // the segment's part of its row, up to where the next one of that row begins
        float* out = part + (int64_t(blockIdx.y) * 2 + (blockIdx.x & 1)) * a.N;
        const int64_t c0 = int64_t(blockIdx.x) * SPAN;
        for (int i = threadIdx.x; i < 2 * SPAN; i += kWarps * 32)
            if (c0 + i < a.N) out[c0 + i] = i < SPAN + V ? sum(i) : 0.f;
        // odd segments' row has nothing before the first of them (one segment alone has
        // fewer than SPAN columns)
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < SPAN && i < a.N; i += kWarps * 32)
                part[(int64_t(blockIdx.y) * 2 + 1) * a.N + i] = 0.f;
    }
}

// the widest power of two that leaves at most 1/8 of its span idle; else the one
// that leaves the least
inline int pick_log2(int64_t n, int64_t unit, int top) {
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
}

template <typename T>
using DropKernel = void (*)(const T*, const T*, const T*, T*, float*, DropArgs);

struct DropCall {
    const void *x, *r, *b;
    void* y;
    float* part;
    int max_partials;
    float* db;
};

// Rows of a chunk: without column sums four waves of CTAs. With them every chunk
// leaves partial rows, and fewer are better: of the vector form two CTAs an SM, whose
// rings keep the memory busy (bf16 16384 x 8192 88 us, with four 99, in two waves of
// those 92; 4096 x 1024 8 us, 9.6 and 11); of the others, which have more to compute, as
// many as fit, and twice as many where a chunk still has 32 rows (bf16 4001 x 4097 23
// us, one wave 26, four 26; 1000 x 1025 8.2 us and 7.5). Whole steps of the CTA unless that leaves
// CTAs idle.
template <typename T>
cudaError_t launch(DropKernel<T> kern, size_t smem, int64_t gx, int64_t step, int64_t unit, int partials,
                   bool rings, const DropCall& c, DropArgs a, const LaunchCfg& cfg) {
    const void* f = reinterpret_cast<const void*>(kern);
    cudaError_t e = allow_smem(f, smem, cfg);
    if (e != cudaSuccess) return e;
    int64_t want = grid_for(f, kWarps * 32, smem, INT64_MAX, cfg);
    if (!c.db) want *= 4;
    else if (rings) want = std::min(want, int64_t(2) * cfg.num_sms);
    else if (a.M * gx / 32 >= 2 * want) want *= 2;
    int64_t chunks = std::max(int64_t(1), want / gx);
    if (c.db) chunks = std::min(chunks, int64_t(c.max_partials / partials));
    chunks = std::min(chunks, int64_t(65535));
    a.chunk_rows = (a.M + chunks - 1) / chunks;
    a.chunk_rows = (a.chunk_rows + unit - 1) / unit * unit;
    if (!c.db || a.M / step >= chunks) a.chunk_rows = (a.chunk_rows + step - 1) / step * step;
    const int64_t gy = (a.M + a.chunk_rows - 1) / a.chunk_rows;
    kern<<<dim3(unsigned(gx), unsigned(gy)), kWarps * 32, smem, cfg.stream>>>(
        static_cast<const T*>(c.x), static_cast<const T*>(c.r), static_cast<const T*>(c.b), static_cast<T*>(c.y),
        c.part, a);
    e = cudaGetLastError();
    return e == cudaSuccess && c.db ? reduce_partials(c.part, partials * gy, a.N, a.N, c.db, nullptr, cfg) : e;
}

template <typename T, bool RNG, bool SUM, bool RES>
cudaError_t dropout_form(const DropCall& c, DropArgs a, int form, const LaunchCfg& cfg) {
    constexpr int V = Elem<T>::kVec;
    if (form == 1)  // shifted: a tail lane behind the last whole vector of a row that starts on a boundary
        return launch<T>(dropout_shifted_kernel<T, RNG, SUM, RES>, size_t(RES ? 8 : 6) * kWarps * 512,
                         (a.N / V + 1 + kSegVecs - 1) / kSegVecs, kWarps * 4, kWarps, 2, false, c, a, cfg);
    a.tl_log2 = pick_log2(a.N, 8, 5);
    const int64_t segs = (a.N + (int64_t(8) << a.tl_log2) - 1) / (int64_t(8) << a.tl_log2);
    a.wx_log2 = pick_log2(segs, 1, 3);
    const int64_t gx = (segs + (1 << a.wx_log2) - 1) >> a.wx_log2;
    const int64_t rows = int64_t(kWarps >> a.wx_log2) * (32 >> a.tl_log2);  // of a CTA at a time
    if (form == 0) {
        constexpr int N = 8 / V * (RES ? 2 : 1), D = N == 1 ? 6 : (N == 2 ? 4 : 3);
        return launch<T>(dropout_kernel<T, RNG, SUM, RES>, size_t(N) * D * kWarps * 512, gx, rows * 4, 1, 1, true, c, a,
                         cfg);
    }
    return launch<T>(dropout_elements_kernel<T, RNG, SUM, 2>, 0, gx, rows * 2, 1, 1, false, c, a, cfg);
}

template <typename T>
cudaError_t dropout(const void* x, const void* r, const void* b, void* y, float* part, int max_partials, float* db,
                    int64_t M, int64_t N, int64_t ld, const DropoutMask& m, bool vec, bool elements,
                    const LaunchCfg& cfg) {
    const DropArgs a{M, N, ld, 0, 0, 0, (m.drop << 16) - 1u,
                     m.drop < 65536u ? 65536.f / float(65536u - m.drop) : 0.f, PhiloxKeys(m.seed), m.offset,
                     m.device_offset};
    const DropCall c{x, r, b, y, part, max_partials, db};
    // Rows at odd offsets, from 64 columns on (a segment has 31 vectors): the
    // lanes' aligned vectors move 31 lanes' 496 bytes in one access where single
    // elements take eight. The column sums need two partial rows a chunk.
    auto off = [](const void* p, const void* q) {
        return (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(q)) & 15u;
    };
    const bool shifted = !elements && off(x, y) == 0 && (!r || off(x, r) == 0) && N >= 64 && (!db || max_partials >= 2);
    const int form = vec ? 0 : (shifted ? 1 : 2);
    if (db)  // the backward pass: no residual
        return m.drop ? dropout_form<T, true, true, false>(c, a, form, cfg)
                      : dropout_form<T, false, true, false>(c, a, form, cfg);
    if (r)
        return m.drop ? dropout_form<T, true, false, true>(c, a, form, cfg)
                      : dropout_form<T, false, false, true>(c, a, form, cfg);
    return m.drop ? dropout_form<T, true, false, false>(c, a, form, cfg)
                  : dropout_form<T, false, false, false>(c, a, form, cfg);
}

}  // namespace

DropoutLaunch dropout_f32() { return dropout<float>; }
DropoutLaunch dropout_bf16() { return dropout<bf16_t>; }

}  // namespace rowops
