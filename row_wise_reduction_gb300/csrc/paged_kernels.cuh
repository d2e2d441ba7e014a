// Attention of one new token a sequence over a paged key-value cache:
//   s_j = scale q k_j;  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// over the positions j in [first, n) of a sequence; position j is slot j mod page of the
// page that the sequence's table names for j / page. One pass with a running maximum
// and sum, as the split-row online softmax has, and the weighted values beside them.
//
// Bound by the cache's traffic: every key and value attended to is read once for a block of
// the heads that share it, which are at most 16 in bf16 and 8 in fp32. Heads beyond read it again, a sequence's positions
// later in the line, so from memory if those are many: 16 sequences of up to 4096 in fp32, D 128, 64 heads over 8 94 us, 128
// over 8 175; 32 of up to 8192 in bf16, 128 over 8 163 us, 256 over 8 313. The work is a line of tiles: for every
// sequence, key head and block of its heads (a unit), the unit's positions in tiles. The persistent grid's
// CTAs take equal stretches of that line, whatever the lengths are: a unit that lies within a stretch is written
// out at once, of one that crosses a border each CTA leaves its part (maximum, sum, weighted
// values) in the workspace, and a second kernel joins them, in order. Which CTA has
// which tiles follows from the lengths alone, so equal calls give equal bits. (Every CTA reads all
// lengths, the second kernel's too, of which there is one a sequence at least: 1024 sequences of 16 positions take 30 us,
// 4096 108, 16384 570, 65536 4428, when each of 65536 CTAs reads 256 KB of lengths.)
//
// Measured, bf16, D 128: 64 sequences of up to 8192, 32 heads over 8, 179 us (160 at the rate of a copy), two of up to
// 131072, 64 heads over 8, 160 us (139).
//
// Few units of short sequences: a cluster of CTAs a unit instead, which join their parts through distributed
// shared memory, so that one launch does it (one sequence of 512: 7.7 us, as a line 10.1).
//
// Within a CTA a warp takes every fourth piece of a tile by itself: it copies the piece's keys
// and values into a ring of its own in shared memory, several pieces ahead and across
// units, so no barrier stands in the loop; the warps meet at a unit's end only.
#pragma once

#include <cooperative_groups.h>

#include "async_ring.cuh"
#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace rowops {

constexpr int kPagedBlock = 32 * kPagedWarps;

// A warp's ring: pieces of a few positions, their keys, then their values.
template <typename T, int DT, int ROWS>
struct PagedRing {
    static constexpr PagedShape kShape = paged_shape(sizeof(T), DT, ROWS);
    static constexpr int kPitch = kShape.pitch;
    static constexpr int kPart = kShape.tokens * kPitch;  // keys, or values
    static constexpr int kCtas = kShape.ctas, kStages = kShape.stages;
    static constexpr int kBytes = kShape.step * kStages;
    static_assert((kBytes + kShape.fixed) * kCtas <= kSmShared);
};

// The tiles of one unit of sequence b, which attends to the positions [first, n); they
// count from `base`.
template <int TILE>
__device__ __forceinline__ uint32_t paged_span(const PagedArgs& a, int b, uint32_t* n, uint32_t* first, uint32_t* base) {
    const int asked = a.lengths[b];
    const int64_t room = a.max_pages * a.page;
    *n = asked <= 0 ? 0u : asked < room ? uint32_t(asked) : uint32_t(room);
    *first = a.window > 0 && *n > a.window ? *n - uint32_t(a.window) : 0u;
    *base = *first & ~15u;
    return (*n - *base + TILE - 1) / TILE;
}
__device__ __forceinline__ bool paged_beyond(const PagedArgs& a, int b) { return a.lengths[b] > a.max_pages * a.page; }

// The tiles of single units over all sequences, and over those before b. `red`: two int64 a
// warp. Every thread of the CTA calls it.
template <int TILE, int THREADS>
__device__ __forceinline__ void paged_count(const PagedArgs& a, int b, int64_t* red, int64_t* total, int64_t* before) {
    int64_t all = 0, some = 0;
    uint32_t n, f, base;
    for (int i = threadIdx.x; i < a.B; i += THREADS) {
        const uint32_t t = paged_span<TILE>(a, i, &n, &f, &base);
        all += t;
        if (i < b) some += t;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        some += __shfl_xor_sync(0xffffffffu, some, o);
    }
    if ((threadIdx.x & 31) == 0) red[2 * (threadIdx.x >> 5)] = all, red[2 * (threadIdx.x >> 5) + 1] = some;
    __syncthreads();
    all = some = 0;
    for (int i = 0; i < THREADS / 32; ++i) all += red[2 * i], some += red[2 * i + 1];
    *total = all;
    *before = some;
}

// CTA c's stretch [begin, end) of the line's `total` tiles, the sequence that it begins in, and
// the tiles of single units of the sequences before that. `sum`: kPagedWarps int64. Every
// thread of the CTA calls it.
template <int TILE>
__device__ __forceinline__ void paged_find(const PagedArgs& a, int units, int64_t* sum, int64_t* total, int c, int ctas,
                                           int64_t* begin, int64_t* end, int* b, int64_t* before) {
    // thread i counts the sequences [i * each, (i + 1) * each)
    const int each = int((a.B + kPagedBlock - 1) / kPagedBlock), i0 = threadIdx.x * each;
    int64_t mine = 0;
    uint32_t n, f, base;
    for (int i = i0; i < i0 + each && i < a.B; ++i) mine += paged_span<TILE>(a, i, &n, &f, &base);
    int64_t run = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t other = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += other;
    }
    if (lane == 31) sum[warp] = run;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int i = 0; i < kPagedWarps; ++i) {
        if (i < warp) run += sum[i];
        all += sum[i];
    }
    __syncthreads();
    *total = all * units;
    if (ctas > *total) ctas = int(*total);  // every CTA that has a stretch has a tile
    *begin = c < ctas ? *total * c / ctas : 0;
    *end = c < ctas ? *total * (c + 1) / ctas : 0;
    const int64_t at = *begin / units;  // in tiles of single units
    if (at >= run - mine && at < run) {
        int64_t p = run - mine;
        int i = i0;
        for (;; ++i) {
            const int64_t t = paged_span<TILE>(a, i, &n, &f, &base);
            if (at < p + t) break;
            p += t;
        }
        sum[0] = i;
        sum[1] = p;
    }
    __syncthreads();
    *b = *begin < *end ? int(sum[0]) : 0;
    *before = sum[1];
    __syncthreads();
}

// A place in the line of tiles.
template <int TILE>
struct PagedCursor {
    const PagedArgs& a;
    int units, b, j;
    uint32_t n, first, base, tile, tiles;
    int64_t left;
    __device__ __forceinline__ PagedCursor(const PagedArgs& a_, int units_, int b_, int64_t in_sequence, int64_t left_)
        : a(a_), units(units_), b(b_), left(left_) {
        j = 0, tile = 0, tiles = 1, n = first = base = 0;
        if (left > 0) {
            tiles = paged_span<TILE>(a, b, &n, &first, &base);
            j = int(in_sequence / tiles);
            tile = uint32_t(in_sequence - int64_t(j) * tiles);
        }
    }
    __device__ __forceinline__ void next() {
        if (--left <= 0) return;
        if (++tile < tiles) return;
        tile = 0;
        if (++j < units) return;
        j = 0;
        do {
            tiles = paged_span<TILE>(a, ++b, &n, &first, &base);
        } while (tiles == 0);  // (the stretch has tiles left, so there is a sequence with some)
    }
};

// What a unit's part is in the workspace: rows of DT weighted values, then a maximum and a sum each
// (rounded up to whole vectors).
template <int DT, int ROWS>
__device__ __forceinline__ constexpr int paged_part_floats() {
    return (ROWS * (DT + 2) + 3) / 4 * 4;
}

// What a head's row of sums becomes: the maximum m in the exponent of 2, the sum l.
struct PagedRow {
    float inv, lse;
    __device__ __forceinline__ PagedRow(float m, float l, bool beyond) {
        if (beyond) l = NAN;
        inv = l == 0.f ? 0.f : 1.f / l;
        lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
    }
};

// CLUSTERED: a cluster of CTAs a unit, its tiles shared out evenly; else equal stretches of the line.
template <class P, bool CLUSTERED>
__global__ void __launch_bounds__(kPagedBlock, P::Ring::kCtas)
    paged_attention_kernel(const __grid_constant__ PagedArgs a, float* parts, int blocks, bool whole) {
    using T = typename P::T;
    using E = Elem<T>;
    using Ring = typename P::Ring;
    constexpr int TK = P::kTokens, TILE = TK * kPagedWarps, S = Ring::kStages, DT = P::kD, ROWS = P::kRows;
    extern __shared__ uint4 smem[];
    char* ring = reinterpret_cast<char*>(smem) + (threadIdx.x >> 5) * (2 * Ring::kPart) * S;
    float* joined = reinterpret_cast<float*>(reinterpret_cast<char*>(smem) + Ring::kBytes);  // [ROWS][P::kPitch]
    float* scratch = joined + ROWS * P::kPitch;                                                     // P's own
    __shared__ float tops[kPagedWarps][ROWS], sums[kPagedWarps][ROWS];
    __shared__ int64_t found[kPagedBlock / 32 * 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = int(a.kv_heads) * blocks;
    const int group = int(a.heads / a.kv_heads);
    __shared__ float told_top[ROWS], told_sum[ROWS];  // CLUSTERED: read by the cluster's CTAs
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = CLUSTERED ? int(cluster.num_blocks()) : 1, rank = CLUSTERED ? int(cluster.block_rank()) : 0;

    P p(scratch);
    int64_t begin, end, before = 0;
    int b;
    if constexpr (CLUSTERED) {
        const int unit = int(blockIdx.x) / C, j = unit % units, head = j / blocks * group + j % blocks * ROWS;
        uint32_t n, first, base;
        b = unit / units;
        // the queries first: they wait for nothing
        p.begin(static_cast<const T*>(a.q) + b * a.ldq + int64_t(head) * a.D, min(ROWS, group - j % blocks * ROWS), int(a.D));
        const int64_t tiles = paged_span<TILE>(a, b, &n, &first, &base);
        begin = j * tiles + tiles * rank / C;
        end = j * tiles + tiles * (rank + 1) / C;
        if (threadIdx.x < ROWS) told_top[threadIdx.x] = -INFINITY, told_sum[threadIdx.x] = 0.f;
    } else {
        int64_t total;
        let_next_start();
        paged_find<TILE>(a, units, found, &total, blockIdx.x, gridDim.x, &begin, &end, &b, &before);
        if (begin >= end) return;
    }

    // columns past D stay zero: nothing is copied there
    if (a.D < DT)
        for (int i = lane; i < S * 2 * Ring::kPart / 16; i += 32)
            if (i % (Ring::kPitch / 16) >= a.D / E::kVec) reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();

    PagedCursor<TILE> in(a, units, b, begin - before * units, end - begin), at = in;
    uint32_t bad = 0;  // ring slots with a position whose page is none
    // Where pages are whole pieces, a piece lies within a page: one entry, and rows a stride apart.
    const uint32_t slots = uint32_t(a.page);
    const bool paged = whole && slots % TK == 0;
    int page = 0;
    auto look = [&] {  // the page of the piece to come, or of this lane's position of it
        const uint32_t t = in.base + in.tile * TILE + warp * TK + (paged ? 0 : lane);
        if (in.left > 0 && (paged ? t + TK > in.first : lane < TK && t >= in.first) && t < in.n)
            page = a.table[int64_t(in.b) * a.table_ld + t / slots];
    };
    constexpr int kRow = DT * int(sizeof(T)) / 16, kLanes = kRow > 16 ? 32 : kRow > 8 ? 16 : 8, kRows = 32 / kLanes;
    const int r0 = lane / kLanes, v0 = lane % kLanes, vectors = int(a.D) / E::kVec;
    auto ask = [&](int slot) {
        if (in.left > 0) {
            const uint32_t t0 = in.base + in.tile * TILE + warp * TK, t = t0 + lane;
            char* to = ring + slot * 2 * Ring::kPart;
            const int64_t head = int64_t(in.j / blocks) * a.head_stride;
            if (paged) {
                const int lo = int(in.first) - int(t0), hi = int(in.n) - int(t0);
                const bool there = page >= 0 && page < a.pages;
                const bool live = hi > 0 && lo < TK;
                bad = live && !there ? bad | 1u << slot : bad & ~(1u << slot);
                const int64_t from = (there && live ? page * a.page_stride + (t0 % slots) * a.slot_stride + head +
                                                          r0 * a.slot_stride
                                                    : 0) + v0 * E::kVec;
                const T* k = static_cast<const T*>(a.k) + from;
                const T* v = static_cast<const T*>(a.v) + from;
                const int64_t step = there && live ? kRows * a.slot_stride : 0;
                char* at = to + r0 * Ring::kPitch + v0 * 16;
#pragma unroll
                for (int r = 0; r < TK; r += kRows) {
                    const unsigned bytes = there && r + r0 >= lo && r + r0 < hi ? 16u : 0u;
#pragma unroll
                    for (int i = 0; i < kRow; i += kLanes)
                        if (v0 + i < vectors) {
                            copy_async_part(at + i * 16, k + i * E::kVec, bytes);
                            copy_async_part(at + i * 16 + Ring::kPart, v + i * E::kVec, bytes);
                        }
                    at += kRows * Ring::kPitch;
                    k += step;
                    v += step;
                }
            } else {
                const bool live = lane < TK && t >= in.first && t < in.n, there = live && page >= 0 && page < a.pages;
                const int64_t off = there ? page * a.page_stride + int64_t(t % slots) * a.slot_stride + head : -1;
                bad = __any_sync(0xffffffffu, live && !there) ? bad | 1u << slot : bad & ~(1u << slot);
                if (whole) {
#pragma unroll
                    for (int r = 0; r < TK; r += kRows) {
                        const int64_t o = __shfl_sync(0xffffffffu, off, r + r0);
#pragma unroll
                        for (int i = 0; i < kRow; i += kLanes)
                            if (v0 + i < vectors) {
                                char* k = to + (r + r0) * Ring::kPitch + (v0 + i) * 16;
                                const int64_t from = (o < 0 ? 0 : o) + (v0 + i) * E::kVec;
                                copy_async_part(k, static_cast<const T*>(a.k) + from, o < 0 ? 0u : 16u);
                                copy_async_part(k + Ring::kPart, static_cast<const T*>(a.v) + from, o < 0 ? 0u : 16u);
                            }
                    }
                } else {
                    for (int r = 0; r < TK; ++r) {
                        const int64_t o = __shfl_sync(0xffffffffu, off, r);
                        T* k = reinterpret_cast<T*>(to + r * Ring::kPitch);
                        T* v = reinterpret_cast<T*>(to + r * Ring::kPitch + Ring::kPart);
                        for (int d = lane; d < a.D; d += 32) {
                            k[d] = o < 0 ? T{} : static_cast<const T*>(a.k)[o + d];
                            v[d] = o < 0 ? T{} : static_cast<const T*>(a.v)[o + d];
                        }
                    }
                }
            }
            in.next();
            look();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look();
    for (int s = 0; s < S; ++s) ask(s);

    const float scale = a.scale * kLog2eF;
    bool fresh = !CLUSTERED, cut = at.tile != 0;  // a unit begins; it began in another CTA
    for (int slot = 0; at.left > 0; slot = slot + 1 == S ? 0 : slot + 1) {
        const int head = at.j / blocks * group + at.j % blocks * ROWS;  // the unit's first
        const int rows = min(ROWS, group - at.j % blocks * ROWS);
        if (fresh) p.begin(static_cast<const T*>(a.q) + at.b * a.ldq + int64_t(head) * a.D, rows, int(a.D));
        fresh = false;
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        __syncwarp();
        const uint32_t t0 = at.base + at.tile * TILE + warp * TK;
        const char* k = ring + slot * 2 * Ring::kPart;
        p.step(k, k + Ring::kPart, int(at.first) - int(t0), int(at.n) - int(t0), scale);
        if (bad >> slot & 1) p.spoil();
        __syncwarp();
        ask(slot);
        const bool done = at.tile + 1 == at.tiles;
        if (done || at.left == 1) {
            // the unit's end, or the stretch's: the warps' sums become one
            p.tell(tops[warp], sums[warp]);
            __syncthreads();
            float top[P::kOwn], factor[P::kOwn];
#pragma unroll
            for (int i = 0; i < P::kOwn; ++i) {
                const int r = p.row(i);
                top[i] = tops[0][r];
                for (int w = 1; w < kPagedWarps; ++w) top[i] = fmaxf(top[i], tops[w][r]);
                factor[i] = top[i] == -INFINITY ? 0.f : ex2_approx(tops[warp][r] - top[i]);
            }
            for (int w = 0; w < kPagedWarps; ++w) {
                if (warp == w) p.add(joined, factor, w == 0);
                __syncthreads();
            }
            const bool part = cut || !done;
            // a CTA leaves two at most: of the unit that it begins in the middle of, and of that which it ends in
            float* out = parts + (int64_t(blockIdx.x) * 2 + !cut) * paged_part_floats<DT, ROWS>();
            for (int r = warp; r < rows; r += kPagedWarps) {
                float m = tops[0][r], l = 0.f;
                for (int w = 1; w < kPagedWarps; ++w) m = fmaxf(m, tops[w][r]);
                for (int w = 0; w < kPagedWarps; ++w)
                    l += m == -INFINITY ? sums[w][r] : sums[w][r] * ex2_approx(tops[w][r] - m);
                if constexpr (CLUSTERED) {
                    if (lane == 0) told_top[r] = m, told_sum[r] = l;
                } else if (part) {
                    for (int d = lane; d < DT; d += 32) out[r * DT + d] = joined[r * P::kPitch + d];
                    if (lane == 0) out[ROWS * DT + 2 * r] = m, out[ROWS * DT + 2 * r + 1] = l;
                } else {
                    const PagedRow row(m, l, paged_beyond(a, at.b));
                    T* o = static_cast<T*>(a.out) + at.b * a.ldo + int64_t(head + r) * a.D;
                    for (int d = lane; d < a.D; d += 32) E::store(o + d, joined[r * P::kPitch + d] * row.inv);
                    if (lane == 0 && a.lse) a.lse[at.b * a.heads + head + r] = row.lse;
                }
            }
            cut = false;
            fresh = true;
            __syncthreads();
        }
        at.next();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (CLUSTERED) {
        // every C-th row of the unit, joined from the CTAs' parts in order (one without a tile has a sum of 0)
        const int j = int(blockIdx.x) / C % units, head = j / blocks * group + j % blocks * ROWS;
        const int rows = min(ROWS, group - j % blocks * ROWS);
        cluster.sync();
        for (int r = rank; r < rows; r += C) {
            const int of = lane & (C - 1);
            const float pm = cluster.map_shared_rank(told_top, of)[r], pl = cluster.map_shared_rank(told_sum, of)[r];
            float m = pm;
#pragma unroll
            for (int o = kPagedCluster / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float take = m == -INFINITY ? 0.f : ex2_approx(pm - m);
            float l = 0.f;
            for (int c = 0; c < C; ++c) l += __shfl_sync(0xffffffffu, m == -INFINITY ? pl : pl * take, c);
            const PagedRow row(m, l, paged_beyond(a, b));
            T* o = static_cast<T*>(a.out) + b * a.ldo + int64_t(head + r) * a.D;
            for (int d0 = 0; d0 < a.D; d0 += kPagedBlock) {
                const int d = d0 + threadIdx.x;
                float x = 0.f;
#pragma unroll
                for (int c = 0; c < kPagedCluster; ++c)
                    if (c < C) {
                        const float w = __shfl_sync(0xffffffffu, take, c), s = __shfl_sync(0xffffffffu, pl, c);
                        if (s != 0.f && d < a.D) x = fmaf(cluster.map_shared_rank(joined, c)[r * P::kPitch + d], w, x);
                    }
                if (d < a.D) E::store(o + d, x * row.inv);
            }
            if (threadIdx.x == 0 && a.lse) a.lse[b * a.heads + head + r] = row.lse;
        }
        cluster.sync();  // no CTA's shared memory goes while it is read
    }
}

// The units that no CTA has written: those cut by a border, joined from their parts in
// order, and those without a position. CTA (x, y): sequence x, every gridDim.y-th unit. A row's parts are
// shared out among as many warps as there are for it; every warp of the row has the parts' maxima and sums, a lane each,
// and adds up the values of its own, several loads at a time. Bound by the latency of those loads, one after
// another: one sequence of 32768 positions, 57 parts a unit, bf16 35.4 us and fp32 57.9 for the whole call, with
// one warp a row 42.8 and 68.3. CTAs of 32 warps where they all fit on the GPU at once, of eight otherwise.
template <class P, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 32 / WARPS) paged_join_kernel(const __grid_constant__ PagedArgs a, const float* parts,
                                                                int blocks, int ctas) {
    using T = typename P::T;
    using E = Elem<T>;
    constexpr int TILE = P::kTokens * kPagedWarps, DT = P::kD, ROWS = P::kRows, VECTORS = DT / 4,
                  EACH = (VECTORS + 31) / 32, FLOATS = paged_part_floats<DT, ROWS>(), U = 4 / EACH;
    __shared__ int64_t red[WARPS * 2];
    __shared__ float4 sums[WARPS][VECTORS];
    const int b = blockIdx.x, units = int(a.kv_heads) * blocks, group = int(a.heads / a.kv_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t total, before;
    paged_count<TILE, 32 * WARPS>(a, b, red, &total, &before);
    total *= units;
    if (ctas > total) ctas = int(total);
    uint32_t n, first, base;
    const int64_t tiles = paged_span<TILE>(a, b, &n, &first, &base);
    const bool beyond = paged_beyond(a, b);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int j = blockIdx.y; j < units; j += gridDim.y) {
        // tile t is CTA c's where total c / ctas <= t < total (c + 1) / ctas, rounded down
        const int64_t t0 = before * units + j * tiles, t1 = t0 + tiles - 1;
        const int c0 = tiles ? int(((t0 + 1) * ctas - 1) / total) : 0, c1 = tiles ? int(((t1 + 1) * ctas - 1) / total) : -1;
        if (tiles && c0 == c1) continue;
        const int head = j / blocks * group + j % blocks * ROWS, rows = min(ROWS, group - j % blocks * ROWS);
        // the CTA that the unit begins in left its part behind that of the unit it began with itself
        const int count = c1 - c0 + 1;
        auto part = [&](int i) { return parts + (int64_t(c0 + i) * 2 + (i == 0)) * FLOATS; };
        int each = WARPS;  // warps a row
        while (each > 1 && (rows * each > WARPS || each > count)) each >>= 1;
        const int sub = warp % each;
        for (int r0 = 0; r0 < rows; r0 += WARPS / each) {
            const int r = r0 + warp / each;
            float4 acc[EACH] = {};
            float m = -INFINITY, l = 0.f;
            if (r < rows) {
                float pm = -INFINITY, pl = 0.f;
                auto told = [&](int i) {
                    const float2 two = *reinterpret_cast<const float2*>(part(i) + ROWS * DT + 2 * r);
                    pm = two.x, pl = two.y;
                };
                for (int i = lane; i < count; i += 32) {
                    told(i);
                    m = fmaxf(m, pm);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                for (int c = 0; c < count; c += 32) {
                    const int here = min(32, count - c), end = here * (sub + 1) / each;
                    float take = 0.f;
                    if (lane < here) {
                        if (count > 32) told(c + lane);
                        take = m == -INFINITY ? 0.f : ex2_approx(pm - m);
                        l += m == -INFINITY ? pl : pl * take;
                    }
                    for (int i = here * sub / each; i < end; i += U) {
                        float4 v[U][EACH];
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int e = 0; e < EACH; ++e)
                                v[u][e] = i + u < end && lane + 32 * e < VECTORS
                                              ? reinterpret_cast<const float4*>(part(c + i + u) + r * DT)[lane + 32 * e]
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const float w = __shfl_sync(0xffffffffu, take, (i + u) & 31);
#pragma unroll
                            for (int e = 0; e < EACH; ++e) {
                                acc[e].x = fmaf(v[u][e].x, w, acc[e].x), acc[e].y = fmaf(v[u][e].y, w, acc[e].y);
                                acc[e].z = fmaf(v[u][e].z, w, acc[e].z), acc[e].w = fmaf(v[u][e].w, w, acc[e].w);
                            }
                        }
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            }
            if (each > 1) {
                if (sub > 0)
#pragma unroll
                    for (int e = 0; e < EACH; ++e)
                        if (lane + 32 * e < VECTORS) sums[warp][lane + 32 * e] = acc[e];
                __syncthreads();
                if (sub == 0)
                    for (int s = 1; s < each; ++s)
#pragma unroll
                        for (int e = 0; e < EACH; ++e)
                            if (lane + 32 * e < VECTORS) {
                                const float4 v = sums[warp + s][lane + 32 * e];
                                acc[e].x += v.x, acc[e].y += v.y, acc[e].z += v.z, acc[e].w += v.w;
                            }
                __syncthreads();
            }
            if (r < rows && sub == 0) {
                const PagedRow row(m, l, beyond);
                T* o = static_cast<T*>(a.out) + b * a.ldo + int64_t(head + r) * a.D;
#pragma unroll
                for (int e = 0; e < EACH; ++e) {
                    const float v[4] = {acc[e].x, acc[e].y, acc[e].z, acc[e].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * (lane + 32 * e) + i < a.D) E::store(o + 4 * (lane + 32 * e) + i, v[i] * row.inv);
                }
                if (lane == 0 && a.lse) a.lse[b * a.heads + head + r] = row.lse;
            }
        }
    }
}

template <class P>
cudaError_t paged_launch(const PagedArgs& a, void* workspace, int blocks, const LaunchCfg& cfg) {
    const int V = 16 / int(sizeof(typename P::T));
    auto even = [&](int64_t count, int64_t stride) { return count <= 1 || stride % V == 0; };
    const bool whole = a.D % V == 0 && even(a.pages, a.page_stride) && even(a.page, a.slot_stride) &&
                       even(a.kv_heads, a.head_stride) && reinterpret_cast<uintptr_t>(a.k) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.v) % 16 == 0;
    const int64_t units = a.kv_heads * blocks;
    const size_t smem = P::Ring::kBytes + size_t(P::kRows) * P::kPitch * 4 + P::kScratch;
    const PagedForm form = paged_form(a.B, a.heads, a.kv_heads, a.D, a.max_pages * a.page, a.window, int(sizeof(typename P::T)));
    if (form.cluster) {
        auto k = paged_attention_kernel<P, true>;
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem, cfg);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t lc = {};
        lc.gridDim = dim3(unsigned(a.B * units * form.cluster));
        lc.blockDim = dim3(kPagedBlock);
        lc.dynamicSmemBytes = smem;
        lc.stream = cfg.stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(form.cluster);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
        return cudaLaunchKernelEx(&lc, k, a, static_cast<float*>(nullptr), blocks, whole);
    }
    auto k = paged_attention_kernel<P, false>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem, cfg);
    if (e != cudaSuccess) return e;
    LaunchCfg one = cfg;
    one.ctas_per_sm = 0;
    const int ctas = std::min(grid_for(reinterpret_cast<const void*>(k), kPagedBlock, smem, form.tiles, one), kPagedMaxCtas);
    k<<<ctas, kPagedBlock, smem, cfg.stream>>>(a, static_cast<float*>(workspace), blocks, whole);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(unsigned(a.B), unsigned(std::min<int64_t>(units, std::max<int64_t>(1, 2048 / a.B))));
    const bool few = a.B * units <= cfg.num_sms;
    lc.blockDim = dim3(32 * (few ? 32 : 8));
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, few ? paged_join_kernel<P, 32> : paged_join_kernel<P, 8>, a,
                              static_cast<const float*>(workspace), blocks, ctas);
}

}  // namespace rowops
