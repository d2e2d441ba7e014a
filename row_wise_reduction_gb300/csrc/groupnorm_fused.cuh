// Group norm + activation and its backward in one kernel that reads every
// tensor once: a cluster of CTAs holds a slab -- a sample's positions of a block
// of whole groups -- in shared memory between the two passes. CTA `rank` of
// the cluster takes positions [rank R, (rank + 1) R).
//
// Vectors: the slab comes in as boxes of rows by tensor copies (a block of groups
// is often narrower than a row, 80 to 640 bytes of it, which costs per-thread
// copies and stores several times the instructions and shared-memory wavefronts
// that it moves data with), is worked on box by box as it arrives, and the
// results go out the same way from the same boxes. Rows that are no whole vectors
// come and go by two elements or one.
//
// As many clusters as the device holds at once take the slabs in turn: as soon as a
// box of one slab has gone out the same box of the next comes in, so the memory
// system works through the exchange, and no cluster waits for another one's
// places to fall free.
//
// The exchange: every CTA writes its groups' sums into the shared memory of
// all CTAs of the cluster and then meets them at one cluster barrier; each adds
// up what it got in order of rank. Sums are joined as (mean, squares about it) about
// one of their own members, so no more than the count of members cancels.
//
// bf16 SiLU B8 S4096 C320: 16 us (2.7 TB/s), backward 33 us (1.9 TB/s); B2 S64 C1280
// 6.2 us, a launch and an exchange. Bound by the arithmetic of the two passes (16 warps
// an SM; the special-function and FMA pipes) and, with few slabs, by the latency of
// copy, exchange and copy out, which follow one another. Two CTAs for each SM: one alone, with
// slabs of twice the size, took 29 us for the first.
#pragma once

#include "groupnorm_kernels.cuh"
#include "row_pipeline.cuh"

namespace rowops {

__device__ __forceinline__ void tensor_load(void* dst, const RowsMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tensor_store(const RowsMap* map, int x, int y, const void* src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                 "r"(y), "r"(smem_addr(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void tensor_stores_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// What a thread of the fused kernels works on: its place in the cluster's slabs, and
// the slab at hand.
template <typename T, int VEC>
struct GnTile {
    using V = Vec<T, VEC>;
    const GnArgs& a;
    const GnFused& f;
    int rank, t, tx, ty;
    int rows;      // positions of the CTA
    bool active;
    unsigned slab, slabs, stride;
    int turn = 0;  // slabs done
    int block;
    int64_t sample, at;  // at: element offset of the thread's channels at the CTA's first position
    __device__ __forceinline__ GnTile(const GnArgs& a_, const GnFused& f_) : a(a_), f(f_) {
        rank = int(blockIdx.x) & (f.cluster - 1);
        t = threadIdx.x;
        ty = t * f.inv_tx >> 16;
        tx = t - ty * f.tx;
        active = ty < f.ty;
        const int64_t left = a.S - int64_t(rank) * f.rows;
        rows = int(left < f.rows ? (left > 0 ? left : 0) : f.rows);
        slab = blockIdx.x >> f.cluster_log2;
        stride = gridDim.x >> f.cluster_log2;
        slabs = unsigned(a.B) * unsigned(f.blocks);
        place();
    }
    __device__ __forceinline__ void place() {
        const unsigned n = slab / unsigned(f.blocks);
        block = int(slab - n * f.blocks);
        sample = n;
        at = first() * a.ld + int64_t(block) * f.W + tx * VEC;
    }
    // element offset of a slab's first channel at its sample's first position
    __device__ __forceinline__ int64_t origin(unsigned s) const {
        const unsigned n = s / unsigned(f.blocks);
        return int64_t(n) * a.S * a.ld + int64_t(s - n * f.blocks) * f.W;
    }
    __device__ __forceinline__ int64_t first() const { return sample * a.S + int64_t(rank) * f.rows; }
    __device__ __forceinline__ bool more() const { return slabs - slab > stride; }
    __device__ __forceinline__ void next() {
        slab += stride;
        ++turn;
        if (slab < slabs) place();
    }
    // g(words of N tiles, place in the tile, position) over the thread's positions, U of
    // them at a time: their words are read before the first is used, and a result kept
    // in the tile does not hold up the next one's. Every thread of the CTA calls
    // need(p) before positions below p are read and done(p) when they are worked on.
    template <int U, int N, typename Need, typename F, typename Done>
    __device__ __forceinline__ void each(const typename V::Word* const (&tiles)[N], Need need, F g, Done done) const {
        const int step = f.ty * f.tx;
        int at = ty * f.tx + tx, i = 0;
        for (; i + U * f.ty <= rows; i += U * f.ty, at += U * step) {
            need(i + U * f.ty);
            if (active) {
                typename V::Word w[U][N];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < N; ++k) w[u][k] = tiles[k][at + u * step];
#pragma unroll
                for (int u = 0; u < U; ++u) g(w[u], at + u * step, i + u * f.ty + ty);
            }
            done(i + U * f.ty);
        }
        for (; i < rows; i += f.ty, at += step) {
            const int end = min(i + f.ty, rows);
            need(end);
            if (active && i + ty < rows) {
                typename V::Word w[N];
#pragma unroll
                for (int k = 0; k < N; ++k) w[k] = tiles[k][at];
                g(w, at, i + ty);
            }
            done(end);
        }
    }
};

// Thread 0 asks for box q of a slab in N tensors.
template <typename T, int VEC, int N>
__device__ __forceinline__ void gn_ask(const GnTile<T, VEC>& k, unsigned slab, const RowsMap* const (&maps)[N],
                                       typename Vec<T, VEC>::Word* tile, uint64_t* bars, int q, unsigned extra) {
    const GnFused& f = k.f;
    const unsigned n = slab / unsigned(f.blocks);
    const int x = int(slab - n * f.blocks) * f.W * int(sizeof(T)) / 8;
    const int y = int(int64_t(n) * k.a.S) + k.rank * f.rows + q * f.box;
    mbar_expect_tx(&bars[q], unsigned(N * f.box * f.W * sizeof(T)) + extra);
#pragma unroll
    for (int i = 0; i < N; ++i) tensor_load(tile + (i * f.boxes + q) * f.pitch, maps[i], x, y, &bars[q]);
}

// The first slab's copies in (one or two elements: every slab's).
template <typename T, int VEC, int N>
__device__ __forceinline__ void gn_fetch(const GnTile<T, VEC>& k, const RowsMap* const (&maps)[N],
                                         const T* const (&from)[N], typename Vec<T, VEC>::Word* tile, uint64_t* bars,
                                         int64_t stall_row) {
    if constexpr (Vec<T, VEC>::kWhole) {
        if (k.t == 0 && k.turn == 0) {
            for (int q = 0; q < k.f.boxes; ++q) mbar_init(&bars[q], 1);
            mbar_init_fence();
            const bool stall = stall_row >= k.first() && stall_row < k.first() + k.rows;
            for (int q = 0; q * k.f.box < k.rows; ++q)
                gn_ask<T, VEC, N>(k, k.slab, maps, tile, bars, q, stall && q == 0 ? 16u : 0u);
        }
    } else {
        if (k.active) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll 8
                for (int r = k.ty; r < k.rows; r += k.f.ty)
                    tile[i * k.f.pitch + r * k.f.tx + k.tx] = Vec<T, VEC>::load(from[i] + k.at + r * k.a.ld);
        }
    }
}

// The first pass: g over the thread's positions as the boxes arrive; nonzero in the
// threads whose wait ran out, which wait for no further box.
template <int U, typename T, int VEC, int N, typename F>
__device__ __forceinline__ int gn_read(const GnTile<T, VEC>& k, const typename Vec<T, VEC>::Word* const (&tiles)[N],
                                       uint64_t* bars, int fail, unsigned long long wait_ns, F g) {
    int late = 0, q = 0;
    k.template each<U, N>(
        tiles,
        [&](int end) {
            if constexpr (Vec<T, VEC>::kWhole)
                for (; q * k.f.box < end; ++q)
                    if (!fail && !late) late = !mbar_wait(&bars[q], k.turn & 1, wait_ns);
        },
        g, [](int) {});
    return late;
}

// The second pass: g(words, place, position, whole) over the thread's positions, whole: the
// result is kept in the first tile; a box that is done goes out and the next slab's comes in.
template <int U, typename T, int VEC, int N, typename F>
__device__ __forceinline__ void gn_write(const GnTile<T, VEC>& k, const RowsMap* const (&maps)[N], const RowsMap* out,
                                         typename Vec<T, VEC>::Word* tile,
                                         const typename Vec<T, VEC>::Word* const (&tiles)[N], uint64_t* bars,
                                         int fail, F g) {
    const GnFused& f = k.f;
    constexpr bool kWhole = Vec<T, VEC>::kWhole;
    const bool more = kWhole && !fail && k.more();
    const int whole = kWhole ? k.rows / f.box * f.box : 0;  // positions that go out as boxes
    int q = 0;
    k.template each<U, N>(
        tiles, [](int) {}, [&](const typename Vec<T, VEC>::Word (&w)[N], int at, int r) { g(w, at, r, r < whole); },
        [&](int end) {
            if constexpr (Vec<T, VEC>::kWhole) {
                for (; min((q + 1) * f.box, k.rows) <= end && q * f.box < k.rows; ++q) {
                    fence_proxy_async_smem();
                    __syncthreads();
                    if (k.t == 0 && !fail) {
                        const bool box = q * f.box < whole;
                        if (box)
                            tensor_store(out, k.block * f.W * int(sizeof(T)) / 8, int(k.first()) + q * f.box,
                                         tile + q * f.pitch);
                        if (more && q > 0) {
                            if (box) tensor_stores_read<1>();
                            else tensor_stores_read<0>();
                            gn_ask<T, VEC, N>(k, k.slab + k.stride, maps, tile, bars, q - 1, 0u);
                        }
                    }
                }
            }
        });
    if (kWhole && k.t == 0 && !fail && k.rows > 0) {
        tensor_stores_read<0>();
        if (more) gn_ask<T, VEC, N>(k, k.slab + k.stride, maps, tile, bars, (k.rows - 1) / f.box, 0u);
    }
}

// After a wait that ran out: nothing more is asked for or written; the copies still
// in flight get one more wait, of one limit for them all, and the error word is set.
template <typename T, int VEC>
__device__ __forceinline__ void break_waits(const GnTile<T, VEC>& k, uint64_t* bars, unsigned* err, unsigned long long wait_ns) {
    if (!Vec<T, VEC>::kWhole || k.t != 0) return;
    const unsigned long long t0 = global_ns();
    for (int q = 0; q * k.f.box < k.rows; ++q) {
        const unsigned long long spent = global_ns() - t0;
        mbar_wait(&bars[q], k.turn & 1, spent < wait_ns ? wait_ns - spent : 0);
    }
    atomicExch(err, kDeviceErrTimeout);
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock, 2)
    gn_fused_kernel(const __grid_constant__ RowsMap mx, const __grid_constant__ RowsMap my, const T* x, T* y,
                    const T* w, const T* b, float2* stats_out, const __grid_constant__ GnArgs a,
                    const __grid_constant__ GnFused f, unsigned* err, unsigned long long wait_ns, int64_t stall_row) {
    using V = Vec<T, VEC>;
    constexpr int P = V::P;
    extern __shared__ __align__(128) char smem[];
    const cg::cluster_group cl = cg::this_cluster();
    if (f.cluster > 1) cl.barrier_arrive();  // met before the first write to another CTA
    GnTile<T, VEC> k(a, f);
    const int Gb = f.W / a.L;
    typename V::Word* tile = reinterpret_cast<typename V::Word*>(smem);
    float* pm = reinterpret_cast<float*>(smem + f.tile);      // [ty][W] the threads' means
    float* pq = pm + f.ty * f.W;                              // [ty][W] and squares
    float2* col = reinterpret_cast<float2*>(pq + f.ty * f.W);  // [W] the channels'
    float2* gs = col + f.W;                                   // [Gb] mean, rstd
    float2* gots = gs + Gb;                                   // [2][cluster][Gb]: every CTA's mean, squares
    uint64_t* bars = reinterpret_cast<uint64_t*>(gots + 2 * f.cluster * Gb);  // [boxes]
    float* count = reinterpret_cast<float*>(bars + f.boxes);  // [ty] positions of the threads
    float* refs = count + f.ty;                               // [Gb] what the means are kept less of
    const RowsMap* const maps[1] = {&mx};
    const T* const from[1] = {x};
    const typename V::Word* const tiles[1] = {tile};
    const float inv_rows = k.rows ? 1.f / float(k.rows) : 0.f;
    const int c = k.tx * VEC;
    int fail = 0;
    // the slab's first refs, a slab ahead; not by the warp that asks for the boxes
    const int own = k.t - 32;
    const bool ahead = own >= 0 && own < Gb;
    float ref = ahead ? Elem<T>::load(x + k.origin(k.slab) + own * a.L) : 0.f;
    for (; k.slab < k.slabs; k.next()) {
        gn_fetch<T, VEC, 1>(k, maps, from, tile, bars, stall_row);
        // two sets, as a CTA may be one exchange behind
        float2* got = gots + (k.turn & 1) * f.cluster * Gb;
        const int cb = k.block * f.W + c;
        float2 mul[P], shift[P];
        if (k.active) {
            load_affine<T, VEC>(w, cb, 1.f, mul);
            load_affine<T, VEC>(b, cb, 0.f, shift);
        }
        if (own >= 0)
            for (int g = own; g < Gb; g += kGnBlock - 32)
                refs[g] = g == own ? ref : Elem<T>::load(x + k.origin(k.slab) + g * a.L);
        __syncthreads();  // they are there, and the barriers are set up

        Shifted<P> sums;
        sums.clear();
        int n = 0;
        const int late = gn_read<4>(k, tiles, bars, fail, wait_ns, [&](const typename V::Word (&wd)[1], int, int) {
            float2 v[P];
            V::get(wd[0], v);
            if (n == 0) sums.start(v);
            sums.add(v);
            ++n;
        });
        if (k.active) {
            sums.template leave<VEC>(n, Groups<VEC>(c, a), refs, pm + k.ty * f.W + c, pq + k.ty * f.W + c);
            if (k.tx == 0) count[k.ty] = float(n);
        }
        const int before = fail;
        fail |= __syncthreads_or(late);
        // the channels: means and squares about them, about the first thread's mean
        by_teams(f.W, f.parts_log2, [&](int ch, int lane, bool live) {
            const float ref = pm[ch];
            float2 s = f2(0.f);
            for (int r = lane; r < f.ty; r += 1 << f.parts_log2) {
                const float m = count[r], d = pm[r * f.W + ch] - ref;
                s.x = fmaf(m, d, s.x);
                s.y += fmaf(m * d, d, pq[r * f.W + ch]);
            }
            s = lanes_sum(s, 1 << f.parts_log2);
            if (live && lane == 0) col[ch] = joined(ref, s, 1.f, inv_rows);
        });
        __syncthreads();
        if (f.cluster > 1 && k.turn == 0) cl.barrier_wait();
        by_teams(Gb, f.team_log2, [&](int g, int lane, bool live) {
            const float2* cg_ = col + g * a.L;
            const float ref = cg_[0].x, m = float(k.rows);
            float2 s = f2(0.f);
            for (int i = lane; i < a.L; i += 1 << f.team_log2) {
                const float d = cg_[i].x - ref;
                s.x += d;
                s.y += fmaf(m * d, d, cg_[i].y);
            }
            s = lanes_sum(s, 1 << f.team_log2);
            const float2 mine = k.rows ? joined(ref, s, m, a.inv_L) : f2(0.f);
            if (live)
                for (int r = lane; r < f.cluster; r += 1 << f.team_log2)
                    *in_cta(cl, &got[k.rank * Gb + g], r, f.cluster) = mine;
        });
        if (f.cluster > 1) cl.sync();
        else __syncthreads();
        by_teams(Gb, f.cluster_log2, [&](int g, int r, bool live) {
            const int64_t left = a.S - int64_t(r) * f.rows;
            const float m = float(left < f.rows ? (left > 0 ? left : 0) : f.rows);
            const float ref = got[g].x;
            const float2 v = got[r * Gb + g];
            const float d = v.x - ref;
            const float2 s = lanes_sum(make_float2(m * d, fmaf(m * float(a.L) * d, d, v.y)), f.cluster);
            if (live && r == 0) {
                const float2 u = joined(ref, s, float(a.L), a.inv_S);
                gs[g] = make_float2(refs[g] + u.x, rsqrtf(u.y * a.inv_m + a.eps));
                if (stats_out && k.rank == 0) stats_out[k.sample * a.G + k.block * Gb + g] = gs[g];
            }
        });
        __syncthreads();
        float2 mean[P];
        if (k.active) {
            const Groups<VEC> g(c, a);
            float2 rstd[P];
            each_channel<VEC>(mean, [&](int e) { return -gs[g.g[e]].x; });
            each_channel<VEC>(rstd, [&](int e) { return gs[g.g[e]].y; });
#pragma unroll
            for (int j = 0; j < P; ++j) mul[j] = f2_mul(mul[j], rstd[j]);
        }
        if (ahead && k.more()) ref = Elem<T>::load(x + k.origin(k.slab + k.stride) + own * a.L);
        T* py = y + k.at;
        gn_write<2>(k, maps, &my, tile, tiles, bars, fail,
                    [&](const typename V::Word (&wd)[1], int at, int r, bool whole) {
                        float2 v[P];
                        V::get(wd[0], v);
#pragma unroll
                        for (int j = 0; j < P; ++j)
                            v[j] = act_of2<ACT>(f2_fma(f2_add(v[j], mean[j]), mul[j], shift[j]));
                        if (whole) V::keep(&tile[at], v);
                        else if (!fail) V::put(py + r * a.ld, v);
                    });
        if (fail && !before) break_waits(k, bars, err, wait_ns);
    }
}

// chan: a row of 2 C sums (dz xh, then dz) for every CTA of a sample.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock, 2)
    gn_bwd_fused_kernel(const __grid_constant__ RowsMap mx, const __grid_constant__ RowsMap md,
                        const __grid_constant__ RowsMap mo, const T* x, const T* dy, T* dx, const T* w, const T* b,
                        const float2* stats, float* chan, const __grid_constant__ GnArgs a,
                        const __grid_constant__ GnFused f, unsigned* err, unsigned long long wait_ns,
                        int64_t stall_row) {
    using E = Elem<T>;
    using V = Vec<T, VEC>;
    constexpr int P = V::P;
    extern __shared__ __align__(128) char smem[];
    const cg::cluster_group cl = cg::this_cluster();
    if (f.cluster > 1) cl.barrier_arrive();
    GnTile<T, VEC> k(a, f);
    const int Gb = f.W / a.L;
    typename V::Word* tx = reinterpret_cast<typename V::Word*>(smem);
    typename V::Word* td = tx + f.boxes * f.pitch;
    float2* red = reinterpret_cast<float2*>(smem + f.tile);  // [ty][W]: the threads' A, Q
    float2* col = red + f.ty * f.W;                          // [W]: the channels', times w
    float2* gs = col + f.W;                                  // [Gb]: -c1, -c2
    float2* gots = gs + Gb;                                  // [2][cluster][Gb]
    uint64_t* bars = reinterpret_cast<uint64_t*>(gots + 2 * f.cluster * Gb);  // [boxes]
    const RowsMap* const maps[2] = {&mx, &md};
    const T* const from[2] = {x, dy};
    const typename V::Word* const tiles[2] = {tx, td};
    const int c = k.tx * VEC;
    int fail = 0;
    let_next_start();
    for (; k.slab < k.slabs; k.next()) {
        gn_fetch<T, VEC, 2>(k, maps, from, tx, bars, stall_row);
        float2* got = gots + (k.turn & 1) * f.cluster * Gb;
        GnSlope<T, VEC, ACT> slope;
        if (k.active) slope.load(w, b, stats + k.sample * a.G + k.block * Gb, c, k.block * f.W + c, a);
        if (k.turn == 0) __syncthreads();

        float2 sa[P], sq[P];
#pragma unroll
        for (int j = 0; j < P; ++j) sa[j] = sq[j] = f2(0.f);
        const int late = gn_read<2>(k, tiles, bars, fail, wait_ns, [&](const typename V::Word (&wd)[2], int, int) {
            slope.add(wd[0], wd[1], sa, sq);
        });
        if (k.active) slope.leave(sa, sq, red + k.ty * f.W + c);
        const int own = k.t >> f.parts_log2;  // the channel of the thread's first team
        const float w_own = w && own < f.W ? E::load(w + k.block * f.W + own) : 1.f;
        const int before = fail;
        fail |= __syncthreads_or(late);
        float* cw = chan + (k.sample * f.cluster + k.rank) * 2 * a.C + k.block * f.W;
        by_teams(f.W, f.parts_log2, [&](int ch, int lane, bool live) {
            float2 s = f2(0.f);
            for (int r = lane; r < f.ty; r += 1 << f.parts_log2) s = f2_add(s, red[r * f.W + ch]);
            s = lanes_sum(s, 1 << f.parts_log2);
            if (live && lane == 0) {
                cw[ch] = s.y;
                cw[a.C + ch] = s.x;
                const float wv = !w || ch == own ? w_own : E::load(w + k.block * f.W + ch);
                col[ch] = make_float2(wv * s.x, wv * s.y);
            }
        });
        __syncthreads();
        if (f.cluster > 1 && k.turn == 0) cl.barrier_wait();
        by_teams(Gb, f.team_log2, [&](int g, int lane, bool live) {
            float2 s = f2(0.f);
            for (int i = lane; i < a.L; i += 1 << f.team_log2) s = f2_add(s, col[g * a.L + i]);
            s = lanes_sum(s, 1 << f.team_log2);
            if (live)
                for (int r = lane; r < f.cluster; r += 1 << f.team_log2)
                    *in_cta(cl, &got[k.rank * Gb + g], r, f.cluster) = s;
        });
        if (f.cluster > 1) cl.sync();
        else __syncthreads();
        by_teams(Gb, f.cluster_log2, [&](int g, int r, bool live) {
            const float2 s = lanes_sum(got[r * Gb + g], f.cluster);
            if (live && r == 0) gs[g] = make_float2(-s.x * a.inv_m, -s.y * a.inv_m);
        });
        __syncthreads();
        if (k.active) slope.means([&](int g) { return gs[g]; }, c, a);
        T* po = dx + k.at;
        gn_write<2>(k, maps, &mo, tx, tiles, bars, fail,
                    [&](const typename V::Word (&wd)[2], int at, int r, bool whole) {
                        float2 v[P];
                        slope.of(wd[0], wd[1], v);
                        if (whole) V::keep(&tx[at], v);
                        else if (!fail) V::put(po + r * a.ld, v);
                    });
        if (fail && !before) break_waits(k, bars, err, wait_ns);
    }
}

// ---- launchers -------------------------------------------------------------
inline cudaError_t gn_cluster_launch(const void* kern, const GnFused& f, int64_t B, const LaunchCfg& cfg,
                                     void** args) {
    cudaError_t e = allow_smem(kern, f.smem, cfg);
    if (e == cudaSuccess && f.cluster > 8)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    const int64_t held = clusters_on_device(kern, kGnBlock, f.smem, f.cluster, cfg);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(unsigned(std::min(B * f.blocks, held) * f.cluster));
    lc.blockDim = dim3(kGnBlock);
    lc.dynamicSmemBytes = f.smem;
    lc.stream = cfg.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(f.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelExC(&lc, kern, args);
}

template <typename T, int VEC>
cudaError_t gn_map(RowsMap* m, const void* p, const GnArgs& a, const GnFused& f) {
    if (!Vec<T, VEC>::kWhole) return cudaSuccess;
    return rows_map(m, p, a.C * int64_t(sizeof(T)), int64_t(a.B) * a.S, a.ld * int64_t(sizeof(T)),
                    f.W * int(sizeof(T)), f.box);
}

template <typename T, int VEC, int ACT>
cudaError_t gn_forward_fused(const void* x, void* y, const void* w, const void* b, float* stats, GnArgs a,
                             const GnFused& f0, const LaunchCfg& cfg) {
    auto kern = gn_fused_kernel<T, VEC, ACT>;
    GnFused f = f0;
    RowsMap mx, my;
    cudaError_t e = gn_map<T, VEC>(&mx, x, a, f);
    if (e == cudaSuccess) e = gn_map<T, VEC>(&my, y, a, f);
    if (e != cudaSuccess) return e;
    unsigned* err = cfg.dev_error;
    unsigned long long wait_ns = cfg.wait_ns;
    int64_t stall = cfg.stall_row;
    void* args[] = {&mx, &my, &x, &y, &w, &b, &stats, &a, &f, &err, &wait_ns, &stall};
    return gn_cluster_launch(reinterpret_cast<const void*>(kern), f, a.B, cfg, args);
}

template <typename T, int VEC, int ACT>
cudaError_t gn_backward_fused(const void* x, const void* dy, const void* w, const void* b, const float* stats,
                              void* dx, float* dw, float* db, void* ws, GnArgs a, const GnFused& f0,
                              const LaunchCfg& cfg) {
    auto kern = gn_bwd_fused_kernel<T, VEC, ACT>;
    GnFused f = f0;
    RowsMap mx, md, mo;
    cudaError_t e = gn_map<T, VEC>(&mx, x, a, f);
    if (e == cudaSuccess) e = gn_map<T, VEC>(&md, dy, a, f);
    if (e == cudaSuccess) e = gn_map<T, VEC>(&mo, dx, a, f);
    if (e != cudaSuccess) return e;
    float* chan = static_cast<float*>(ws);
    unsigned* err = cfg.dev_error;
    unsigned long long wait_ns = cfg.wait_ns;
    int64_t stall = cfg.stall_row;
    void* args[] = {&mx, &md, &mo, &x, &dy, &dx, &w, &b, &stats, &chan, &a, &f, &err, &wait_ns, &stall};
    e = gn_cluster_launch(reinterpret_cast<const void*>(kern), f, a.B, cfg, args);
    return e == cudaSuccess ? gn_reduce_channels(chan, int64_t(a.B) * f.cluster, a.C, dw, db, cfg) : e;
}

}  // namespace rowops
