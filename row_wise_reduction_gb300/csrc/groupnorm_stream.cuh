// Group norm + activation and its backward for samples too large to hold: one
// persistent kernel that reads the tensors twice, forward the second time from L2.
//
// The work is a sequence of items, each a chunk of a sample's positions: one that
// adds up ("sums") and one that writes ("apply"). CTAs take them off the sequence
// with a counter. An apply item stands behind all sums of its sample, by as much as
// the CTAs have in hand, so its sample's results are there when it is taken. In batches
// of more chunks than that (a sample's and one for every CTA), sums of later samples and
// writes of earlier ones share the memory system meanwhile; in all others the two kinds
// are two phases, one after the other. Forward at most 456 chunks of 192 KiB and a sample
// lie between a chunk's two reads, 90 MB, which L2 (129 MB) holds; backward 304 of 512
// KiB, 160 MB and more, so x and dy come from memory a second time (shorter distances by
// smaller chunks cost more than that: gn_plan). Whoever finishes a sample's last sums adds up its
// chunks, in order. An apply item that comes too early waits (with a limit); it
// waits for items before it in the sequence alone, and sums never wait, so the
// waits end whatever CTAs run at the same time.
//
// bf16 SiLU B32 S4096 C320: 47.4 us (3.5 TB/s of what must be moved once), backward 77 us
// (3.3 TB/s); B1 S262144 C128: 50.6 us. The reads of the sums run at 5 TB/s beside the
// write-back of what the last call wrote; forward the second pass takes as long from L2
// as the first from memory; where there are two phases nothing is done while the sums
// are joined (7 us).
#pragma once

#include "async_ring.cuh"
#include "groupnorm_kernels.cuh"
#include "row_pipeline.cuh"

namespace rowops {

// A thread's n positions, `step` elements apart, of N tensors (LAST: for the last time, so
// that they give up their places in L2 first: 2% on every size measured): run(f) calls f(words)
// for each in order. Vectors come through a ring of copies, D positions on their
// way, the first of them asked for by the constructor: what else a pass needs first
// (its parameters, a wait) goes between. One or two elements: U positions at a time.
template <typename T, int VEC, int D, int N, bool LAST>
struct Walk {
    using V = Vec<T, VEC>;
    const T* p[N];
    int64_t step;
    int n;
    uint4* at;
    uint64_t policy = 0;
    __device__ __forceinline__ Walk(const T* const (&from)[N], int64_t step_, int n_, uint4* slots)
        : step(step_), n(n_), at(slots + threadIdx.x) {
#pragma unroll
        for (int k = 0; k < N; ++k) p[k] = from[k];
        if constexpr (LAST && V::kWhole) policy = evict_first_policy();
        if constexpr (V::kWhole)
#pragma unroll
            for (int d = 0; d < D - 1; ++d) ask(d, d);
    }
    __device__ __forceinline__ void ask(int d, int i) {
        if (i < n)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if constexpr (LAST) copy_async16(at + (d * N + k) * kGnBlock, p[k], policy);
                else copy_async<16>(at + (d * N + k) * kGnBlock, p[k]);
                p[k] += step;
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // for a walk that does not run
    __device__ __forceinline__ void drop() const {
        if constexpr (V::kWhole) asm volatile("cp.async.wait_all;" ::: "memory");
    }
    template <typename F>
    __device__ __forceinline__ void run(F f) {
        if constexpr (V::kWhole) {
            // unrolled over the ring, so that a slot's place is a constant
#pragma unroll 1
            for (int i = 0; i < n; i += D) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    ask((d + D - 1) % D, i + d + D - 1);
                    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
                    if (i + d < n) {
                        typename V::Word w[N];
#pragma unroll
                        for (int k = 0; k < N; ++k) w[k] = at[(d * N + k) * kGnBlock];
                        f(w);
                    }
                }
            }
        } else {
            constexpr int U = 4;
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
    }
};
template <typename T, int VEC, int D, int N>
constexpr size_t walk_smem() {
    return Vec<T, VEC>::kWhole ? size_t(D) * N * kGnBlock * 16 : 0;
}

// The workspace: the item counter and counters for each sample (zeroed before the
// kernel), results for each sample's groups, sums of each chunk's and bunch's.
struct GnStreamWs {
    unsigned* next;
    unsigned* done;        // [B] sets of sums added up; kGnThere: the results are there
    unsigned* bunch_done;  // [B bunches] chunks added up
    float2* result;        // [B][G] mean, rstd; backward -c1, -c2
    float2* part;          // [B chunks][G]
    float2* bunch;         // [B bunches][G]
    float* chans;    // backward: [B chunks][2 C] sums of dz xh, dz
};

static __global__ void gn_zero_kernel(unsigned* p, int64_t n) {
    let_next_start();
    grid_wait();
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0u;
}

constexpr unsigned kGnThere = 0x80000000u;
constexpr int kGnStreamDepth = 6, kGnStreamDepthBwd = 4;

// Items of the sequence: `lag` sums, then apply and sums in turn, then apply.
struct GnItem {
    bool apply;
    int sample, chunk;
    __device__ __forceinline__ GnItem(unsigned i, const GnArgs& a) {
        const unsigned N = unsigned(a.B) * a.chunks, lag = unsigned(a.lag);
        unsigned k = i;
        apply = false;
        if (i >= lag) {
            const unsigned j = i - lag;
            if (j < 2 * (N - lag)) {
                apply = !(j & 1);
                k = apply ? j >> 1 : lag + (j >> 1);
            } else {
                apply = true;
                k = j - (N - lag);
            }
        }
        sample = int(k / unsigned(a.chunks));
        chunk = int(k - unsigned(sample) * a.chunks);
        if (apply) chunk = a.chunks - 1 - chunk;  // what was read last first
    }
};

// The thread's share of an item.
struct GnShare {
    int tx, ty, n, rows;   // n: its positions; rows: the chunk's
    int64_t first, step;   // element offsets of its first position (channel 0), between them
    __device__ __forceinline__ GnShare(const GnArgs& a, const GnItem& it) {
        ty = int(threadIdx.x) * a.inv_tx >> 16;
        tx = int(threadIdx.x) - ty * a.tx;
        const int64_t r0 = int64_t(it.chunk) * a.chunk_rows, left = a.S - r0;
        rows = int(left < a.chunk_rows ? left : a.chunk_rows);
        n = ty < a.ty && rows > ty ? (rows - ty + a.ty - 1) / a.ty : 0;
        first = (int64_t(it.sample) * a.S + r0 + ty) * a.ld;
        step = int64_t(a.ty) * a.ld;
    }
};

// Counts the CTA's sums in; true in every thread where they were the last of `sets`.
__device__ __forceinline__ bool gn_last(unsigned* done, int sets, unsigned* word) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        *word = atomicAdd(done, 1u);
    }
    __syncthreads();
    if (*word != unsigned(sets - 1)) return false;
    __threadfence();
    return true;
}

// The CTA adds up n sets of sums of G groups, in order; set i is of `rows` positions,
// S in all. Forward (MEANS: a group's mean, less its first value, and squares about it) the
// means enter less the first set's; to[g] is the same of all sets or, `last`, mean and
// rstd (x: the sample's first position). Backward the
// plain sums, times -inv_m at the last. A function of its own, and a short one: it runs
// once or twice in a CTA, and its time is that of fetching its code and waiting for
// its loads.
template <bool MEANS, typename T>
__device__ __noinline__ void gn_join(const float2* sets, int n, int64_t S, int64_t rows, bool last, float2* to,
                                     float2* also, const T* x, const GnArgs& a) {
    by_teams(a.G, a.last_log2, [&](int g, int lane, bool live) {
        const float2* p = sets + g;
        const float first = MEANS && last ? Elem<T>::load(x + g * a.L) : 0.f;
        const float ref = MEANS ? __ldcg(p).x : 0.f;
        const int step = 1 << a.last_log2;
        float2 s = f2(0.f);
#pragma unroll 1
        for (int i = lane; i < n; i += 4 * step) {
            float2 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u * step < n) v[u] = __ldcg(p + int64_t(i + u * step) * a.G);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u * step < n) {
                    if constexpr (MEANS) {
                        const int64_t left = S - (i + u * step) * rows;
                        const float m = float(left < rows ? left : rows), d = v[u].x - ref;
                        s.x = fmaf(m, d, s.x);
                        s.y += fmaf(m * float(a.L) * d, d, v[u].y);
                    } else {
                        s = f2_add(s, v[u]);
                    }
                }
        }
        s = lanes_sum(s, step);
        if (!live || lane != 0) return;
        if constexpr (MEANS) {
            s = joined(ref, s, float(a.L), 1.f / float(S));
            if (last) s = make_float2(first + s.x, rsqrtf(s.y * a.inv_m + a.eps));
        } else if (last) {
            s = make_float2(-s.x * a.inv_m, -s.y * a.inv_m);
        }
        to[g] = s;
        if (also) also[g] = s;
    });
}

// A sample's chunks' sums (or a bunch's, where chunks go in bunches) are in: joins them.
template <bool MEANS, typename T>
__device__ __forceinline__ bool gn_joined(const GnItem& it, const GnArgs& a, const GnStreamWs& ws, const T* x,
                                          float2* stats, unsigned* word) {
    const float2* part = ws.part + int64_t(it.sample) * a.chunks * a.G;
    int n = a.chunks;
    int64_t rows = a.chunk_rows;
    if (a.bunches > 1) {
        const int k = it.chunk / a.bunch, first = k * a.bunch, size = min(a.bunch, a.chunks - first);
        if (!gn_last(&ws.bunch_done[int64_t(it.sample) * a.bunches + k], size, word)) return false;
        float2* to = ws.bunch + int64_t(it.sample) * a.bunches * a.G;
        const int64_t at = first * rows, left = a.S - at;
        gn_join<MEANS>(part + int64_t(first) * a.G, size, left < a.bunch * rows ? left : a.bunch * rows, rows, false,
                       to + k * a.G, nullptr, x, a);
        part = to;
        n = a.bunches;
        rows *= a.bunch;
    }
    if (!gn_last(&ws.done[it.sample], n, word)) return false;
    gn_join<MEANS>(part, n, a.S, rows, true, ws.result + int64_t(it.sample) * a.G,
                   stats ? stats + int64_t(it.sample) * a.G : nullptr, x + it.sample * a.S * a.ld, a);
    __syncthreads();
    return true;
}

// Every thread of the CTA: the sample's results are there; false where the wait ran out.
__device__ __forceinline__ bool gn_ready(const unsigned* done, unsigned long long wait_ns) {
    int ok = 1;
    if (threadIdx.x == 0) {
        auto there = [&] {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
            return v == kGnThere;
        };
        if (!there()) {
            const unsigned long long t0 = global_ns();
            ok = 0;
            for (uint32_t i = 0; i < (1u << 26) && !ok; ++i) {
                __nanosleep(100);
                ok = there();
                if (!ok && global_ns() - t0 > wait_ns) break;
            }
        }
    }
    return __syncthreads_and(ok);
}

// The sequence's items, one after the other: sums(item, share, walked), which leaves a
// chunk's sums and calls walked() once it has read the chunk, join(item), true where
// that made a sample's results, and apply(item, share, ready), which calls ready()
// before it uses them and ends where that is false: its CTA then takes no further item
// and leaves none to the others, whose own waits, one each at most, end the same way.
// (Chunks applied in two parts, for
// a more even end, cost B1 S262144 C128 bf16 59 us instead of 52: an item's start and
// end are the dearer.)
template <typename Sums, typename Join, typename Apply>
__device__ __forceinline__ void gn_sequence(const GnArgs& a, const GnStreamWs& ws, unsigned* err,
                                            unsigned long long wait_ns, int stall, Sums sums, Join join,
                                            Apply apply) {
    __shared__ unsigned word[2];
    const int t = threadIdx.x;
    grid_wait();
    if (t == 0) word[0] = atomicAdd(ws.next, 1u);
    __syncthreads();
    const unsigned items = 2u * unsigned(a.B) * unsigned(a.chunks);
    for (unsigned i = word[0]; i < items;) {
        // the next one while this one is worked on; where a CTA has only a few, which
        // would keep a second one from a CTA that has none, while its sums are joined
        unsigned after = 0;
        if (t == 0 && a.early) after = atomicAdd(ws.next, 1u);
        const GnItem it(i, a);
        const GnShare k(a, it);
        if (it.apply) {
            bool there = true;
            apply(it, k, [&] { return there = gn_ready(&ws.done[it.sample], wait_ns); });
            if (!there) {
                if (t == 0) {
                    atomicExch(ws.next, items);
                    atomicExch(err, kDeviceErrTimeout);
                }
                return;
            }
        } else {
            sums(it, k, [&] {
                if (t == 0 && !a.early) after = atomicAdd(ws.next, 1u);
            });
            if (join(it, &word[1]) && t == 0 && it.sample != stall) {
                __threadfence();
                atomicExch(&ws.done[it.sample], kGnThere);
            }
        }
        if (t == 0 && !a.early && it.apply) after = atomicAdd(ws.next, 1u);
        __syncthreads();
        if (t == 0) word[0] = after;
        __syncthreads();
        i = word[0];
    }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock, 3)
    gn_stream_kernel(const T* x, T* y, const T* w, const T* b, float2* stats_out, const __grid_constant__ GnStreamWs ws,
                     const __grid_constant__ GnArgs a, unsigned* err, unsigned long long wait_ns, int stall) {
    using V = Vec<T, VEC>;
    constexpr int P = V::P, D = kGnStreamDepth;
    extern __shared__ __align__(16) uint4 slots[];  // the positions on their way, then:
    const int W = a.tx * VEC;
    float* pm = reinterpret_cast<float*>(slots) + walk_smem<T, VEC, D, 1>() / 4;  // [ty][W] the threads' means
    float* pq = pm + a.ty * W;                               // [ty][W] and squares
    float2* col = reinterpret_cast<float2*>(pq + a.ty * W);  // [C] the channels'
    float* refs = reinterpret_cast<float*>(col + a.C);       // [G] what the means are kept less of
    auto sums = [&](const GnItem& it, const GnShare& k, auto walked) {
        const float inv_rows = 1.f / float(k.rows);
        for (int tile = 0; tile < a.tiles; ++tile) {
            const int c0 = tile * W, c = c0 + k.tx * VEC;
            Shifted<P> s;
            s.clear();
            const bool mine = k.n > 0 && c < a.C;
            const T* const from[1] = {x + (mine ? k.first + c : 0)};
            bool first = true;
            Walk<T, VEC, D, 1, false> walk(from, k.step, mine ? k.n : 0, slots);
            if (tile == 0) {  // while the first copies are on their way
                const T* origin = x + it.sample * a.S * a.ld;
                for (int g = threadIdx.x; g < a.G; g += kGnBlock) refs[g] = Elem<T>::load(origin + g * a.L);
                __syncthreads();
            }
            walk.run([&](const typename V::Word (&wd)[1]) {
                float2 v[P];
                V::get(wd[0], v);
                if (first) s.start(v);
                first = false;
                s.add(v);
            });
            if (tile == a.tiles - 1) walked();
            if (k.ty < a.ty)
                s.template leave<VEC>(c < a.C ? k.n : 0, Groups<VEC>(c < a.C ? c : 0, a), refs,
                                      pm + k.ty * W + k.tx * VEC, pq + k.ty * W + k.tx * VEC);
            __syncthreads();
            const int each = k.rows / a.ty, more = k.rows - each * a.ty;  // positions of row r: each + (r < more)
            by_teams(min(W, a.C - c0), a.parts_log2, [&](int ch, int lane, bool live) {
                const float ref = pm[ch];
                float2 s2 = f2(0.f);
                for (int r = lane; r < a.ty; r += 1 << a.parts_log2) {
                    const float m = float(each + (r < more)), d = pm[r * W + ch] - ref;
                    s2.x = fmaf(m, d, s2.x);
                    s2.y += fmaf(m * d, d, pq[r * W + ch]);
                }
                s2 = lanes_sum(s2, 1 << a.parts_log2);
                if (live && lane == 0) col[c0 + ch] = joined(ref, s2, 1.f, inv_rows);
            });
            __syncthreads();
        }
        float2* out = ws.part + (int64_t(it.sample) * a.chunks + it.chunk) * a.G;
        by_teams(a.G, a.team_log2, [&](int g, int lane, bool live) {
            const float2* cg_ = col + g * a.L;
            const float ref = cg_[0].x, m = float(k.rows);
            float2 s = f2(0.f);
            for (int i = lane; i < a.L; i += 1 << a.team_log2) {
                const float d = cg_[i].x - ref;
                s.x += d;
                s.y += fmaf(m * d, d, cg_[i].y);
            }
            s = lanes_sum(s, 1 << a.team_log2);
            if (live && lane == 0) out[g] = joined(ref, s, m, a.inv_L);
        });
    };
    auto join = [&](const GnItem& it, unsigned* word) { return gn_joined<true>(it, a, ws, x, stats_out, word); };
    auto apply = [&](const GnItem& it, const GnShare& k, auto ready) {
        for (int tile = 0; tile < a.tiles; ++tile) {
            const int c = (tile * a.tx + k.tx) * VEC;
            const bool mine = k.n > 0 && c < a.C;
            const int64_t at = mine ? k.first + c : 0;
            const T* const from[1] = {x + at};
            Walk<T, VEC, D, 1, true> walk(from, k.step, mine ? k.n : 0, slots);
            float2 mean[P], mul[P], add[P], rstd[P];
            load_affine<T, VEC>(w, mine ? c : 0, 1.f, mul);
            load_affine<T, VEC>(b, mine ? c : 0, 0.f, add);
            if (tile == 0 && !ready()) return walk.drop();
            if (!mine) continue;
            const Groups<VEC> g(c, a);
            // past L1: another SM wrote them during this kernel
            const float2* res = ws.result + int64_t(it.sample) * a.G;
            each_channel<VEC>(mean, [&](int e) { return -__ldcg(&res[g.g[e]]).x; });
            each_channel<VEC>(rstd, [&](int e) { return __ldcg(&res[g.g[e]]).y; });
#pragma unroll
            for (int j = 0; j < P; ++j) mul[j] = f2_mul(mul[j], rstd[j]);
            T* py = y + at;
            walk.run([&](const typename V::Word (&wd)[1]) {
                float2 v[P];
                V::get(wd[0], v);
#pragma unroll
                for (int j = 0; j < P; ++j) v[j] = act_of2<ACT>(f2_fma(f2_add(v[j], mean[j]), mul[j], add[j]));
                V::put(py, v);
                py += k.step;
            });
        }
    };
    gn_sequence(a, ws, err, wait_ns, stall, sums, join, apply);
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnBlock, 2)
    gn_bwd_stream_kernel(const T* x, const T* dy, T* dx, const T* w, const T* b, const float2* stats,
                         const __grid_constant__ GnStreamWs ws, const __grid_constant__ GnArgs a, unsigned* err,
                         unsigned long long wait_ns, int stall) {
    using E = Elem<T>;
    using V = Vec<T, VEC>;
    constexpr int P = V::P, D = kGnStreamDepthBwd;
    extern __shared__ __align__(16) uint4 slots[];  // the positions on their way, then:
    const int W = a.tx * VEC;
    float2* red = reinterpret_cast<float2*>(slots) + walk_smem<T, VEC, D, 2>() / 8;  // [ty][W] the threads' A, Q
    float2* col = red + a.ty * W;  // [C] the channels', times w
    let_next_start();
    auto sums = [&](const GnItem& it, const GnShare& k, auto walked) {
        const int64_t slot = int64_t(it.sample) * a.chunks + it.chunk;
        float* cw = ws.chans + slot * 2 * a.C;
        for (int tile = 0; tile < a.tiles; ++tile) {
            const int c0 = tile * W, c = c0 + k.tx * VEC;
            GnSlope<T, VEC, ACT> slope;
            float2 sa[P], sq[P];
#pragma unroll
            for (int j = 0; j < P; ++j) sa[j] = sq[j] = slope.rstd[j] = f2(0.f);
            if (k.n > 0 && c < a.C) {
                const T* const from[2] = {x + k.first + c, dy + k.first + c};
                Walk<T, VEC, D, 2, false> walk(from, k.step, k.n, slots);
                slope.load(w, b, stats + int64_t(it.sample) * a.G, c, c, a);
                walk.run([&](const typename V::Word (&wd)[2]) { slope.add(wd[0], wd[1], sa, sq); });
            }
            if (tile == a.tiles - 1) walked();
            if (k.ty < a.ty) slope.leave(sa, sq, red + k.ty * W + k.tx * VEC);
            __syncthreads();
            by_teams(min(W, a.C - c0), a.parts_log2, [&](int ch, int lane, bool live) {
                float2 s = f2(0.f);
                for (int r = lane; r < a.ty; r += 1 << a.parts_log2) s = f2_add(s, red[r * W + ch]);
                s = lanes_sum(s, 1 << a.parts_log2);
                if (live && lane == 0) {
                    cw[c0 + ch] = s.y;
                    cw[a.C + c0 + ch] = s.x;
                    const float wv = w ? E::load(w + c0 + ch) : 1.f;
                    col[c0 + ch] = make_float2(wv * s.x, wv * s.y);
                }
            });
            __syncthreads();
        }
        by_teams(a.G, a.team_log2, [&](int g, int lane, bool live) {
            float2 s = f2(0.f);
            for (int i = lane; i < a.L; i += 1 << a.team_log2) s = f2_add(s, col[g * a.L + i]);
            s = lanes_sum(s, 1 << a.team_log2);
            if (live && lane == 0) ws.part[slot * a.G + g] = s;
        });
    };
    auto join = [&](const GnItem& it, unsigned* word) { return gn_joined<false>(it, a, ws, x, nullptr, word); };
    auto apply = [&](const GnItem& it, const GnShare& k, auto ready) {
        for (int tile = 0; tile < a.tiles; ++tile) {
            const int c = (tile * a.tx + k.tx) * VEC;
            const bool mine = k.n > 0 && c < a.C;
            const int64_t at = mine ? k.first + c : 0;
            const T* const from[2] = {x + at, dy + at};
            Walk<T, VEC, D, 2, true> walk(from, k.step, mine ? k.n : 0, slots);
            GnSlope<T, VEC, ACT> slope;
            slope.load(w, b, stats + int64_t(it.sample) * a.G, mine ? c : 0, mine ? c : 0, a);
            if (tile == 0 && !ready()) return walk.drop();
            if (!mine) continue;
            // past L1: another SM wrote them during this kernel
            const float2* res = ws.result + int64_t(it.sample) * a.G;
            slope.means([&](int g) { return __ldcg(&res[g]); }, c, a);
            T* po = dx + at;
            walk.run([&](const typename V::Word (&wd)[2]) {
                float2 v[P];
                slope.of(wd[0], wd[1], v);
                V::put(po, v);
                po += k.step;
            });
        }
    };
    gn_sequence(a, ws, err, wait_ns, stall, sums, join, apply);
}

// ---- launchers -------------------------------------------------------------
// A launch that may start while the one before it drains: every kernel here waits
// for that one before it touches memory.
inline cudaError_t gn_launch(const void* kern, int grid, int block, size_t smem, const LaunchCfg& cfg, void** args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(unsigned(grid));
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

// Channel vectors side by side: in equal tiles of a row (of 128 bytes or more), which a
// CTA takes one after the other. A further tile is worth its start and end, taken as an
// eighth, where it puts more threads to work: 135 vectors side by side leave 121 of
// 256 threads idle, three tiles of 45 have 225 at work.
inline void gn_tiles(GnArgs& a, int vec, int es) {
    auto log2_floor = [](int v) {
        int l = 0;
        while (v > 1) v >>= 1, ++l;
        return l;
    };
    const int nv = (a.C + vec - 1) / vec, least = (nv + kGnBlock - 1) / kGnBlock;
    double best = 0.0;
    for (int tiles = least; tiles <= least + 3; ++tiles) {
        const int tx = (nv + tiles - 1) / tiles;
        if (tiles > least && tx * vec * es < 128) break;
        const double use = double(nv) / tiles * (kGnBlock / tx) / kGnBlock * (1.0 - 0.125 * (tiles - least));
        if (use > best) {
            best = use;
            a.tiles = tiles;
            a.tx = tx;
        }
    }
    a.ty = kGnBlock / a.tx;
    a.inv_tx = (65536 + a.tx - 1) / a.tx;
    a.parts_log2 = std::min(5, log2_floor(std::max(1, std::min(kGnBlock / (a.tx * vec), a.ty))));
    a.last_log2 = std::min(5, log2_floor(kGnBlock / std::min(kGnBlock, a.G)));
    a.team_log2 = std::min(a.last_log2, log2_floor(2 * a.L - 1));
}

// Lays out the workspace, zeroes its counters and launches the kernel.
inline cudaError_t gn_stream_launch(const void* kern, GnArgs& a, GnStreamWs& ws, void* workspace, int vec, size_t smem,
                                    bool backward, void** args, const LaunchCfg& cfg) {
    cudaError_t e = allow_smem(kern, smem, cfg);
    if (e != cudaSuccess) return e;
    const int64_t N = int64_t(a.B) * a.chunks;
    const int grid = grid_for(kern, kGnBlock, smem, 2 * N, cfg);
    a.lag = int(std::min<int64_t>(N, int64_t(a.chunks) + grid));
    a.early = 2 * N >= 8 * int64_t(grid);
    char* p = static_cast<char*>(workspace);
    ws.next = reinterpret_cast<unsigned*>(p);
    ws.done = ws.next + 1;
    ws.bunch_done = ws.done + a.B;
    p += gn_counter_bytes(a);
    ws.result = reinterpret_cast<float2*>(p);
    ws.part = ws.result + int64_t(a.B) * a.G;
    ws.bunch = ws.part + N * a.G;
    if (backward) ws.chans = reinterpret_cast<float*>(ws.bunch + gn_bunches(a) * a.G);
    unsigned* counters = ws.next;
    int64_t n = 1 + a.B + gn_bunches(a);
    void* zero_args[] = {&counters, &n};
    e = gn_launch(reinterpret_cast<const void*>(gn_zero_kernel), 1, 1024, 0, cfg, zero_args);
    return e == cudaSuccess ? gn_launch(kern, grid, kGnBlock, smem, cfg, args) : e;
}

template <typename T, int VEC, int ACT>
cudaError_t gn_forward_stream(const void* x, void* y, const void* w, const void* b, float* stats, void* workspace,
                              GnArgs a, const LaunchCfg& cfg) {
    gn_tiles(a, VEC, int(sizeof(T)));
    GnStreamWs ws{};
    unsigned* err = cfg.dev_error;
    unsigned long long wait_ns = cfg.wait_ns;
    int stall = cfg.stall_row < 0 ? -1 : int(cfg.stall_row / a.S);
    void* args[] = {&x, &y, &w, &b, &stats, &ws, &a, &err, &wait_ns, &stall};
    return gn_stream_launch(reinterpret_cast<const void*>(gn_stream_kernel<T, VEC, ACT>), a, ws, workspace, VEC,
                            walk_smem<T, VEC, kGnStreamDepth, 1>() + 8 * (size_t(a.ty) * a.tx * VEC + a.C) + 4 * size_t(a.G),
                            false, args,
                            cfg);
}

template <typename T, int VEC, int ACT>
cudaError_t gn_backward_stream(const void* x, const void* dy, const void* w, const void* b, const float* stats,
                               void* dx, float* dw, float* db, void* workspace, GnArgs a, const LaunchCfg& cfg) {
    gn_tiles(a, VEC, int(sizeof(T)));
    GnStreamWs ws{};
    unsigned* err = cfg.dev_error;
    unsigned long long wait_ns = cfg.wait_ns;
    int stall = cfg.stall_row < 0 ? -1 : int(cfg.stall_row / a.S);
    void* args[] = {&x, &dy, &dx, &w, &b, &stats, &ws, &a, &err, &wait_ns, &stall};
    const cudaError_t e =
        gn_stream_launch(reinterpret_cast<const void*>(gn_bwd_stream_kernel<T, VEC, ACT>), a, ws, workspace, VEC,
                         walk_smem<T, VEC, kGnStreamDepthBwd, 2>() + 8 * (size_t(a.ty) * a.tx * VEC + a.C), true, args,
                         cfg);
    return e == cudaSuccess ? gn_reduce_channels(ws.chans, int64_t(a.B) * a.chunks, a.C, dw, db, cfg) : e;
}

}  // namespace rowops
