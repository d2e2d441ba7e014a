// Attention of one new token a sequence over a paged key-value cache:
//   s_j = scale q k_j;  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// over the positions j in [first, length) of the sequence; position j is slot
// j mod page of the page that the sequence's table names for j / page.
#include <algorithm>

#include "rowops_device.cuh"
#include "rowops_launch.h"

namespace rowops {
namespace {

constexpr int kBlock = 128;

// One CTA per sequence and head, tiles of as many positions as it has threads: a
// thread has the score of one position, then some columns of the output.
template <typename T>
__global__ void __launch_bounds__(kBlock) paged_attention_kernel(const PagedArgs a) {
    using E = Elem<T>;
    __shared__ float q[256], p[kBlock], red[4][kBlock / 32];
    __shared__ const T* rows[kBlock];
    const int b = blockIdx.x / a.heads, h = blockIdx.x % a.heads, kv = h / (a.heads / a.kv_heads);
    const T* qp = static_cast<const T*>(a.q) + b * a.ldq + int64_t(h) * a.D;
    for (int d = threadIdx.x; d < a.D; d += kBlock) q[d] = E::load(qp + d);
    const int64_t room = a.max_pages * a.page;
    const int64_t asked = a.lengths[b], n = asked < room ? (asked > 0 ? asked : 0) : room;
    const int64_t first = a.window > 0 && n > a.window ? n - a.window : 0;
    float m = -INFINITY, l = asked > room ? NAN : 0.f, acc[2] = {0.f, 0.f};
    int turn = 0;
    for (int64_t t0 = first; t0 < n; t0 += kBlock, turn ^= 2) {
        const int64_t t = t0 + threadIdx.x;
        float s = -INFINITY;
        const T* v = nullptr;
        __syncthreads();
        if (t < n) {
            const int64_t at = a.table[b * a.table_ld + t / a.page];
            if (at < 0 || at >= a.pages) {
                s = NAN;
            } else {
                const int64_t off = at * a.page_stride + (t % a.page) * a.slot_stride + kv * a.head_stride;
                const T* k = static_cast<const T*>(a.k) + off;
                v = static_cast<const T*>(a.v) + off;
                float dot = 0.f;
                for (int d = 0; d < a.D; ++d) dot = fmaf(q[d], E::load(k + d), dot);
                s = dot * a.scale;
            }
        }
        const float top = group_reduce<kBlock>(s, red[turn], OpMax());
        const float next = fmaxf(m, top), base = next == -INFINITY ? 0.f : next;
        const float keep = ex2_approx((m - base) * kLog2eF);
        p[threadIdx.x] = ex2_approx((s - base) * kLog2eF);
        rows[threadIdx.x] = v;
        l = l * keep + group_reduce<kBlock>(p[threadIdx.x], red[turn + 1], OpSum());
        m = next;
        const int count = int(n - t0 < kBlock ? n - t0 : kBlock);
        for (int i = 0; i < 2; ++i) {
            const int d = threadIdx.x + i * kBlock;
            acc[i] *= keep;
            if (d < a.D)
                for (int j = 0; j < count; ++j)
                    if (rows[j]) acc[i] = fmaf(p[j], E::load(rows[j] + d), acc[i]);
        }
    }
    T* out = static_cast<T*>(a.out) + b * a.ldo + int64_t(h) * a.D;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = 0; i < 2; ++i)
        if (threadIdx.x + i * kBlock < a.D) E::store(out + threadIdx.x + i * kBlock, acc[i] * inv);
    if (threadIdx.x == 0 && a.lse) a.lse[int64_t(b) * a.heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename T>
cudaError_t launch(const PagedArgs& a, void*, const LaunchCfg& cfg) {
    paged_attention_kernel<T><<<unsigned(a.B * a.heads), kBlock, 0, cfg.stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

PagedLaunch paged_attention_f32() { return launch<float>; }
PagedLaunch paged_attention_bf16() { return launch<bf16_t>; }

}  // namespace rowops
