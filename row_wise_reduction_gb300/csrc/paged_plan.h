// Shapes and forms of the attention over a paged cache (paged_kernels.cuh): what a CTA needs
// of an SM, how many share one, and which form a call takes. Pure host arithmetic (no CUDA
// call), so that it is tested on the CPU.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace rowops {

constexpr int kPagedMaxD = 256;
constexpr int kPagedWarps = 4;

// At most kPagedMaxCtas CTAs (three a SM), each of which leaves two parts: for a block of heads their
// weighted values, a maximum and a sum each, D rounded up to one of the kernels' widths.
constexpr int kPagedMaxCtas = 3 * 152;
constexpr int kPagedWidths[] = {64, 80, 96, 128, 160, 192, 256};
inline int paged_width(int64_t D) {
    for (int w : kPagedWidths)
        if (D <= w) return w;
    return 0;
}
inline int paged_rows(int64_t group, int es) { return es == 2 ? (group > 8 ? 16 : 8) : group > 4 ? 8 : group > 1 ? 4 : 1; }

// What an SM has of shared memory for its CTAs, and what the system keeps of it for each.
constexpr int kSmShared = 228 * 1024, kCtaReserved = 1024;

// A CTA's shared memory and how many CTAs share an SM, for elements of `es` bytes, heads of `width` and
// blocks of `rows` heads.
struct PagedShape {
    int tokens;   // positions of a warp's piece
    int pitch;    // bytes from a position's row to the next: an odd number of 16-byte vectors, so eight rows' vectors
                  // lie in different banks
    int step;     // bytes of one step of all warps' rings: keys, then values
    int joined;   // floats from a head's row of the joined values to the next
    int scratch;  // bytes of the form's own: queries, and fp32's weights
    int fixed;    // bytes beside the rings: joined rows, scratch, static arrays (at most), the system's
    int ctas, stages;
};
// As many steps (6 at most) as let three CTAs share an SM, if those are two and the registers allow it (rows at most
// 8), else two CTAs, else three steps in one; of what all else leaves, and no more than 72000 and 104448 bytes. Three for
// two: D 64, heads before slots, 64 sequences of up to 8192, bf16 131 to 110 us, fp32 268 to 213; D 128 186 to 182.
// fp32 in two CTAs: two steps (8 heads of 128 have room for a third; with it 64 heads over 8, 16 sequences of
// up to 4096, 94.1 to 95.1 us, 8 over 1, one of 32768, 36.3 to 39.1).
constexpr PagedShape paged_shape(int es, int width, int rows) {
    PagedShape s = {};
    s.tokens = es == 2 ? 16 : 8;
    s.pitch = (width * es / 16 | 1) * 16;
    s.step = 2 * s.tokens * s.pitch * kPagedWarps;
    s.joined = es == 2 ? width + 4 : width;
    // bf16: long heads' queries; fp32: queries, and each warp's weights and factors
    s.scratch = es == 2 ? (width * rows < 2560 ? 0 : width * rows * 2) : rows * width * 4 + kPagedWarps * rows * 9 * 4 + 16;
    s.fixed = rows * s.joined * 4 + s.scratch + 40 * rows + 64 + kCtaReserved;
    const int three = std::min(72000, kSmShared / 3 - s.fixed) / s.step;
    const int two = std::min(104448, kSmShared / 2 - s.fixed) / s.step;
    s.ctas = rows <= 8 && three >= 2 ? 3 : two >= 2 ? 2 : 1;
    s.stages = s.ctas == 1 ? 3 : s.ctas == 3 ? std::min(6, three) : es == 4 ? 2 : std::min(6, two);
    return s;
}

constexpr int kPagedCluster = 8;
// Clusters of this many CTAs, one a unit (0: the line of tiles, with parts in the workspace); the most tiles that
// the sequences can have.
struct PagedForm {
    int cluster;
    int64_t tiles;
};
// One cluster a unit, where all fit on the GPU at once (two CTAs an SM at most), saves the second launch and the parts'
// way through memory; the line shares the tiles out evenly. In times of a tile (of 64 positions in bf16, 32 in fp32), by
// the table's room: a cluster's share of its unit against the line's share and eight more. 32 heads over 8, D 128, one
// sequence, clusters and line: room for 512 7.7 and 10.1 us, 4096 14.9 and 15.4, 8192 24.0 and 17.9.
inline PagedForm paged_form(int64_t B, int64_t heads, int64_t kv_heads, int64_t D, int64_t room, int64_t window, int es) {
    const int64_t rows = paged_rows(heads / kv_heads, es), units = B * kv_heads * ((heads / kv_heads + rows - 1) / rows);
    const int64_t tile = es == 2 ? 64 : 32, most = window > 0 && window < room ? std::min(room, window + 15) : room;
    const int64_t each = (most + tile - 1) / tile, slots = 152 * std::min(2, paged_shape(es, paged_width(D), int(rows)).ctas);
    PagedForm f = {0, std::min<int64_t>(each, 1 << 20) * units};
    int C = kPagedCluster;
    while (C > 1 && (units * C > slots || C >= 2 * each)) C /= 2;
    if (units * C <= slots && (each + C - 1) / C <= each * units / slots + 8) f.cluster = C;
    return f;
}
inline size_t paged_bytes(int64_t B, int64_t heads, int64_t kv_heads, int64_t D, int64_t room, int64_t window, int es) {
    if (paged_form(B, heads, kv_heads, D, room, window, es).cluster) return 0;
    return size_t(kPagedMaxCtas) * 2 * ((paged_rows(heads / kv_heads, es) * (paged_width(D) + 2) + 3) / 4 * 4) * 4;
}

}  // namespace rowops
