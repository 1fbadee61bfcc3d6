// Joining the parts of rows whose keys were cut evenly (EvenSplit), or in pieces.
#pragma once

#include <algorithm>

#include "attention_paged.h"

namespace sg {

// One wavefront per token and `each` query heads joins their parts, in their order, so that
// the bits are the same every time. A chain of loads (6 to 10 us for few rows): where the text and
// its range are, the parts' maxima and sums, then the parts, four at a time. Parts of
// ranges lie as [slot][key head][tile][row of tile_rows], of pieces as PagedArgs
// has it; their weights are held times 2^shift.
template <class T, int SEQS, bool ONE>
__global__ __launch_bounds__(4 * kWave) void k_join_parts(PagedArgs a, int32_t tiles,
                                                          int32_t tile_rows, int32_t keys,
                                                          float shift, int32_t heads) {
    const int each = ONE ? 1 : heads;  // (known to be one it takes fewer registers)
    const int groups = (a.s.hq + each - 1) / each;
    const int64_t group = grid_block() * 4 + threadIdx.x / kWave;
    if (group >= a.tokens * groups) return;
    const int64_t token = group / groups;
    const int hq0 = (int)(group - token * groups) * each;
    Sequence sq;
    int64_t s = upper_index(a.q_rowptr, int64_t(0), a.seqs, token);
    if (!find_sequence(a, token, s, sq) || sq.bad) return;
    const int sees = sq.length - sq.fresh + 1 + (int)(token - sq.q0);
    int count, range = 0;
    int64_t step, late = 0;  // in rows of parts
    if (a.ranges) {
        const EvenParts parts(EvenSplit<SEQS>(a, keys), __builtin_amdgcn_readfirstlane((int)s), keys,
                              sees);
        count = parts.count;
        range = parts.range;
        const int64_t slot = (int64_t)a.s.hkv * tiles * tile_rows;
        step = 2 * slot;
        late = parts.late ? slot : 0;
    } else {
        count = sees <= a.piece ? 0 : (sees + a.piece - 1) / a.piece;
        step = a.tokens * a.s.hq;
    }
    if (count == 0) return;
#pragma unroll 1
    for (int hq = hq0; hq < min(hq0 + each, a.s.hq); ++hq) {
        const int64_t unit = token * a.s.hq + hq;
        int64_t first = unit;
        if (a.ranges) {
            const int h = hq / a.s.group;
            const int row = (int)(token - sq.q0) * a.s.group + hq - h * a.s.group, tile = row / tile_rows;
            first = range * step + ((int64_t)h * tiles + tile) * tile_rows + row - tile * tile_rows;
        }
        const auto at = [&](int i) { return first + i * step + (i == 0 ? late : 0); };
        float m = -INFINITY, l = 0.f;
        for (int i = lane_id(); i < count; i += kWave) m = fmaxf(m, a.part_ml[2 * at(i)]);
#pragma unroll
        for (int d = kWave / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
        m = m == -INFINITY ? 0.f : m;
        for (int i = lane_id(); i < count; i += kWave)
            l += a.part_ml[2 * at(i) + 1] * fast_exp2(a.part_ml[2 * at(i)] - m);
        l = wave_reduce_sum(l);
        const float f = l == 0.f ? 0.f : 1.f / l;
        char* row = a.out.base + token * a.out.row + hq * a.out.head;
        for (int d = 4 * lane_id(); d < a.s.dim; d += 4 * kWave) {
            f32x4 x{0, 0, 0, 0};
#pragma unroll 4
            for (int i = 0; i < count; ++i)
                x += *reinterpret_cast<const f32x4*>(a.part + at(i) * a.s.dim + d) *
                     fast_exp2(a.part_ml[2 * at(i)] - m);
            x *= f;
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<u32x2*>(row + 2 * d) = u32x2{pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3])};
            else
                *reinterpret_cast<f32x4*>(row + 4 * d) = x;
        }
        if (a.lse && lane_id() == 0)
            a.lse[unit] = l == 0.f ? -INFINITY : (m - shift + fast_log2(l)) * kLn2;
    }
}

template <class T, int SEQS>
void join_parts(const PagedArgs& a, int32_t tiles, int32_t tile_rows, int32_t keys, float shift,
                hipStream_t st) {
    // Rows that are not cut leave after the first half of that chain. Of many rows most
    // are not, and the fewer wavefronts look: the absorbed form of 1000 texts up to 4096,
    // 128 heads, takes 1076 us with 7 heads each, 1272 with one. Those that are cut then
    // follow each other: 200 texts, one of them 64 times the others' length, 188 us with 8
    // heads, 140 with one.
    const int32_t each = (int32_t)std::min<int64_t>(std::max<int64_t>(a.tokens * a.s.hq / 16384, 1), 8);
    const auto run = each == 1 ? k_join_parts<T, SEQS, true> : k_join_parts<T, SEQS, false>;
    hipLaunchKernelGGL(run, grid_2d(ceil_div(a.tokens * ceil_div(a.s.hq, each), 4)), dim3(4 * kWave), 0,
                       st, a, tiles, tile_rows, keys, shift, each);
    SG_LAUNCH_CHECK();
}

}  // namespace sg
