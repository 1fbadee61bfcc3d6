// Joining the parts of rows whose keys were cut evenly (EvenSplit), or in pieces.
#pragma once

#include "attention_paged.h"

namespace sg {

// One wavefront per token and query head joins its parts, in their order, so that
// the bits are the same every time. A chain of loads (6 to 10 us for few rows): where the text and
// its range are, the parts' maxima and sums, then the parts, four at a time. Parts of
// ranges lie as [slot][key head][tile][row of tile_rows], of pieces as PagedArgs
// has it; their weights are held times 2^shift.
template <class T>
__global__ __launch_bounds__(4 * kWave) void k_join_parts(PagedArgs a, int32_t tiles,
                                                          int32_t tile_rows, int32_t keys,
                                                          float shift) {
    const int64_t unit = grid_block() * 4 + threadIdx.x / kWave;
    if (unit >= a.tokens * a.s.hq) return;
    const int64_t token = unit / a.s.hq;
    const int hq = (int)(unit - token * a.s.hq);
    Sequence sq;
    int64_t s = upper_index(a.q_rowptr, int64_t(0), a.seqs, token);
    if (!find_sequence(a, token, s, sq) || sq.bad) return;
    const int sees = sq.length - sq.fresh + 1 + (int)(token - sq.q0);
    int count;
    int64_t first, step, late = 0;  // in rows of parts
    if (a.ranges) {
        const EvenParts parts(EvenSplit(a, keys), __builtin_amdgcn_readfirstlane((int)s), keys, sees);
        const int h = hq / a.s.group;
        const int row = (int)(token - sq.q0) * a.s.group + hq - h * a.s.group, tile = row / tile_rows;
        count = parts.count;
        const int64_t slot = (int64_t)a.s.hkv * tiles * tile_rows;
        step = 2 * slot;
        first = parts.range * step + ((int64_t)h * tiles + tile) * tile_rows + row - tile * tile_rows;
        late = parts.late ? slot : 0;
    } else {
        count = sees <= a.piece ? 0 : (sees + a.piece - 1) / a.piece;
        step = a.tokens * a.s.hq;
        first = unit;
    }
    if (count == 0) return;
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

template <class T>
void join_parts(const PagedArgs& a, int32_t tiles, int32_t tile_rows, int32_t keys, float shift,
                hipStream_t st) {
    hipLaunchKernelGGL(k_join_parts<T>, grid_2d(ceil_div(a.tokens * a.s.hq, 4)), dim3(4 * kWave), 0,
                       st, a, tiles, tile_rows, keys, shift);
    SG_LAUNCH_CHECK();
}

}  // namespace sg
