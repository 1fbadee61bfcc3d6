// What kernels over a paged cache share: the batch's sequences, read and
// checked on the device, their tiles of rows, and how a row's result leaves.
#pragma once

#include "attention.h"

namespace sg {

// One sequence of the batch, checked where it is read.
struct Sequence {
    int64_t q0;      // its first new token's row
    int32_t fresh;   // new tokens, at most max_new
    int32_t length;  // cached tokens
    int64_t page0;   // its first page's entry
    bool bad;        // breaks the batch's rules
    bool none;       // has no rows to write
};
__device__ __forceinline__ Sequence read_sequence(const PagedArgs& a, int64_t s) {
    const int64_t q0 = a.q_rowptr[s], q1 = a.q_rowptr[s + 1];
    const int64_t p0 = a.rowptr[s], p1 = a.rowptr[s + 1], len = a.lengths[s];
    Sequence x;
    x.q0 = q0;
    x.none = q1 <= q0 || q0 < 0 || q0 >= a.tokens;
    const bool pages_ok = p0 >= 0 && p1 >= p0 && p1 <= a.room;
    // (p1 - p0 < 2^31 and the page size < 2^31, so the product fits)
    x.bad = q1 > a.tokens || q1 - q0 > a.max_new || len < q1 - q0 || len > a.max_length ||
            !pages_ok || (p1 - p0) * (int64_t)a.page_div.d < len || a.npages == 0;
    x.fresh = (int32_t)min(min(q1, a.tokens) - q0, (int64_t)a.max_new);
    x.length = x.bad ? 0 : (int32_t)len;
    x.page0 = p0;
    return x;
}

// The sequence s that has `token` (the same in all lanes) among its new ones, and
// whether there is one; by a whole wavefront. s: what a search of ascending starts finds.
// A broken sequence's start may be out of order and mislead that search, so where it
// finds none whose starts fit, all are looked at, 64 at a time, and one whose starts fit
// goes before one that has too many new tokens: rows of no sequence pay for that.
__device__ __forceinline__ bool find_sequence(const PagedArgs& a, int64_t token, int64_t& s,
                                              Sequence& sq) {
    const auto has = [&](int64_t q0, int64_t q1) {
        return q0 >= 0 && q0 <= token && token < min(q1, q0 + a.max_new);
    };
    const auto fits = [&](int64_t q0, int64_t q1) { return q1 <= a.tokens && q1 - q0 <= a.max_new; };
    const int64_t q0 = a.q_rowptr[s], q1 = a.q_rowptr[s + 1];
    if (!has(q0, q1) || !fits(q0, q1)) {
        s = -1;
#pragma unroll 1
        for (int64_t first = 0; first < a.seqs; first += kWave) {
            const int64_t i = min(first + lane_id(), a.seqs - 1), x0 = a.q_rowptr[i], x1 = a.q_rowptr[i + 1];
            const uint64_t any = __ballot(has(x0, x1)), best = __ballot(has(x0, x1) && fits(x0, x1));
            if (best || (any && s < 0)) s = first + __builtin_ctzll(best ? best : any);
            if (best) break;
        }
        if (s < 0) return false;
    }
    sq = read_sequence(a, s);
    return true;
}

// What a work group or wavefront has to do for a tile of `rows` rows of one
// sequence (its new tokens' query heads of one key head, the heads of a token
// next to each other) and one piece of its keys.
struct TileJob {
    Sequence sq;
    int rows;    // of the whole sequence
    int first;   // the tile's first row
    int before;  // keys that the sequence's first new token sees
    int k0, k1;  // the keys
    bool idle;
};
__device__ __forceinline__ TileJob tile_job(const PagedArgs& a, int64_t s, int tile, int tile_rows,
                                            int piece) {
    TileJob j;
    j.sq = read_sequence(a, s);
    j.rows = j.sq.fresh * a.s.group;
    j.first = tile * tile_rows;
    j.idle = j.sq.none || j.first >= j.rows;
    j.before = j.sq.length - j.sq.fresh + 1;
    const int last = min(j.first + tile_rows, j.rows) - 1;
    j.k0 = piece * a.piece;
    j.k1 = min(j.k0 + a.piece, j.before + last / a.s.group);
    return j;
}

// One row of a tile: its new token (of the sequence) and query head.
struct TileRow {
    bool has;
    int t, hq;
    int64_t token;
};
__device__ __forceinline__ TileRow tile_row(const PagedArgs& a, const TileJob& j, int row, int h) {
    TileRow r;
    r.has = row < j.rows;
    const int x = min(row, j.rows - 1);
    r.t = (int)a.group_div.div(x);
    r.hq = h * a.s.group + x - r.t * a.s.group;
    r.token = j.sq.q0 + r.t;
    return r;
}

// NaN for one row of a sequence that breaks the rules, by the four lanes that
// share it.
template <class T>
__device__ __forceinline__ void store_nan(const PagedArgs& a, const TileRow& r) {
    if (!r.has) return;
    T* out = reinterpret_cast<T*>(a.out.base + r.token * a.out.row + r.hq * a.out.head);
    for (int d = lane_id() >> 4; d < a.s.dim; d += 4) out[d] = (T)NAN;
    if (a.lse && lane_id() < 16) a.lse[r.token * a.s.hq + r.hq] = NAN;
}

// A row's result, finished if the first piece holds all keys that it sees,
// otherwise as this piece's part of it.
template <class G, class T>
__device__ __forceinline__ void store_values(const typename G::Acc& o, float f, bool part,
                                             char* at, int dim) {
#pragma unroll
    for (int u = 0; u < G::U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (part)
                G::store_part(o, u, i, f, reinterpret_cast<float*>(at), dim);
            else
                G::store_out(o, u, i, f, at, dim * (int)sizeof(T));
        }
}
template <class G, class T>
__device__ __forceinline__ void store_values(const typename G::AccB& o, float f, bool part,
                                             char* at, int dim) {
#pragma unroll
    for (int b = 0; b < G::NB; ++b) {
        const int d = 16 * b + 4 * (lane_id() >> 4);
        if (!G::kFull && d >= dim) continue;
        if (part)
            *reinterpret_cast<f32x4*>(at + 4 * d) = o.o[b] * f;
        else
            G::store_four(o.o[b] * f, at + d * (int)sizeof(T));
    }
}
// at: where it goes as a part
template <class G, class T, class A>
__device__ __forceinline__ void store_row_at(const PagedArgs& a, const TileRow& r, bool whole,
                                             int64_t at, const A& o, const Softmax<G, T>& sm) {
    if (whole) {
        store_values<G, T>(o, sm.factor(), false,
                           a.out.base + r.token * a.out.row + r.hq * a.out.head, a.s.dim);
        if (a.lse && lane_id() < 16) a.lse[r.token * a.s.hq + r.hq] = sm.lse();
    } else {
        store_values<G, T>(o, 1.f, true, reinterpret_cast<char*>(a.part + at * a.s.dim), a.s.dim);
        if (lane_id() < 16) {
            a.part_ml[2 * at] = sm.m;
            a.part_ml[2 * at + 1] = sm.l;
        }
    }
}
template <class G, class T, class A>
__device__ __forceinline__ void store_row(const PagedArgs& a, const TileJob& j, const TileRow& r,
                                          int piece, const A& o, const Softmax<G, T>& sm) {
    const int sees = j.before + r.t;
    if (!r.has || sees <= j.k0) return;
    store_row_at<G, T>(a, r, sees <= a.piece,
                       (int64_t)piece * a.tokens * a.s.hq + r.token * a.s.hq + r.hq, o, sm);
}

// A batch's tiles of `keys` keys, one sequence after another, cut into ranges of
// one length: wavefronts or work groups that take a range each end together,
// whatever the texts' lengths. A sequence's part of a range is a segment; the
// segments of a sequence that lies in several ranges are joined. Range i leaves
// such a part in slot 2 i if the range begins with it, else in 2 i + 1. By a whole
// wavefront; up to SEQS sequences of less than 2^31 tiles.
template <int SEQS>
struct EvenSplit {
    static constexpr int kEach = SEQS / kWave;
    int n[kEach];  // tiles of sequences lane, 64 + lane, ...
    int total = 0, per;
    __device__ __forceinline__ EvenSplit(const PagedArgs& a, int keys) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) n[i] = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (i * kWave >= a.seqs) break;
            const int64_t s = i * kWave + lane_id();
            if (s < a.seqs) {
                const Sequence sq = read_sequence(a, s);
                n[i] = sq.none ? 0 : sq.bad ? 1 : (sq.length + keys - 1) / keys;
            }
            total += last(wave_inclusive_scan_i32(n[i]));
        }
        per = max((total + a.ranges - 1) / a.ranges, 1);
    }
    static __device__ __forceinline__ int last(int x) { return __builtin_amdgcn_readlane(x, kWave - 1); }
    // The sequence that tile `pos` < total is of, and the tiles before it.
    __device__ __forceinline__ void locate(int pos, int& s, int& before) const {
        before = s = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int in = wave_inclusive_scan_i32(n[i]);
            const uint64_t past = __ballot(before + in > pos);
            if (past) {
                const int l = __builtin_ctzll(past);
                s = i * kWave + l;
                before += __builtin_amdgcn_readlane(in - n[i], l);
                return;
            }
            before += last(in);
        }
    }
    // The tiles before sequence s (the same in all lanes), and its own.
    __device__ __forceinline__ void sequence(int s, int& before, int& own) const {
        before = own = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (s < i * kWave) break;
            const int in = wave_inclusive_scan_i32(n[i]);
            if (s >= (i + 1) * kWave) {
                before += last(in);
            } else {
                own = __builtin_amdgcn_readlane(n[i], s % kWave);
                before += __builtin_amdgcn_readlane(in, s % kWave) - own;
            }
        }
    }
};
// A row's parts under an even split: of `count` ranges (0: its result is whole) from
// `range` on, the first of which begins with the row's sequence or (late) with
// another one; only those that begin with a key that the row sees.
struct EvenParts {
    int range, count;
    bool late;
    template <int SEQS>
    __device__ __forceinline__ EvenParts(const EvenSplit<SEQS>& e, int s, int keys, int sees) {
        int before, own;
        e.sequence(s, before, own);
        range = before / e.per;
        late = before > range * e.per;
        const bool whole = (before + own - 1) / e.per == range;
        count = whole ? 0 : (before + (sees + keys - 1) / keys - 1) / e.per - range + 1;
    }
};

}  // namespace sg
