// Attention of new tokens over a paged key/value cache.
#include "attention.h"

namespace sg {

namespace {

constexpr int kWaves = 4;

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

// One wavefront: 16 rows (neighbouring new tokens' query heads of one key
// head, the heads of a token next to each other) against one piece of the
// sequence's keys. A token whose keys all lie in the first piece is finished
// here; the others leave their pieces to k_paged_join.
template <class G, class T>
__global__ __launch_bounds__(kWaves* kWave) void k_paged(PagedArgs a, int32_t tiles) {
    const int lane = lane_id();
    int64_t unit = xcd_block() * kWaves + threadIdx.x / kWave;
    if (unit >= a.seqs * a.s.hkv * a.npieces * tiles) return;
    const int tile = (int)(unit % tiles);
    unit /= tiles;
    const int piece = (int)(unit % a.npieces);
    unit /= a.npieces;
    const int64_t s = unit % a.seqs;
    const int h = (int)(unit / a.seqs);

    const Sequence sq = read_sequence(a, s);
    if (sq.none) return;
    const int n = lane & 15;
    const int row_bytes = a.s.dim * (int)sizeof(T);
    const int first_row = 16 * tile;                 // of the sequence's fresh * group rows
    const int rows = sq.fresh * a.s.group;
    if (first_row >= rows) return;
    const int row = first_row + n;
    const bool has = row < rows;
    const int t = min(row, rows - 1) / a.s.group, g = min(row, rows - 1) - t * a.s.group;
    const int hq = h * a.s.group + g;
    const int64_t token = sq.q0 + t;
    char* out = a.out.base + token * a.out.row + hq * a.out.head;
    if (sq.bad) {
        if (piece == 0 && has) {
            for (int d = lane >> 4; d < a.s.dim; d += 4) reinterpret_cast<T*>(out)[d] = (T)NAN;
            if (a.lse && lane < 16) a.lse[token * a.s.hq + hq] = NAN;
        }
        return;
    }
    // keys this lane's token sees, and those that any row of the tile sees
    const int before = sq.length - sq.fresh + 1;
    const int sees = before + t;
    const int least = before + first_row / a.s.group;
    const int most = before + min(first_row + 15, rows - 1) / a.s.group;
    const int k0 = piece * a.piece;
    const int k1 = min(k0 + a.piece, most);
    if (k0 >= k1) return;

    typename G::RowFrag q;
    G::zero_row(q);
    if (has) G::load_row(a.q.base + token * a.q.row + hq * a.q.head, row_bytes, q);
    typename G::Acc o;
    G::zero_acc(o);
    float m = -INFINITY, l = 0.f;
    bool wrong = false;  // a page outside the cache
    const char* kb = a.k + h * a.k_head;
    const char* vb = a.v + h * a.v_head;
    const int32_t* pages = a.col + sq.page0;
    for (int t0 = k0; t0 < k1; t0 += G::KT) {
        const int left = k1 - t0;
        const uint32_t key = (uint32_t)(t0 + min(lane & (G::KT - 1), left - 1));
        const uint32_t pg = a.page_div.div(key), slot = key - pg * a.page_div.d;
        uint32_t id = (uint32_t)pages[pg];
        if (id >= (uint64_t)a.npages) {
            wrong = true;
            id = 0;
        }
        const uint32_t ko = id * a.k_page + slot * a.k_slot, vo = id * a.v_page + slot * a.v_slot;
        f32x4 sc[G::KSUB];
#pragma unroll
        for (int b = 0; b < G::KSUB; ++b) {
            const uint32_t off = __shfl(ko, 16 * b + n, kWave);
            typename G::RowFrag k;
            G::load_row(kb + ((uint64_t)off << a.k_shift), row_bytes, k);
            sc[b] = G::dot(k, q, f32x4{0, 0, 0, 0});
        }
        const int limit = min(left, sees - t0);
        float p[G::VK], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < G::VK; ++j) {
            p[j] = G::key_of(j) < limit ? sc[j >> 2][j & 3] * a.s.c : -INFINITY;
            top = fmaxf(top, p[j]);
        }
        const float mn = fmaxf(m, quad_max(top));
        const float ms = mn == -INFINITY ? 0.f : mn;
        const float fix = fast_exp2(m - ms);
        m = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < G::VK; ++j) {
            p[j] = fast_exp2(p[j] - (ms - kProbShift<T>));
            sum += p[j];
        }
        l = l * fix + sum;
        G::scale_acc(o, fix);
        typename G::Probs pr;
        G::pack_probs(p, pr);
        const bool crosses = t0 + G::KT > least;  // some row may not see some key
#pragma unroll
        for (int u = 0; u < G::U; ++u) {
            typename G::VBlock v;
            bool wild = false;
#pragma unroll
            for (int j = 0; j < G::VK; ++j) {
                const uint32_t off = __shfl(vo, G::key_of(j), kWave);
                G::load_chunk(vb + ((uint64_t)off << a.v_shift), u, row_bytes, v.w[j]);
                if (G::key_of(j) >= left) {  // 0 weight times what the place holds may be NaN
#pragma unroll
                    for (int i = 0; i < G::VW; ++i) v.w[j][i] = 0;
                }
                if (crosses) wild |= G::chunk_wild(v.w[j]);
            }
            if (!crosses || !__any(wild)) {
                G::accumulate(v, pr, u, o);
            } else {
                // an infinity or NaN that some of the rows must not see: one
                // token at a time
                const int tok = first_row / a.s.group;
                G::accumulate_seen(v, pr, u, most - before - tok + 1, t - tok,
                                   [&](int i, int j) {
                                       return t0 + G::key_of(j) < before + tok + i;
                                   },
                                   o);
            }
        }
    }
    l = quad_sum(l);
    if (__any(wrong)) l = NAN;
    if (!has || sees <= k0) return;
    if (sees <= a.piece) {
        const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) G::store_out(o, u, r, f, out, row_bytes);
        if (a.lse && lane < 16)
            a.lse[token * a.s.hq + hq] =
                l == 0.f ? -INFINITY : (m - kProbShift<T> + fast_log2(l)) * kLn2;
    } else {
        const int64_t at = ((int64_t)piece * a.tokens + token) * a.s.hq + hq;
        float* dst = a.part + at * a.s.dim;
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) G::store_part(o, u, r, 1.f, dst, a.s.dim);
        if (lane < 16) {
            a.part_ml[2 * at] = m;
            a.part_ml[2 * at + 1] = l;
        }
    }
}

// One wavefront per token and query head joins its pieces, in their order.
template <class T>
__global__ __launch_bounds__(kWaves* kWave) void k_paged_join(PagedArgs a) {
    const int lane = lane_id();
    const int64_t unit = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
    if (unit >= a.tokens * a.s.hq) return;
    const int64_t token = unit / a.s.hq;
    const int hq = (int)(unit - token * a.s.hq);
    if (token < a.q_rowptr[0]) return;
    const int64_t s = upper_index(a.q_rowptr, int64_t(0), a.seqs, token);
    const Sequence sq = read_sequence(a, s);
    if (sq.none || sq.bad || token < sq.q0 || token - sq.q0 >= sq.fresh) return;
    const int sees = sq.length - sq.fresh + 1 + (int)(token - sq.q0);
    if (sees <= a.piece) return;
    const int count = (sees + a.piece - 1) / a.piece;
    const int64_t step = a.tokens * a.s.hq;
    float m = -INFINITY;
    for (int i = lane; i < count; i += kWave) m = fmaxf(m, a.part_ml[2 * (i * step + unit)]);
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave] = {};
    for (int i = 0; i < count; ++i) {
        const int64_t at = i * step + unit;
        const float w = fast_exp2(a.part_ml[2 * at] - ms);
        l += a.part_ml[2 * at + 1] * w;
        const float* src = a.part + at * a.s.dim;
#pragma unroll
        for (int j = 0; j < SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave; ++j)
            if (j * kWave + lane < a.s.dim) o[j] += src[j * kWave + lane] * w;
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    T* dst = reinterpret_cast<T*>(a.out.base + token * a.out.row + hq * a.out.head);
#pragma unroll
    for (int j = 0; j < SPGEMM_ATTENTION_MAX_HEAD_DIM / kWave; ++j)
        if (j * kWave + lane < a.s.dim) dst[j * kWave + lane] = (T)(o[j] * f);
    if (a.lse && lane == 0)
        a.lse[unit] = l == 0.f ? -INFINITY : (m - kProbShift<T> + fast_log2(l)) * kLn2;
}

}  // namespace

void paged_attention(const PagedArgs& a, hipStream_t st) {
    const int64_t tiles = ceil_div((int64_t)a.max_new * a.s.group, 16);
    if (a.seqs == 0 || a.tokens == 0 || tiles == 0) return;
    if (tiles > 0x7fffffffLL) throw OverflowError("more rows per sequence than supported");
    const int64_t units = a.seqs * a.s.hkv * a.npieces * tiles;
    with_type(a.s.type, a.s.dim, [&](auto tag) {
        using Tag = decltype(tag);
        auto run = k_paged<typename Tag::Geo, typename Tag::Elem>;
        hipLaunchKernelGGL(run, dim3(grid_1d(xcd_grid(ceil_div(units, kWaves)))),
                           dim3(kWaves * kWave), 0, st, a, (int32_t)tiles);
        SG_LAUNCH_CHECK();
        if (a.npieces > 1) {
            hipLaunchKernelGGL(k_paged_join<typename Tag::Elem>,
                               dim3(grid_1d(ceil_div(a.tokens * a.s.hq, kWaves))),
                               dim3(kWaves * kWave), 0, st, a);
            SG_LAUNCH_CHECK();
        }
    });
}

}  // namespace sg
