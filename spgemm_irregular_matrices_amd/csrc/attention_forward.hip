// Softmax attention over the entries of a CSR mask, forward.
#include "attention.h"

namespace sg {

namespace {

constexpr int kWaves = 4;

// One wavefront: 16 query heads [16*mt, 16*mt+16) of a key head's group
// against `each` pieces in turn. The tiles of all its pieces form one stream,
// so that a short row costs no idle trip to memory: while a tile is computed
// the next one's key and value rows are under way and the indices of the one
// after that. All rows are loaded as chunks, 16 lanes to a row: loaded as rows
// (a lane to a row) each lane's 16 bytes are an access of their own to the
// first-level cache, four times as many, and that rate is what bound this
// kernel. K takes the other layout through the wavefront's own LDS.
// With SHARED a piece belongs to a block of rows: the tile's queries are heads
// of several rows, and each sees the keys that its row stores.
// What bounds it is the gather of rows that do not fit the 4 MB L2 of an XCD:
// 509 K entries of 16384 rows, 32 heads of 128 on 8, in 261 us (2.1 GB
// gathered, 1.5 GB of them from the last-level cache); 512 keys of 65536 for
// each of 4096 rows, 32 heads on 2, in 180 us (2.1 GB and 1.2 GB). Vector and
// matrix units are a third and a tenth busy.
template <class G, class T, bool SHARED>
__global__ __launch_bounds__(kWaves* kWave, G::kDim <= 128 ? 2 : 1) void k_attn_forward(
    ForwardArgs a, int each, int64_t groups) {
    __shared__ __align__(16) char stage[kWaves][G::KT * G::kRowBytes];
    const int lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    char* krows = stage[w];
    const int64_t block = xcd_block();
    const int hm = (int)(block / groups);  // key head and 16 query heads
    if (hm >= a.s.hkv * a.s.mtiles) return;
    const int64_t u0 = (block - hm * groups) * kWaves * each + w;
    const int h = hm / a.s.mtiles, mt = hm - h * a.s.mtiles;
    const int block_rows = SHARED ? kRowBlock : 1;
    const AttnColumn me(a.s, block_rows, h, mt);
    const int row_bytes = a.s.dim * (int)sizeof(T);
    const auto row_of = [&](int row) { return (int64_t)row * block_rows + me.rr; };
    const auto here = [&](int64_t row) { return me.has && (!SHARED || row < a.nrows); };

    PieceStream st(a.side, u0, kWaves, each);
    for (uint64_t e = st.empty; e; e &= e - 1) {
        const int64_t row = row_of(st.row(__builtin_ctzll(e)));
        if (!here(row)) continue;
        typename G::Acc zero;
        G::zero_acc(zero);
        char* out = a.out.base + row * a.out.row + me.hq * a.out.head;
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) G::store_out(zero, u, r, 0.f, out, row_bytes);
        if (a.lse && lane < 16) a.lse[row * a.s.hq + me.hq] = -INFINITY;
    }
    if (!st.todo) return;

    const char* kb = a.k.base + h * a.k.head;
    const char* vb = a.v.base + h * a.v.head;
    const int rbase = G::row_base(0), cbase = G::chunk_base(0);
    typename G::RowFrag q;
    typename G::VBlock k[G::U], v[G::U];
    const auto load_q = [&](int i) {
        G::zero_row(q);
        const int64_t row = row_of(st.row(i));
        if (here(row)) G::load_row(a.q.base + row * a.q.row + me.hq * a.q.head, row_bytes, q);
        G::sign_row(q, a.s.c);
    };
    const auto load = [&](typename G::VBlock (&x)[G::U], const char* base, uint32_t off,
                          uint32_t shift) {
#pragma unroll
        for (int j = 0; j < G::VK; ++j) {
            const char* row =
                base + ((uint64_t)(uint32_t)__shfl(off, G::key_of(j), kWave) << shift);
#pragma unroll
            for (int u = 0; u < G::U; ++u) G::load_chunk(row, u, row_bytes, x[u].w[j]);
        }
    };
    const auto load_k = [&](uint32_t id) { load(k, kb, id * a.k.unit, a.k.shift); };
    const auto load_v = [&](uint32_t id) { load(v, vb, id * a.v.unit, a.v.shift); };

    PieceStream::Cursor cur, ahead;  // ahead: the tile whose entries are loaded
    st.open(cur);
    PieceStream::Entry now = st.entry<SHARED>(cur, G::KT), next;
    load_q(cur.i);
    load_k(now.id);
    load_v(now.id);
    ahead = cur;
    st.next(ahead, G::KT);
    if (ahead.more) next = st.entry<SHARED>(ahead, G::KT);

    typename G::Acc o;
    G::zero_acc(o);
    Softmax<G, T> sm;
    while (true) {
        const int left = cur.len - cur.t0;
        const bool last = left <= G::KT, more = ahead.more;
        wave_lds_sync();
        G::stage_tile(krows, cbase, k);
        wave_lds_sync();
        const PieceStream::Entry then = next;
        if (more) load_k(then.id);
        f32x4 s[1][G::KSUB];
#pragma unroll
        for (int b = 0; b < G::KSUB; ++b) {
            typename G::RowFrag x;
            G::staged_row(krows, rbase, 16 * b, x);
            s[0][b] = G::dot(x, q, f32x4{0, 0, 0, 0});
        }
        if (more && last) load_q(ahead.i);
        const PieceStream::Cursor after = ahead;
        if (more) {
            st.next(ahead, G::KT);
            if (ahead.more) next = st.entry<SHARED>(ahead, G::KT);
        }
        typename G::Probs pr[1];
        const Seen seen = SHARED ? me.seen(now.bits) : Seen::first(left);
        sm.step(s, seen, a.s.mag, o, pr);
        if (left < G::KT) G::clear_past(v, left);
#pragma unroll
        for (int u = 0; u < G::U; ++u) {
            if constexpr (SHARED) {
                // a key that a row does not store must not reach it as 0
                // times an infinity or a NaN
                float z = 0.f;
#pragma unroll
                for (int j = 0; j < G::VK; ++j) z = G::chunk_zero(v[u].w[j], z);
                if (__any(z != 0.f))
                    G::add_wild_keys(
                        v[u], pr[0], u, row_bytes,
                        [&](int key) {
                            const uint32_t off = __shfl(now.id * a.v.unit, key, kWave);
                            return vb + ((uint64_t)off << a.v.shift);
                        },
                        [&](int key) { return __shfl(now.bits, key, kWave) >> me.rr & 1; }, o);
            }
            G::accumulate(v[u], pr[0], u, o);
        }
        if (more) load_v(then.id);
        if (last) {
            sm.finish(a.s.mag);
            const int slot = st.slot(cur.i);
            const int64_t row = row_of(st.row(cur.i));
            if (here(row) && slot < 0) {
                const float f = sm.factor();
                char* out = a.out.base + row * a.out.row + me.hq * a.out.head;
#pragma unroll
                for (int u = 0; u < G::U; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) G::store_out(o, u, r, f, out, row_bytes);
                if (a.lse && lane < 16) a.lse[row * a.s.hq + me.hq] = sm.lse();
            } else if (here(row)) {
                const int64_t at = ((int64_t)slot * block_rows + me.rr) * a.s.hq + me.hq;
                float* dst = a.part + at * a.s.dim;
#pragma unroll
                for (int u = 0; u < G::U; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) G::store_part(o, u, r, 1.f, dst, a.s.dim);
                if (lane < 16) {
                    a.part_ml[2 * at] = sm.m;
                    a.part_ml[2 * at + 1] = sm.l;
                }
            }
            if (!more) break;
            G::zero_acc(o);
            sm = Softmax<G, T>();
        }
        cur = after;
        now = then;
    }
}

// The rows of more than one piece: one wavefront per row and query head
// joins the pieces, in their order (15 us of 270 where 509 K entries make
// 16384 rows of a power law).
template <class T>
__global__ __launch_bounds__(kWaves* kWave) void k_attn_join(ForwardArgs a) {
    const int lane = lane_id();
    const int64_t unit = grid_block() * kWaves + threadIdx.x / kWave;
    const int64_t lines = (int64_t)a.side.block * a.s.hq;
    if (unit >= a.side.nsplits * lines) return;
    const int64_t sp = unit / lines, line = unit - sp * lines;
    const AttnSplit s = a.side.splits[sp];
    const int64_t row = (int64_t)s.row * a.side.block + line / a.s.hq;
    const int hq = (int)(line % a.s.hq);
    if (row >= a.nrows) return;
    const int64_t first = (int64_t)s.slot * lines + line;
    const float* ml = a.part_ml + 2 * first;
    float m, l;
    join_sums(ml, lines, s.count, m, l);
    const JoinedRow o(a.part + first * a.s.dim, lines * a.s.dim, s.count, a.s.dim,
                      [&](int i) { return fast_exp2(ml[2 * i * lines] - m); });
    o.store<T>(a.out.base + row * a.out.row + hq * a.out.head, l == 0.f ? 0.f : 1.f / l, a.s.dim);
    if (a.lse && lane == 0)
        a.lse[row * a.s.hq + hq] = l == 0.f ? -INFINITY : (m - kProbShift<T> + fast_log2(l)) * kLn2;
}

}  // namespace

void attention_forward(const ForwardArgs& a, hipStream_t st) {
    const int64_t heads = (int64_t)a.s.hkv * a.s.mtiles;
    if (a.side.npieces == 0) return;
    const int each = pieces_per_wave(a.side.npieces * heads);
    const int64_t groups = ceil_div(a.side.npieces, kWaves * each);
    with_type(a.s.type, a.s.dim, [&](auto tag) {
        using Tag = decltype(tag);
        auto run = a.side.block > 1 ? k_attn_forward<typename Tag::Geo, typename Tag::Elem, true>
                                    : k_attn_forward<typename Tag::Geo, typename Tag::Elem, false>;
        hipLaunchKernelGGL(run, grid_2d(xcd_grid(groups * heads)), dim3(kWaves * kWave), 0,
                           st, a, each, groups);
        SG_LAUNCH_CHECK();
        if (a.side.nsplits > 0) {
            hipLaunchKernelGGL(k_attn_join<typename Tag::Elem>,
                               grid_2d(ceil_div(a.side.nsplits * a.side.block * a.s.hq, kWaves)),
                               dim3(kWaves * kWave), 0, st, a);
            SG_LAUNCH_CHECK();
        }
    });
}

}  // namespace sg
