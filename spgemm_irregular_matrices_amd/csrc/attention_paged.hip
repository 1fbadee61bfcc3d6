// Attention of new tokens over a paged key/value cache.
#include "attention_paged.h"

namespace sg {

namespace {

constexpr int kWaves = 4;

// Few rows per sequence and key head: one wavefront takes 16 rows and one
// piece of the keys, straight from memory. The next tile's rows are under way
// while one is computed, as in the forward pass over a mask. Bound by memory:
// the next token of 64 sequences of 8.5 K tokens on average, 8 key heads of
// 128, reads 2.2 GB in 468 us with the join (4.7 TB/s; a large copy moves 4.9).
template <class G, class T>
__global__ __launch_bounds__(kWaves* kWave, G::kDim <= 128 ? 2 : 1) void k_paged(PagedArgs a,
                                                                                 int32_t tiles) {
    __shared__ __align__(16) char stage[kWaves][G::KT * G::kRowBytes];
    const int lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    char* krows = stage[w];
    const int rbase = G::row_base(0), cbase = G::chunk_base(0);
    int64_t unit = xcd_block() * kWaves + w;
    if (unit >= a.seqs * a.s.hkv * a.npieces * tiles) return;
    const int tile = (int)(unit % tiles);
    unit /= tiles;
    const int piece = (int)(unit % a.npieces);
    unit /= a.npieces;
    const int64_t s = unit % a.seqs;
    const int h = (int)(unit / a.seqs);
    const TileJob job = tile_job(a, s, tile, 16, piece);
    if (job.idle) return;
    const int n = lane & 15;
    const int row_bytes = a.s.dim * (int)sizeof(T);
    const TileRow r = tile_row(a, job, job.first + n, h);
    if (job.sq.bad) {
        if (piece == 0) store_nan<T>(a, r);
        return;
    }
    if (job.k0 >= job.k1) return;
    const int lo = __builtin_amdgcn_readfirstlane(r.t);

    typename G::RowFrag q;
    typename G::VBlock k[G::U], v[G::U];
    G::zero_row(q);
    if (r.has) G::load_row(a.q.base + r.token * a.q.row + r.hq * a.q.head, row_bytes, q);
    G::sign_row(q, a.s.c);
    const char* kb = a.k + h * a.k_head;
    const char* vb = a.v + h * a.v_head;
    const int32_t* pages = a.col + job.sq.page0;
    bool wrong = false;  // a page outside the cache
    struct Place {
        uint32_t id, slot;
    };
    // lanes past the piece's end repeat its last key
    const auto place = [&](int t0) {
        const uint32_t key = (uint32_t)min(t0 + (lane & (G::KT - 1)), job.k1 - 1);
        const uint32_t pg = a.page_div.div(key);
        return Place{(uint32_t)pages[pg], key - pg * a.page_div.d};
    };
    const auto checked = [&](Place& x) {
        if (x.id >= (uint64_t)a.npages) {
            wrong = true;
            x.id = 0;
        }
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
    const auto load_k = [&](const Place& x) {
        load(k, kb, x.id * a.k_page + x.slot * a.k_slot, a.k_shift);
    };
    const auto load_v = [&](const Place& x) {
        load(v, vb, x.id * a.v_page + x.slot * a.v_slot, a.v_shift);
    };
    Place now = place(job.k0), here = now;  // here: of the tile that is computed
    Place next = now;
    if (job.k0 + G::KT < job.k1) next = place(job.k0 + G::KT);
    checked(now);
    load_k(now);
    load_v(now);

    typename G::Acc o;
    G::zero_acc(o);
    Softmax<G, T> sm;
    for (int t0 = job.k0; t0 < job.k1; t0 += G::KT) {
        const int left = job.k1 - t0;
        const bool more = left > G::KT;
        wave_lds_sync();
        G::stage_tile(krows, cbase, k);
        wave_lds_sync();
        here = now;
        if (more) {
            now = next;
            checked(now);
            load_k(now);
            if (left > 2 * G::KT) next = place(t0 + 2 * G::KT);
        }
        f32x4 sc[1][G::KSUB];
#pragma unroll
        for (int b = 0; b < G::KSUB; ++b) {
            typename G::RowFrag x;
            G::staged_row(krows, rbase, 16 * b, x);
            sc[0][b] = G::dot(x, q, f32x4{0, 0, 0, 0});
        }
        typename G::Probs pr[1];
        sm.step(sc, Seen::first(min(left, job.before + r.t - t0)), a.s.mag, o, pr);
        if (left < G::KT) G::clear_past(v, left);
        const bool crosses = t0 + G::KT > job.before + lo;  // some row may not see some key
#pragma unroll
        for (int u = 0; u < G::U; ++u) {
            if (crosses) {
                // a key that a row does not see must not reach it as 0 times
                // an infinity or a NaN
                float z = 0.f;
#pragma unroll
                for (int j = 0; j < G::VK; ++j) z = G::chunk_zero(v[u].w[j], z);
                if (__any(z != 0.f))
                    G::add_wild_keys(
                        v[u], pr[0], u, row_bytes,
                        [&](int key) {
                            const uint32_t off =
                                __shfl(here.id * a.v_page + here.slot * a.v_slot, key, kWave);
                            return vb + ((uint64_t)off << a.v_shift);
                        },
                        [&](int key) { return t0 + key < job.before + r.t; }, o);
            }
            G::accumulate(v[u], pr[0], u, o);
        }
        if (more) load_v(now);
    }
    sm.finish(a.s.mag);
    if (__any(wrong)) sm.l = NAN;
    store_row<G, T>(a, job, r, piece, o, sm);
}

// Many rows: a work group of 4 wavefronts takes 4 * 16 * QB rows, a wavefront
// 16 * QB of them, and BK keys at a time are shared in LDS. Each operand made
// from the shared keys serves QB products. 2596 new tokens of two sequences,
// 46 K tokens together, 32 heads of 128: 1.2 TFLOP in 1400 us, 840 TFLOP/s. The
// vector unit's softmax and the matrix units are 50 % and 39 % busy, which with
// two wavefronts to a SIMD (254 of 256 registers each) hide each other only in
// part. Padded widths of up to 128 values spill 15 registers, 58 in single
// precision (4 without padding): 80 values take 1900 us.
template <class G, class T>
struct Wide {
    static constexpr int QB = G::kDim <= 128 ? 2 : 1;  // 16-row blocks per wavefront
    static constexpr int BM = kWaves * 16 * QB;
    static_assert(BM <= kPagedTileMost, "the limit of rows counts on it");
    static constexpr int BK = G::kRowBytes <= 256 ? 64 : 32;
    // Tiles of keys per step of the softmax. Two share its reductions, its
    // rescale and the branches: chunks of 2048 over 32768 keys, 32 heads,
    // 1650 -> 1500 us, 64-wide heads 236 -> 181 us. Single precision has no
    // registers for a second tile (174 -> 200 us: many more spilled than its 4).
    static constexpr int NS = sizeof(T) == 2 && BK > G::KT ? 2 : 1;
};

template <class G, class T>
__global__ __launch_bounds__(kWaves* kWave, G::kDim <= 128 ? 2 : 1) void k_paged_wide(
    PagedArgs a, int32_t tiles) {
    using W = Wide<G, T>;
    constexpr int NT = kWaves * kWave, BK = W::BK, QB = W::QB, NS = W::NS;
    constexpr int kPieces = G::kRowBytes / 16, kLoads = BK * kPieces / NT, kStep = NT / kPieces;
    static_assert(BK * kPieces % NT == 0 && BK % (NS * G::KT) == 0, "tile shape");
    __shared__ __align__(16) char rows[2][BK * G::kRowBytes];  // k, v
    __shared__ uint32_t off[2][2][BK];       // of this tile and the next, k and v
    __shared__ unsigned long long wild_s[2];  // keys whose value rows are not all finite
    __shared__ int wrong_s;
    const int tid = threadIdx.x, lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    int64_t unit = xcd_block();
    if (unit >= a.seqs * a.s.hkv * a.npieces * tiles) return;
    const int tile = tiles - 1 - (int)(unit % tiles);  // the longest first
    unit /= tiles;
    const int piece = (int)(unit % a.npieces);
    unit /= a.npieces;
    const int64_t s = unit % a.seqs;
    const int h = (int)(unit / a.seqs);
    const TileJob job = tile_job(a, s, tile, W::BM, piece);
    if (job.idle) return;
    const int n = lane & 15;
    const int row_bytes = a.s.dim * (int)sizeof(T);
    const int row0 = job.first + 16 * QB * w;  // this wavefront's first row
    TileRow r[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) r[b] = tile_row(a, job, row0 + 16 * b + n, h);
    if (job.sq.bad) {
        if (piece == 0)
#pragma unroll
            for (int b = 0; b < QB; ++b) store_nan<T>(a, r[b]);
        return;
    }
    if (job.k0 >= job.k1) return;
    if (tid == 0) {
        wrong_s = 0;
        wild_s[0] = 0;
    }
    // keys that some row of the wavefront sees (none: it only helps to load)
    const int lo = __builtin_amdgcn_readfirstlane(r[0].t);
    const int hi = __builtin_amdgcn_readlane(r[QB - 1].t, 15);
    const int mine = row0 < job.rows ? min(job.k1, job.before + hi) : 0;
    const int full = min(job.k1, job.before + lo);  // that all of them see

    typename G::RowFrag q[QB];
    typename G::AccB o[QB];
    Softmax<G, T> sm[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        G::zero_row(q[b]);
#pragma unroll
        for (int i = 0; i < G::NB; ++i) o[b].o[i] = f32x4{0, 0, 0, 0};
        if (r[b].has)
            G::load_row(a.q.base + r[b].token * a.q.row + r[b].hq * a.q.head, row_bytes, q[b]);
        G::sign_row(q[b], a.s.c);
    }
    const char* kb = a.k + h * a.k_head;
    const char* vb = a.v + h * a.v_head;
    const int32_t* pages = a.col + job.sq.page0;
    // thread i < BK looks key i of a tile up
    uint32_t id = 0;
    const auto load_id = [&](int t0) {
        if (tid < BK && t0 + tid < job.k1) id = (uint32_t)pages[a.page_div.div(t0 + tid)];
    };
    const auto put_offsets = [&](int t0, int par) {
        if (tid < BK && t0 + tid < job.k1) {
            if (id >= (uint64_t)a.npages) {
                wrong_s = 1;
                id = 0;
            }
            const uint32_t key = t0 + tid, slot = key - a.page_div.div(key) * a.page_div.d;
            off[par][0][tid] = id * a.k_page + slot * a.k_slot;
            off[par][1][tid] = id * a.v_page + slot * a.v_slot;
        }
    };
    u32x4 fly[2][kLoads];
    const int prow = tid / kPieces, pbyte = tid % kPieces * 16;
    const bool inside = G::kFull || pbyte < row_bytes;
    const char* kp = kb + (inside ? pbyte : 0);
    const char* vp = vb + (inside ? pbyte : 0);
    const auto load_rows = [&](int t0, int par) {
        const int left = job.k1 - t0;
        if (left >= BK) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int p = i * kStep + prow;
                fly[0][i] = *reinterpret_cast<const u32x4*>(kp + ((uint64_t)off[par][0][p] << a.k_shift));
                fly[1][i] = *reinterpret_cast<const u32x4*>(vp + ((uint64_t)off[par][1][p] << a.v_shift));
            }
        } else {
            // places past the end read the tile's first key and become 0
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int p = i * kStep + prow;
                const bool in = p < left;
                const u32x4 x = *reinterpret_cast<const u32x4*>(
                    kp + ((uint64_t)off[par][0][in ? p : 0] << a.k_shift));
                const u32x4 y = *reinterpret_cast<const u32x4*>(
                    vp + ((uint64_t)off[par][1][in ? p : 0] << a.v_shift));
                fly[0][i] = in ? x : u32x4{0, 0, 0, 0};
                fly[1][i] = in ? y : u32x4{0, 0, 0, 0};
            }
        }
        if (!inside) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) fly[0][i] = fly[1][i] = u32x4{0, 0, 0, 0};
        }
    };
    load_id(job.k0);
    __syncthreads();  // wrong_s, wild_s
    put_offsets(job.k0, 0);
    __syncthreads();
    load_rows(job.k0, 0);
    load_id(job.k0 + BK);
    int par = 0;
    for (int t0 = job.k0; t0 < job.k1; t0 += BK, par ^= 1) {
        __syncthreads();  // the last tile's readers are done
        if (t0 + BK > job.before + job.first / a.s.group) {
            // some row may not see some key: a value row with an infinity or
            // a NaN is staged as 0, so that 0 times it stays 0, and is added
            // on its own below for the rows that see it
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t x[4] = {fly[1][i][0], fly[1][i][1], fly[1][i][2], fly[1][i][3]};
                const uint64_t b = __ballot(G::words_wild(x));
                const int lane0 = lane / kPieces * kPieces;  // of this row's pieces
                const uint64_t whole = kPieces == 64 ? ~0ull : (1ull << (kPieces & 63)) - 1;
                if (b >> lane0 & whole) {
                    fly[1][i] = u32x4{0, 0, 0, 0};
                    if (lane == lane0) atomicOr(&wild_s[par], 1ull << (i * kStep + prow));
                }
            }
        }
        const int put = G::stage_at(prow, pbyte);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = G::stage_more(put, i * kStep, 0);
            *reinterpret_cast<u32x4*>(rows[0] + at) = fly[0][i];
            *reinterpret_cast<u32x4*>(rows[1] + at) = fly[1][i];
        }
        put_offsets(t0 + BK, par ^ 1);
        __syncthreads();
        if (tid == 0) wild_s[par ^ 1] = 0;
        if (t0 + BK < job.k1) {
            load_rows(t0 + BK, par ^ 1);
            load_id(t0 + 2 * BK);
        }
        const uint64_t wild = wild_s[par];
#pragma unroll 1
        for (int at = 0; at < BK; at += NS * G::KT) {  // the first staged row of NS tiles
            const int t = t0 + at;
            if (t >= mine) break;
            f32x4 sc[QB][NS][G::KSUB];
            const auto scores = [&](int at) {
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const int rb = G::row_base(at + i * G::KT);
#pragma unroll
                    for (int b = 0; b < G::KSUB; ++b) {
                        typename G::RowFrag k;
                        G::staged_row(rows[0], rb, 16 * b, k);
#pragma unroll
                        for (int x = 0; x < QB; ++x)
                            sc[x][i][b] = G::dot(k, q[x], f32x4{0, 0, 0, 0});
                    }
                }
                if (t + NS * G::KT > full) {  // some row does not see some key
#pragma unroll
                    for (int x = 0; x < QB; ++x)
#pragma unroll
                        for (int i = 0; i < NS; ++i)
                            sm[x].hide(sc[x][i], Seen::first(min(job.k1, job.before + r[x].t) - t -
                                                             i * G::KT));
                }
            };
            scores(at);
            typename G::Probs pr[QB][NS];
            float fix[QB], old[QB];
            // Queries whose scores are far from 0 (see Softmax) get their
            // weights again, after those of the others: asked before the
            // exponentials, which it keeps from running beside each other,
            // the branch took 1494 -> 1524 us for chunks of 2048 over 32768
            // keys. Padded widths have no registers for that (192 values:
            // 9190 us asked before, 10297 after).
            constexpr bool kAgain = G::kFull;
            bool moved = false, far = false;
#pragma unroll
            for (int x = 0; x < QB; ++x) {
                bool one;
                old[x] = sm[x].l;
                fix[x] = sm[x].template weigh<!kAgain>(sc[x], a.s.mag, pr[x], one);
                moved |= fix[x] != 1.f;
                far |= kAgain && one;
            }
            if (__any(moved || far)) {
                if (__any(far)) {
                    // Hardly ever, so the scores are made again; from 128 values on
                    // they look like others to the compiler, which would keep
                    // them through every step in registers that are not there.
                    int again = at;
                    if constexpr (G::kDim > 64) asm volatile("" : "+s"(again));
                    scores(again);
#pragma unroll
                    for (int x = 0; x < QB; ++x)
                        sm[x].weigh_far(sc[x], a.s.mag, old[x], fix[x], pr[x]);
                }
#pragma unroll
                for (int x = 0; x < QB; ++x) G::scale_acc(o[x], fix[x]);
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int vbase = G::value_base(at + i * G::KT);
#pragma unroll
                for (int b = 0; b < G::NB; ++b) {
                    const u32x4 v = G::value_frag(rows[1], vbase, b);
#pragma unroll
                    for (int x = 0; x < QB; ++x) o[x].o[b] = G::add_block(v, pr[x][i], o[x].o[b]);
                }
            }
            if (wild == 0) continue;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int first = at + i * G::KT;
#pragma unroll 1
                for (int key = 0; key < G::KT; ++key) {
                    if (!(wild >> (first + key) & 1)) continue;
                    const char* row = vb + ((uint64_t)off[par][1][first + key] << a.v_shift);
#pragma unroll
                    for (int x = 0; x < QB; ++x) {
                        const float p = G::prob_of(pr[x][i], key);
                        if (t0 + first + key >= job.before + r[x].t) continue;
#pragma unroll
                        for (int b = 0; b < G::NB; ++b) {
                            const int d = 16 * b + 4 * (lane >> 4);
                            if (G::kFull || d < a.s.dim)
                                o[x].o[b] = G::add_four(row + d * (int)sizeof(T), p, o[x].o[b]);
                        }
                    }
                }
            }
        }
    }
    if (row0 >= job.rows) return;
    const bool wrong = wrong_s != 0;
#pragma unroll
    for (int x = 0; x < QB; ++x) {
        sm[x].finish(a.s.mag);
        if (wrong) sm[x].l = NAN;
        store_row<G, T>(a, job, r[x], piece, o[x], sm[x]);
    }
}

// One wavefront per token and query head joins its pieces, in their order.
template <class T>
__global__ __launch_bounds__(kWaves* kWave) void k_paged_join(PagedArgs a) {
    const int lane = lane_id();
    const int64_t unit = grid_block() * kWaves + threadIdx.x / kWave;
    if (unit >= a.tokens * a.s.hq) return;
    const int64_t token = unit / a.s.hq;
    const int hq = (int)(unit - token * a.s.hq);
    Sequence sq;
    int64_t s = upper_index(a.q_rowptr, int64_t(0), a.seqs, token);
    if (!find_sequence(a, token, s, sq) || sq.bad) return;
    const int sees = sq.length - sq.fresh + 1 + (int)(token - sq.q0);
    if (sees <= a.piece) return;
    const int count = (sees + a.piece - 1) / a.piece;
    const int64_t step = a.tokens * a.s.hq;
    const float* ml = a.part_ml + 2 * unit;
    float m, l;
    join_sums(ml, step, count, m, l);
    const JoinedRow o(a.part + unit * a.s.dim, step * a.s.dim, count, a.s.dim,
                      [&](int i) { return fast_exp2(ml[2 * i * step] - m); });
    o.store<T>(a.out.base + token * a.out.row + hq * a.out.head, l == 0.f ? 0.f : 1.f / l,
               a.s.dim);
    if (a.lse && lane == 0)
        a.lse[unit] = l == 0.f ? -INFINITY : (m - kProbShift<T> + fast_log2(l)) * kLn2;
}

}  // namespace

// 16 sequences of 4.2 K tokens on average, 4 key heads, bf16 of 128 values a
// head: 20 rows 55 us by single wavefronts, 45 us shared (16 rows: 56 and 46, but
// with 64 values 29 and 33). The shared tiles are of 128 rows whatever is there
// (64 from 129 values on), which costs more where products take longer: 256
// values 87 and 108 us at 20 rows, 112 and 114 at 48, 150 and 116 at 64; single
// precision 98 and 186 at 20, 229 and 308 at 96 (64 values: 178 and 175).
bool paged_wide(const AttnShape& s, int64_t rows) {
    return rows > (s.type == SPGEMM_TYPE_F32 ? 96 : s.dim > 128 ? 48 : 16);
}

int paged_tile_rows(const AttnShape& s, int64_t rows) {
    if (!paged_wide(s, rows)) return 16;
    const int dim = s.dim;
    int bm = 0;
    with_dim<float>(dim, [&](auto tag) { bm = Wide<typename decltype(tag)::Geo, float>::BM; });
    return bm;
}

void paged_attention(const PagedArgs& a, hipStream_t st) {
    const int64_t rows = (int64_t)a.max_new * a.s.group;
    const int64_t tiles = ceil_div(rows, paged_tile_rows(a.s, rows));
    if (a.seqs == 0 || a.tokens == 0 || tiles == 0) return;
    const int64_t units = a.seqs * a.s.hkv * a.npieces * tiles;
    with_type(a.s.type, a.s.dim, [&](auto tag) {
        using Tag = decltype(tag);
        using G = typename Tag::Geo;
        using T = typename Tag::Elem;
        if (paged_wide(a.s, rows)) {
            auto run = k_paged_wide<G, T>;
            hipLaunchKernelGGL(run, grid_2d(xcd_grid(units)), dim3(kWaves * kWave), 0, st, a,
                               (int32_t)tiles);
        } else {
            auto run = k_paged<G, T>;
            hipLaunchKernelGGL(run, grid_2d(xcd_grid(ceil_div(units, kWaves))),
                               dim3(kWaves * kWave), 0, st, a, (int32_t)tiles);
        }
        SG_LAUNCH_CHECK();
    });
    if (a.npieces > 1) paged_join(a, st);
}

void paged_join(const PagedArgs& a, hipStream_t st) {
    const auto run = a.s.type == SPGEMM_TYPE_BF16  ? k_paged_join<__bf16>
                     : a.s.type == SPGEMM_TYPE_F16 ? k_paged_join<_Float16>
                                                   : k_paged_join<float>;
    hipLaunchKernelGGL(run, grid_2d(ceil_div(a.tokens * a.s.hq, kWaves)), dim3(kWaves * kWave), 0, st,
                       a);
    SG_LAUNCH_CHECK();
}

}  // namespace sg
