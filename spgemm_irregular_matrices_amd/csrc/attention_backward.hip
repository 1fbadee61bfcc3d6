// Gradients of softmax attention over the entries of a CSR mask. The
// probabilities are recomputed twice from q, k and the log-sum-exp: once row
// by row for dq, once column by column for dk and dv. No pass adds to memory
// that another work group adds to, so nothing depends on the order of work
// groups and no buffer has to be cleared.
#include "attention.h"

namespace sg {

namespace {

constexpr int kWaves = 4;

// Half precision: dS is scaled by a power of two that follows its largest
// magnitude so far (about 2^11 for that one), as the running maximum of a
// softmax does, because gradients can lie anywhere in the floats' range while
// the type ends at 65504 and loses bits below 2^-14. Values that are small
// beside the largest lose nothing that the sum would keep.
struct HalfScale {
    float s = 0x1p60f;
    // The factor for sums made so far, after admitting magnitude mx (alike
    // in all lanes whose sums share a column).
    __device__ __forceinline__ float admit(float mx) {
        if (!(mx * s > 32768.f) || !(mx < INFINITY)) return 1.f;
        const int e = (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127;
        const float to = __builtin_bit_cast(float, (uint32_t)(127 + 11 - e) << 23);
        const float f = to / s;
        s = to;
        return f;
    }
};
// Probabilities of a half-precision dv: times 2^14, as in the forward pass.
template <class T>
constexpr float kProbScale = std::is_same<T, _Float16>::value ? 0x1p14f : 1.f;

// dq: one wavefront per piece of a row and 16 query heads of a key head, its
// pieces' tiles in one stream as in the forward pass. S^T and dP^T = V dO^T
// take the gathered rows as rows, dQ^T += K^T dS^T takes K as chunks: all come
// from memory as chunks, a tile ahead (see there), and are staged in the
// wavefront's own LDS for the other layout. Bound by the same gather as the
// forward pass: 509 K entries of 16384 rows, 32 heads of 128 on 8, in 330 us.
// Heads of 128 over blocks of rows spill 21 registers (fp16 10, fp32 61).
template <class G, class T, bool SHARED>
__global__ __launch_bounds__(kWaves* kWave, G::kDim <= 128 ? 2 : 1) void k_attn_grad_q(
    BackwardArgs a, int each, int64_t groups) {
    __shared__ __align__(16) char stage[kWaves][2][G::KT * G::kRowBytes];
    const int lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t block = xcd_block();
    const int hm = (int)(block / groups);
    if (hm >= a.s.hkv * a.s.mtiles) return;
    const int64_t u0 = (block - hm * groups) * kWaves * each + w;
    const int h = hm / a.s.mtiles, mt = hm - h * a.s.mtiles;
    const int block_rows = SHARED ? kRowBlock : 1;
    const AttnColumn me(a.s, block_rows, h, mt);
    const int row_bytes = a.s.dim * (int)sizeof(T);
    const auto row_of = [&](int row) { return (int64_t)row * block_rows + me.rr; };
    const auto here = [&](int64_t row) { return me.has && (!SHARED || row < a.nrows); };
    char* krows = stage[w][0];
    char* vrows = stage[w][1];
    const int rbase = G::row_base(0), cbase = G::chunk_base(0);

    PieceStream st(a.rows, u0, kWaves, each);
    for (uint64_t e = st.empty; e; e &= e - 1) {
        const int64_t row = row_of(st.row(__builtin_ctzll(e)));
        if (!here(row)) continue;
        typename G::Acc zero;
        G::zero_acc(zero);
        char* dst = a.dq.base + row * a.dq.row + me.hq * a.dq.head;
#pragma unroll
        for (int u = 0; u < G::U; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) G::store_out(zero, u, r, 0.f, dst, row_bytes);
    }
    if (!st.todo) return;

    const char* kb = a.k.base + h * a.k.head;
    const char* vb = a.v.base + h * a.v.head;
    typename G::RowFrag q, dout, out;
    typename G::VBlock k[G::U], v[G::U];
    float lse = INFINITY;  // lanes without a head: weights 0
    const auto load_q = [&](int i) {
        const int64_t row = row_of(st.row(i));
        G::zero_row(q);
        G::zero_row(dout);
        G::zero_row(out);
        if (here(row)) {
            G::load_row(a.q.base + row * a.q.row + me.hq * a.q.head, row_bytes, q);
            G::load_row(a.dout.base + row * a.dout.row + me.hq * a.dout.head, row_bytes, dout);
            G::load_row(a.out.base + row * a.out.row + me.hq * a.out.head, row_bytes, out);
            lse = a.lse[row * a.s.hq + me.hq];
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
    const auto load_k = [&](uint32_t id) { load(k, kb, id * a.k.unit, a.k.shift); };
    const auto load_v = [&](uint32_t id) { load(v, vb, id * a.v.unit, a.v.shift); };

    PieceStream::Cursor cur, ahead;
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
    HalfScale hs;
    float seen_lse = 0.f, delta = 0.f;  // of the piece that is computed
    bool fresh = true;  // first tile of its piece
    while (true) {
        const int left = cur.len - cur.t0;
        const bool last = left <= G::KT, more = ahead.more;
        if (fresh) {
            // summed as dP is, so that a row's only key, whose value is `out`,
            // has dS = 0 to the last bit
            delta = G::dot_own(out, dout);
            seen_lse = lse;
            const int64_t row = row_of(st.row(cur.i));
            if (here(row) && lane < 16 && st.lead(cur.i)) a.delta[row * a.s.hq + me.hq] = delta;
            fresh = false;
        }
        if (left < G::KT) G::clear_past(k, left);
        wave_lds_sync();
        G::stage_tile(krows, cbase, k);
        G::stage_tile(vrows, cbase, v);
        wave_lds_sync();
        const PieceStream::Entry then = next;
        if (more) {
            load_k(then.id);
            load_v(then.id);
        }
        f32x4 s[G::KSUB], dp[G::KSUB];
#pragma unroll
        for (int b = 0; b < G::KSUB; ++b) {
            typename G::RowFrag x;
            G::staged_row(krows, rbase, 16 * b, x);
            s[b] = G::dot(x, q, f32x4{0, 0, 0, 0});
            G::staged_row(vrows, rbase, 16 * b, x);
            dp[b] = G::dot_halves(x, dout);
        }
        if (more && last) load_q(ahead.i);
        const PieceStream::Cursor after = ahead;
        if (more) {
            st.next(ahead, G::KT);
            if (ahead.more) next = st.entry<SHARED>(ahead, G::KT);
        }
        const Seen seen = SHARED ? me.seen(now.bits) : Seen::first(left);
        float wild = 0.f;  // a NaN where a key's row may not be finite (see k_attn_grad_kv)
        if constexpr (SHARED) {
#pragma unroll
            for (int j = 0; j < G::VK; ++j) wild = fmaf(s[j >> 2][j & 3], 0.f, wild);
        }
        float ds[G::VK];
#pragma unroll
        for (int j = 0; j < G::VK; ++j) {
            const float p = weight<T>(s[j >> 2][j & 3], a.s.c, a.s.c_low, seen_lse);
            ds[j] = seen.pick(j, p * (dp[j >> 2][j & 3] - delta), 0.f);
        }
        if constexpr (std::is_same<T, _Float16>::value) {
            float mx = 0.f;
#pragma unroll
            for (int j = 0; j < G::VK; ++j) mx = fmaxf(mx, fabsf(ds[j]));
            const float f = hs.admit(quad_max(mx));
            if (__any(f != 1.f)) G::scale_acc(o, f);
#pragma unroll
            for (int j = 0; j < G::VK; ++j) ds[j] *= hs.s;
        }
        typename G::Probs pr;
        G::pack_probs(ds, pr);
#pragma unroll
        for (int u = 0; u < G::U; ++u) {
            typename G::VBlock x;
#pragma unroll
            for (int j = 0; j < G::VK; ++j) G::staged_chunk(krows, cbase, 0, j, u, x.w[j]);
            if constexpr (SHARED) {
                if (__any(wild != 0.f))
                    G::add_wild_keys(
                        x, pr, u, row_bytes,
                        [&](int key) {
                            const uint32_t off = __shfl(now.id * a.k.unit, key, kWave);
                            return kb + ((uint64_t)off << a.k.shift);
                        },
                        [&](int key) { return __shfl(now.bits, key, kWave) >> me.rr & 1; }, o);
            }
            G::accumulate(x, pr, u, o);
        }
        if (last) {
            float f = a.s.scale;
            if constexpr (std::is_same<T, _Float16>::value) f /= hs.s;
            const int slot = st.slot(cur.i);
            const int64_t row = row_of(st.row(cur.i));
            if (here(row) && slot < 0) {
                char* dst = a.dq.base + row * a.dq.row + me.hq * a.dq.head;
#pragma unroll
                for (int u = 0; u < G::U; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) G::store_out(o, u, r, f, dst, row_bytes);
            } else if (here(row)) {
                float* dst =
                    a.part_q + (((int64_t)slot * block_rows + me.rr) * a.s.hq + me.hq) * a.s.dim;
#pragma unroll
                for (int u = 0; u < G::U; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) G::store_part(o, u, r, f, dst, a.s.dim);
            }
            if (!more) break;
            G::zero_acc(o);
            hs = HalfScale();
            fresh = true;
        }
        cur = after;
        now = then;
    }
}

// dk and dv: one work group of 4 wavefronts per piece of a block of 16 columns
// and key head. The gathered list is the (row, query head) pairs of the
// piece's entries, kTilePairs at a time; the other operand of S and dP is the
// block's 16 k (or v) rows, and an entry's bits say which of the 16 scores
// are the mask's. A tile's q and dout rows come from memory once, a tile ahead
// of their use, and are shared in LDS. S and dP of a tile are spread over the
// wavefronts: 16 pairs each for tiles of 64, S and dP apart for tiles of 32, and
// by halves of the head dimension too for tiles of 16 (with rows of 512 and
// 1024 bytes these tiles let two work groups share a unit; in single precision,
// where the products take longest, two wavefronts with all of S and dP took
// 1260 us for 1150 with 128 values a head and, in tiles of 32, 1775 for 1390
// with 256). After P and dS are exchanged in LDS too, each wavefront makes one
// output (dv from dout and P, dk from q and dS) of one half of the head
// dimension: that keeps the accumulators at an eighth of the output each, where
// one wavefront with both outputs would need over 256 registers with a tile
// under way. The rows are turned over for it by transposing reads; as words
// that a byte permutation sorts it took a fifth more vector instructions (heads
// of 256 values: 620 -> 586 us).
// What bounds it is the gather where q and dout of the key head's group do not
// fit a 4 MB L2: 16384 rows of 4 heads, 509 K entries on 8 key heads, 8.3 GB
// in 1060 us, 7.5 GB of them from the last-level cache. Where they fit,
// the four barriers per tile, with three or four work groups to a unit: 1000 rows
// of 8 heads of 64, 1.2 GB in 237 us.
constexpr int kKvWaves = 4;
template <class G>
constexpr int kTilePairs = G::kRowBytes <= 256 ? 64 : G::kRowBytes <= 512 ? 32 : 16;

template <class G, class T>
__global__ __launch_bounds__(kKvWaves* kWave, G::kDim <= 128 ? 3 : 2) void k_attn_grad_kv(
    BackwardArgs a) {
    constexpr bool half = std::is_same<T, _Float16>::value;
    constexpr int TP = kTilePairs<G>, NT = kKvWaves * kWave;
    constexpr int kPieces = G::kRowBytes / 16;        // 16-byte pieces of a row
    constexpr int kLoads = TP * kPieces / NT;         // of each tensor per thread
    constexpr int kPitch = TP * (int)sizeof(T) + 16;  // bytes between keys of P and dS
    constexpr int kSets = G::kDim / 32;               // 16-index results per wavefront
    constexpr int kSteps = TP / G::KT;                // products over G::KT pairs each
    constexpr int kBlocks = TP / 16;                  // of 16 pairs, each S and dP of
    constexpr int kParts = kKvWaves / kBlocks;        // so many wavefronts
    static_assert(TP * kPieces % NT == 0 && kSets >= 1, "tile shape");
    __shared__ __align__(16) char rows[2][TP * G::kRowBytes];  // q, dout
    __shared__ __align__(16) char weights[2][kColBlock * kPitch];  // dS, P: [key][pair]
    __shared__ __align__(16) char keys[2][kColBlock * G::kRowBytes];  // k, v
    __shared__ uint32_t off[2][TP];
    __shared__ __align__(16) float lse_s[TP], delta_s[TP];
    __shared__ __align__(16) uint32_t bits_s[TP];
    __shared__ float most[kKvWaves][kColBlock];
    __shared__ int wild_s[kKvWaves];
    __shared__ __align__(16) f32x4 part_s[kParts > 1 ? kKvWaves : 1][kWave];

    const int tid = threadIdx.x, lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    // every XCD has an eighth of each head's pieces, and all are at one head
    // at a time: what they gather of it together stays in the last-level cache
    const uint32_t per = (uint32_t)ceil_div(a.cols.npieces, kXcds);
    const uint32_t turn = (uint32_t)(grid_block() / kXcds);  // (2^32 would write 2^42 bytes)
    const int h = (int)(turn / per);
    const int64_t piece = (int64_t)(blockIdx.x % kXcds) * per + turn % per;
    if (h >= a.s.hkv || piece >= a.cols.npieces) return;
    const AttnPiece pc = a.cols.pieces[piece];
    const int n = lane & 15, quad = lane >> 4;
    const int64_t col = (int64_t)pc.row * kColBlock + n;  // this lane's key
    const int row_bytes = a.s.dim * (int)sizeof(T);

    // the block's k and v rows wait in LDS too: 32 registers more (at 128 x 16
    // bits) would cost a third of the wavefronts
    if (w < 2) {
        typename G::RowFrag f;
        G::zero_row(f);
        const AttnRows& src = w ? a.vrow : a.krow;
        if (col < a.ncols) G::load_row(src.base + col * src.row + h * src.head, row_bytes, f);
#pragma unroll
        for (int t = 0; t < G::QS; ++t)
            *reinterpret_cast<u32x4*>(keys[w] + G::stage_at(n, 64 * t + 16 * quad)) = f.w[t];
    }
    f32x4 acc[kSets];
#pragma unroll
    for (int i = 0; i < kSets; ++i) acc[i] = f32x4{0, 0, 0, 0};
    HalfScale hs;
    const char* qb = a.gq.base + (int64_t)h * a.s.group * a.gq.head;
    const char* gb = a.gdout.base + (int64_t)h * a.s.group * a.gdout.head;
    const uint32_t qhead = (uint32_t)(a.gq.head >> a.gq.shift);
    const uint32_t ghead = (uint32_t)(a.gdout.head >> a.gdout.shift);
    const int32_t* idx = a.cols.idx + pc.first;
    const uint16_t* bits = a.cols.bits + pc.first;
    const int pairs = pc.len * a.s.group;

    // one pair per thread of the first TP: its row, then what belongs to it
    uint32_t id = 0, mine = 0;
    float lse = 0.f, delta = 0.f;
    const auto load_id = [&](int t0) {
        if (tid < TP && t0 + tid < pairs) id = (uint32_t)idx[a.group_div.div(t0 + tid)];
    };
    const auto put_offsets = [&](int t0) {
        if (tid < TP && t0 + tid < pairs) {
            const uint32_t g = t0 + tid - a.group_div.div(t0 + tid) * a.s.group;
            off[0][tid] = id * a.gq.unit + g * qhead;
            off[1][tid] = id * a.gdout.unit + g * ghead;
        }
    };
    u32x4 fly[2][kLoads];
    constexpr int kStep = NT / kPieces;  // rows that one load of the work group covers
    const int prow = tid / kPieces, pbyte = tid % kPieces * 16;  // this thread's place in them
    const bool inside = G::kFull || pbyte < row_bytes;
    const char* qp = qb + (inside ? pbyte : 0);
    const char* gp = gb + (inside ? pbyte : 0);
    const auto load_rows = [&](int t0) {
        if (t0 + TP <= pairs) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int p = i * kStep + prow;
                fly[0][i] = *reinterpret_cast<const u32x4*>(qp + ((uint64_t)off[0][p] << a.gq.shift));
                fly[1][i] =
                    *reinterpret_cast<const u32x4*>(gp + ((uint64_t)off[1][p] << a.gdout.shift));
            }
        } else {
            // pairs past the end read the first row and become 0
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int p = i * kStep + prow;
                const bool in = t0 + p < pairs;
                const u32x4 x = *reinterpret_cast<const u32x4*>(
                    qp + (in ? (uint64_t)off[0][p] << a.gq.shift : 0));
                const u32x4 y = *reinterpret_cast<const u32x4*>(
                    gp + (in ? (uint64_t)off[1][p] << a.gdout.shift : 0));
                fly[0][i] = in ? x : u32x4{0, 0, 0, 0};
                fly[1][i] = in ? y : u32x4{0, 0, 0, 0};
            }
        }
        if (!inside) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) fly[0][i] = fly[1][i] = u32x4{0, 0, 0, 0};
        }
        mine = 0;
        lse = -INFINITY;
        delta = 0.f;
        if (tid < TP && t0 + tid < pairs) {
            const uint32_t e = a.group_div.div(t0 + tid), g = t0 + tid - e * a.s.group;
            const int64_t at = (int64_t)id * a.s.hq + h * a.s.group + g;
            mine = bits[e];
            lse = a.lse[at];
            delta = a.delta[at];
        }
    };
    if (pairs > 0) {
        load_id(0);
        put_offsets(0);
        __syncthreads();
        load_rows(0);
        load_id(TP);
    }
    for (int t0 = 0; t0 < pairs; t0 += TP) {
        __syncthreads();  // the last tile's readers are done
        const int put = G::stage_at(prow, pbyte);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = G::stage_more(put, i * kStep, 0);
            *reinterpret_cast<u32x4*>(rows[0] + at) = fly[0][i];
            *reinterpret_cast<u32x4*>(rows[1] + at) = fly[1][i];
        }
        if (tid < TP) {
            lse_s[tid] = lse;
            delta_s[tid] = delta;
            bits_s[tid] = mine;
        }
        put_offsets(t0 + TP);
        __syncthreads();
        if (t0 + TP < pairs) {
            load_rows(t0 + TP);
            load_id(t0 + 2 * TP);
        }
        // S, P, dP and dS of 16 pairs: by one wavefront, or S by one and dP by
        // another, or of halves of the head dimension by four
        const int blk = w % kBlocks, part = w / kBlocks;
        f32x4 s{0, 0, 0, 0}, dp{0, 0, 0, 0};
        {
            int mine_at = G::stage_at(16 * blk + n, 16 * quad), rbase = G::row_base(0);
            if constexpr (kParts == 1) {
                s = G::template dot_staged<G::QS>(rows[0], mine_at, keys[0], rbase);
                dp = G::template dot_staged<G::QS>(rows[1], mine_at, keys[1], rbase);
            } else {
                const int skip = kParts == 4 ? (part >> 1) * (G::kRowBytes / 2) : 0;
                s = G::template dot_staged<2 * G::QS / kParts>(rows[part & 1], mine_at ^ skip,
                                                               keys[part & 1], rbase ^ skip);
                part_s[w][lane] = s;
                __syncthreads();
                if (part == 0) {
                    dp = part_s[kBlocks + blk][lane];
                    if constexpr (kParts == 4) {
                        s += part_s[2 * kBlocks + blk][lane];
                        dp += part_s[3 * kBlocks + blk][lane];
                    }
                }
            }
        }
        float pr[4] = {}, ds[4] = {};  // (wavefronts without a block scale and drop these)
        float wild = 0.f;
        if (16 * w < TP) {
            const f32x4 l2 = *reinterpret_cast<const f32x4*>(lse_s + 16 * w + 4 * quad);
            const f32x4 dl = *reinterpret_cast<const f32x4*>(delta_s + 16 * w + 4 * quad);
            const u32x4 sees = *reinterpret_cast<const u32x4*>(bits_s + 16 * w + 4 * quad);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // 0 times any score: NaN if one is not finite, which it cannot
                // be where the pair's q or dout row holds an infinity or NaN
                wild = fmaf(s[r], 0.f, wild);
                wild = fmaf(dp[r], 0.f, wild);
                const bool on = sees[r] >> n & 1;
                pr[r] = on ? weight<T>(s[r], a.s.c, a.s.c_low, l2[r]) : 0.f;
                ds[r] = on ? pr[r] * (dp[r] - dl[r]) : 0.f;
                pr[r] *= kProbScale<T>;
            }
        }
        float fix = 1.f;
        if constexpr (half) {
            if (16 * w < TP) {
                float mx = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, fabsf(ds[r]));
                mx = quad_max(mx);
                if (quad == 0) most[w][n] = mx;
            }
            __syncthreads();
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < TP / 16; ++i) mx = fmaxf(mx, most[i][n]);
            fix = hs.admit(mx);
#pragma unroll
            for (int r = 0; r < 4; ++r) ds[r] *= hs.s;
        }
        if (16 * w < TP) {
            char* at = weights[0] + n * kPitch + (16 * w + 4 * quad) * (int)sizeof(T);
            char* ap = weights[1] + n * kPitch + (16 * w + 4 * quad) * (int)sizeof(T);
            if constexpr (G::k16) {
                *reinterpret_cast<u32x2*>(at) = u32x2{pack2<T>(ds[0], ds[1]), pack2<T>(ds[2], ds[3])};
                *reinterpret_cast<u32x2*>(ap) = u32x2{pack2<T>(pr[0], pr[1]), pack2<T>(pr[2], pr[3])};
            } else {
                *reinterpret_cast<f32x4*>(at) = f32x4{ds[0], ds[1], ds[2], ds[3]};
                *reinterpret_cast<f32x4*>(ap) = f32x4{pr[0], pr[1], pr[2], pr[3]};
            }
            const bool any = __any(wild != 0.f);
            if (lane == 0) wild_s[w] = any;
        }
        __syncthreads();
        // this wavefront's output: dk from q and dS (w even), dv from dout
        // and P (w odd), half w / 2 of the head dimension
        bool tame = true;
#pragma unroll
        for (int i = 0; i < TP / 16; ++i) tame = tame && wild_s[i] == 0;
        if constexpr (half) {
            if ((w & 1) == 0 && __any(fix != 1.f)) {
#pragma unroll
                for (int i = 0; i < kSets; ++i) acc[i] *= fix;
            }
        }
        const char* x = rows[w & 1];
        const char* y = weights[w & 1] + n * kPitch;
        const int half_at = (w >> 1) * (G::kRowBytes / 2);
        // of the pairs G::KT * st + G::key_of(j)
        const auto probs_at = [&](int st) {
            const char* at = y + (G::KT * st + 4 * quad) * (int)sizeof(T);
            if constexpr (G::k16) {
                const u32x2 lo = *reinterpret_cast<const u32x2*>(at);
                const u32x2 hi = *reinterpret_cast<const u32x2*>(at + 16 * sizeof(T));
                return typename G::Probs{{lo[0], lo[1], hi[0], hi[1]}};
            } else {
                const u32x4 b = *reinterpret_cast<const u32x4*>(at);
                return typename G::Probs{{b[0], b[1], b[2], b[3]}};
            }
        };
        // opaque, so that the tile's addresses are made again in each round
        // instead of held in registers throughout
        int base0 = G::value_base(0) ^ half_at;
        asm volatile("" : "+v"(base0));
        if (tame) {
#pragma unroll (G::k16 ? 1 : kSteps)
            for (int st = 0; st < kSteps; ++st) {
                const int base = G::stage_more(base0, G::KT * st, 0);
                const typename G::Probs pb = probs_at(st);
#pragma unroll
                for (int i = 0; i < kSets; ++i)
                    acc[i] = G::add_block(G::value_frag(x, base, i), pb, acc[i]);
            }
        } else {
            // key by key, with the pairs that do not have it as 0; the products
            // and their order are the same, so other keys get the same bits
#pragma unroll 1
            for (int st = 0; st < kSteps; ++st) {
                const int base = G::stage_more(base0, G::KT * st, 0);
                const typename G::Probs pb = probs_at(st);
                uint32_t has[G::VK];
#pragma unroll
                for (int j = 0; j < G::VK; ++j) has[j] = bits_s[G::KT * st + G::key_of(j)];
#pragma unroll
                for (int i = 0; i < kSets; ++i) {
                    const u32x4 all = G::value_frag(x, base, i);
                    const f32x4 old = acc[i];
#pragma unroll 1
                    for (int key = 0; key < kColBlock; ++key) {
                        const f32x4 z = G::add_block(
                            G::keep(all, [&](int j) { return has[j] >> key & 1; }), pb, old);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][r] = key == n ? z[r] : acc[i][r];
                    }
                }
            }
        }
    }
    if (col >= a.ncols) return;
    float f = (w & 1) ? 1.f / kProbScale<T> : a.s.scale;
    if constexpr (half) f = (w & 1) ? f : f / hs.s;
    const AttnRows& out = (w & 1) ? a.dv : a.dk;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
        const int d = (w >> 1) * (G::kDim / 2) + 16 * i + 4 * quad;
        if (!G::kFull && d >= a.s.dim) continue;
        const f32x4 z = acc[i] * f;
        if (pc.slot >= 0) {
            float* part = a.part_kv +
                          ((((int64_t)pc.slot * a.s.hkv + h) * kColBlock + n) * 2 + (w & 1)) * a.s.dim;
            *reinterpret_cast<f32x4*>(part + d) = z;
        } else {
            G::store_four(z, out.base + col * out.row + h * out.head + d * (int)sizeof(T));
        }
    }
}

// The sums of the rows, and of the blocks of columns, of more than one piece,
// in the pieces' order: one wavefront per row and head of dq, and per head,
// column and output of dk and dv. A piece's results lie side by side.
template <class T>
__global__ __launch_bounds__(kWaves* kWave) void k_attn_join_sum(BackwardArgs a) {
    int64_t unit = grid_block() * kWaves + threadIdx.x / kWave;
    const int64_t row_units = a.rows.nsplits * a.rows.block * a.s.hq;
    const bool col_side = unit >= row_units;
    if (col_side) unit -= row_units;
    const AttnSide& side = col_side ? a.cols : a.rows;
    const int64_t per = col_side ? (int64_t)a.s.hkv * 2 * kColBlock : (int64_t)side.block * a.s.hq;
    if (unit >= side.nsplits * per) return;
    const int64_t sp = unit / per, hl = unit - sp * per;
    const AttnSplit s = side.splits[sp];
    const int line = (int)(hl % (2 * kColBlock));
    const int h = (int)(col_side ? hl / (2 * kColBlock) : hl % a.s.hq);
    const int64_t row = col_side ? (int64_t)s.row * kColBlock + line / 2
                                 : (int64_t)s.row * side.block + hl / a.s.hq;
    if (row >= (col_side ? a.ncols : a.nrows)) return;
    const float* part = (col_side ? a.part_kv : a.part_q) + ((int64_t)s.slot * per + hl) * a.s.dim;
    const AttnRows& o = !col_side ? a.dq : line & 1 ? a.dv : a.dk;
    JoinedRow(part, per * a.s.dim, s.count, a.s.dim, [](int) { return 1.f; })
        .store<T>(o.base + row * o.row + h * o.head, 1.f, a.s.dim);
}

}  // namespace

void attention_backward(const BackwardArgs& a, hipStream_t st) {
    with_type(a.s.type, a.s.dim, [&](auto tag) {
        using Tag = decltype(tag);
        using T = typename Tag::Elem;
        if (a.rows.npieces > 0) {
            const int64_t heads = (int64_t)a.s.hkv * a.s.mtiles;
            const int each = pieces_per_wave(a.rows.npieces * heads);
            const int64_t groups = ceil_div(a.rows.npieces, kWaves * each);
            auto run = a.rows.block > 1 ? k_attn_grad_q<typename Tag::Geo, T, true>
                                        : k_attn_grad_q<typename Tag::Geo, T, false>;
            hipLaunchKernelGGL(run, grid_2d(xcd_grid(groups * heads)), dim3(kWaves * kWave),
                               0, st, a, each, groups);
            SG_LAUNCH_CHECK();
        }
        const int64_t cols = xcd_grid(a.cols.npieces) * a.s.hkv;
        if (cols > 0) {
            auto run = k_attn_grad_kv<typename Tag::Geo, T>;
            hipLaunchKernelGGL(run, grid_2d(cols), dim3(kKvWaves * kWave), 0, st, a);
            SG_LAUNCH_CHECK();
        }
        const int64_t joins = a.rows.nsplits * a.rows.block * a.s.hq +
                              a.cols.nsplits * a.s.hkv * 2 * kColBlock;
        if (joins > 0) {
            hipLaunchKernelGGL(k_attn_join_sum<T>, grid_2d(ceil_div(joins, kWaves)),
                               dim3(kWaves * kWave), 0, st, a);
            SG_LAUNCH_CHECK();
        }
    });
}

}  // namespace sg
