// Attention over a paged cache of latent vectors, in the latents' space
// (absorbed) or over keys and values that were made from them (expanded).
#include <algorithm>

#include "attention_join.h"
#include "latent.h"

namespace sg {

namespace {

// What places without a source read: as long as the longest row.
__device__ const u32x4 g_zero[SPGEMM_LATENT_MAX_DIM / 8 + SPGEMM_LATENT_MAX_ROPE / 8] = {};

typedef __attribute__((address_space(1))) const void GlobalBytes;
typedef __attribute__((address_space(3))) void LdsBytes;

// 16 bytes a lane from memory to LDS, lane after lane from `dst` on. (The
// restricted parameters keep reads of other LDS buffers from waiting for it.)
__device__ __forceinline__ void load_to_lds(const char* __restrict__ src, char* __restrict__ dst) {
    __builtin_amdgcn_global_load_lds((GlobalBytes*)src, (LdsBytes*)dst, 16, 0, 0);
}
// Everything that load_to_lds() of this wavefront asked for is there.
__device__ __forceinline__ void wait_for_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// A tile's rows in LDS: plane after plane of 64 values (128 bytes) of KEYS rows,
// which one load fills 8 rows at a time. A row's 16-byte pieces are exchanged
// by bits of its number, so that one piece of 16 rows in sequence, and two of
// every fourth row (the transposing read), fall on different banks.
template <int KEYS>
struct Planes {
    static constexpr int kPlane = KEYS * 128;
    static constexpr __device__ __forceinline__ int swap(int r) {
        return ((r >> 3) & 1) | ((r >> 1) & 1) << 1 | ((r >> 2) & 1) << 2;
    }
    static __device__ __forceinline__ int at(int r, int byte) {
        return (byte >> 7) * kPlane + r * 128 + ((byte & 127) ^ (swap(r) << 4));
    }
    // at(r | dr, byte | dbyte) from at(r, byte), for constants that share no bit
    // with r (whose exchanged bits they are none of) and byte
    static __device__ __forceinline__ int more(int base, int dr, int dbyte) {
        return (base ^ (dbyte & 127)) + (dbyte >> 7) * kPlane + dr * 128;
    }
    // an operand of 16 rows: 16 bytes, of step t, of row first + l % 16
    static __device__ __forceinline__ int row_base(int first, int lane) {
        return at(first + (lane & 15), 16 * (lane >> 4));
    }
    static __device__ __forceinline__ u32x4 row(const char* lds, int base, int dr, int t) {
        return *reinterpret_cast<const u32x4*>(lds + more(base, dr, 64 * t));
    }
    // 16 columns, block b's, of rows first + 4 (l / 16) + 0..3 and 16 more, turned over
    static __device__ __forceinline__ int value_base(int first, int lane) {
        const int l = lane & 15, quad = lane >> 4;
        return at(first + 4 * quad + (l >> 2), 8 * (l & 3));
    }
    static __device__ __forceinline__ u32x4 value(const char* lds, int base, int b) {
        using s16x4 = short __attribute__((ext_vector_type(4)));
        using lds_s16x4 = __attribute__((address_space(3))) s16x4;
        const u32x2 lo = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + more(base, 0, 32 * b))));
        const u32x2 hi = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + more(base, 16, 32 * b))));
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
};

// A lane's rows of a tile: of blocks of 8 rows first, first + 1, ... row l / 8, and
// of each the piece of 16 bytes that lies l % 8 places into LDS. Their pages are
// looked up a tile ahead; the rest is made anew from the lane for every tile, as
// registers are dearer than that.
template <class P, int BLOCKS>
struct TileRows {
    uint32_t id[BLOCKS] = {};
    bool wrong = false;
    static __device__ __forceinline__ int row(int lane, int block) { return 8 * block + (lane >> 3); }
    static __device__ __forceinline__ uint32_t byte(int lane, int block) {
        return 16 * ((lane & 7) ^ P::swap(row(lane, block)));
    }
    static __device__ __forceinline__ int anew(int lane) {
        asm volatile("" : "+v"(lane));
        return lane;
    }
    __device__ __forceinline__ void look_up(const PagedArgs& a, const int32_t* pages, int lane, int first,
                                            int t0, int k1) {
        lane = anew(lane);
#pragma unroll
        for (int i = 0; i < BLOCKS; ++i) {
            const int key = t0 + row(lane, first + i);
            if (key < k1) id[i] = (uint32_t)pages[a.page_div.div(key)];
        }
    }
    // The latent row of `key`, which is the i-th of this lane's in the tile; past
    // the end the row of zeros.
    __device__ __forceinline__ const char* latent(const PagedArgs& a, int key, int k1, int i) {
        if (id[i] >= (uint32_t)a.npages) {
            wrong |= key < k1;
            id[i] = 0;
        }
        const uint32_t slot = key - a.page_div.div(key) * a.page_div.d;
        const uint64_t at = (uint64_t)(id[i] * a.k_page + slot * a.k_slot) << a.k_shift;
        return key < k1 ? a.k + at : reinterpret_cast<const char*>(g_zero);
    }
};

// 16 bytes of a query row from byte `at` on, 0 past `end`. (Whatever is done with
// them waits for them: first all are asked for.)
__device__ __forceinline__ u32x4 load_query(const LatentArgs& a, const TileRow& r, int at, int end) {
    const char* row = a.q.base + r.token * a.q.row + r.hq * a.q.head;
    return *reinterpret_cast<const u32x4*>(
        r.has && at < end ? row + at : reinterpret_cast<const char*>(g_zero));
}
// Queries with the sign of the scores' factor (0: see Softmax).
template <class G>
__device__ __forceinline__ u32x4 sign_query(const LatentArgs& a, u32x4 q) {
    if (a.s.c < 0.f) return q ^ 0x80008000u;
    return u32x4{G::times0(q[0]), G::times0(q[1]), G::times0(q[2]), G::times0(q[3])};
}

// Weights are taken relative to a reference that only moves when a score
// passes it by more than 2^kSlack, which few tiles do: only then are sums
// rescaled. Half precision, whose range is short at both ends, holds them times
// 2^kShift. Products are rounded before the reference is subtracted, so that
// the difference is exact and the reference's own weight 1 for scores of any
// size.
constexpr float kSlack = 8.f;
template <class T>
constexpr float kShift = std::is_same<T, _Float16>::value ? 7.f : 0.f;
// (The difference, not the sum: where floats' steps are 16, ref + 8 may be ref + 16, and a
// weight of 2^16 passes half precision's range. Of two infinities it is a NaN: no.)
__device__ __forceinline__ bool passes(float ref, float top) { return top - ref > kSlack; }
// Moves a query's reference if its keys' largest score asks for it (whatever other
// queries ask for), and returns the factor of what was summed before.
__device__ __forceinline__ float move(float& ref, float top) {
    if (!passes(ref, top)) return 1.f;
    const float fix = fast_exp2(ref - top);
    ref = top;
    return fix;
}
__device__ __forceinline__ float weight_of(float s, float c, float ref, float shift) {
#pragma clang fp contract(off)
    const float x = s * c - ref;
    return fast_exp2(shift == 0.f ? x : x + shift);
}

// Keys that not all rows of a work group see. An infinity or a NaN in one's value
// must not reach a row that does not see it as 0 times it: in the tiles that
// hold such keys those elements are made 0 in LDS, and at the end they are added
// to the rows that see their keys, times their weights: any weight gives the element
// itself but that of a score of -infinity, which is 0 and gives NaN. (So does a weight
// that its type rounds to 0, in the tiles that all rows see.)
template <int KEYS, int ROWS>
struct Crossing {
    static constexpr int kKeys = KEYS, kTiles = ROWS / KEYS + 2;
    int from;  // the first such tile's first key
    __device__ __forceinline__ Crossing(const TileJob& j, int first_token)
        : from(j.k0 + max(j.before + first_token - j.k0, 0) / kKeys * kKeys) {}
    // Clears such elements of this thread's row of the planes at `vals` (8 threads
    // to a row); whether there were any.
    template <class G, int THREADS>
    static __device__ __forceinline__ bool clear(char* vals, int planes) {
        static_assert(THREADS == 8 * KEYS, "a thread stays with its row");
        bool any = false;
#pragma unroll 1
        for (int g = 0; g < planes; ++g) {
            char* at = vals + g * KEYS * 128 + 16 * threadIdx.x;
            u32x4 x = *reinterpret_cast<const u32x4*>(at);
            const uint32_t words[4] = {x[0], x[1], x[2], x[3]};
            if (!G::words_wild(words)) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t low[1] = {x[i] & 0xffffu}, high[1] = {x[i] & 0xffff0000u};
                x[i] &= (G::words_wild(low) ? 0u : 0xffffu) | (G::words_wild(high) ? 0u : 0xffff0000u);
            }
            *reinterpret_cast<u32x4*>(at) = x;
            any = true;
        }
        return any;
    }
    // All threads' rows, from bit i of `mine` for the i-th such tile, in LDS that
    // is not used otherwise any more.
    static __device__ __forceinline__ void gather(uint32_t mine, unsigned long long* wild) {
        if (threadIdx.x < kTiles) wild[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
            if (mine >> i & 1) atomicOr(&wild[i], 1ull << (threadIdx.x / 8));
        __syncthreads();
    }
    // o plus the elements that are not finite of the keys below `sees` that were
    // cleared; row(key): where the key's values of o begin, weight(key): 0 if its
    // weight is, else 1.
    template <class T, int NB, class Row, class Weight>
    __device__ __forceinline__ void add(const unsigned long long* wild, int sees, int dim, Row&& row,
                                        Weight&& weight, f32x4 (&o)[NB]) const {
#pragma unroll 1
        for (int i = 0; i < kTiles; ++i)
#pragma unroll 1
            for (uint64_t m = wild[i]; m; m &= m - 1) {
                const int key = from + kKeys * i + __builtin_ctzll(m);
                if (key >= sees) break;
                const char* at = row(key);
                if (!at) break;
                const float w = weight(key);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (16 * b + 4 * (lane_id() >> 4) >= dim) continue;
                    const u32x2 x = *reinterpret_cast<const u32x2*>(at + 32 * b + 8 * (lane_id() >> 4));
                    float y[4];
                    unpack2<T>(x[0], y[0], y[1]);
                    unpack2<T>(x[1], y[2], y[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[b][j] += __builtin_isfinite(y[j]) ? 0.f : y[j] * w;
                }
            }
    }
};

// ---------------------------------------------------------------- absorbed
// Keys of up to DK and values of up to DV elements, a value the first part of its
// key. A team of KH * DH wavefronts takes 32 rows. For the scores they cut a tile's
// keys in KH and the sum over its elements in DH (2: whole queries of 576 elements
// leave no registers to read keys ahead; partial sums go through LDS), for the
// result its columns in KH * DH.
// FULL: the keys have DK elements, so that no piece of theirs needs a check (the
// time below; with the checks 179 us).
//
// A token's row is read once from memory for all heads and serves both products.
// At 128 heads bytes and products take about as long (70 and 54 us for the next token
// of 32 texts of up to 16384, rows of 512 + 64): 164 us, 2.0 TB/s and 470 TFLOP/s. A
// tile of 64 keys takes 7500 cycles, its bytes 4900: scores 1400, their exchange 1500,
// weights 700, a barrier 800, results 2100, with one work group per compute unit (its
// two tiles fill LDS), so that these follow each other. Two tiles a step would need
// LDS twice.
template <class T, int DK, int DV, int KH_, int DH_, bool FULL>
struct AbsorbedGeo : Tile<T, 64, true> {
    static constexpr bool kWhole = FULL;
    static constexpr int kKeys = kAbsorbedKeys, kDv = DV, kPlanes = DK / 64;
    static constexpr int KH = KH_, DH = DH_, CG = KH * DH, NW = 8, QB = 2, BM = NW / CG * 16 * QB;
    static constexpr int QS = DK / 32 / DH, NB = DV / 16 / CG;
    static constexpr int KS = kKeys / 16 / KH;  // 16-key blocks of a wavefront's products,
    static constexpr int FB = KS / DH;          // and of those those whose weights it makes
    // Planes of the next tile that are asked for during the scores' products, around
    // the weights and during the results' products. A compute unit has some 12 KB
    // under way at once, and further loads stop the wavefront that asks: spread
    // over the tile's time they do not.
    static constexpr int kLoad0 = (4 * kPlanes + 8) / 9, kLoad1 = kLoad0 + (kPlanes - kLoad0 + 3) / 4,
                         kLoad2 = kLoad1 + (kPlanes - kLoad1 + 2) / 4;
    // what a wavefront is sent and leaves in LDS: partial sums, then weights,
    // largest scores and a flag
    static constexpr int kTops = QB * FB * kWave * 8, kFlag = kTops + QB * 64;
    static constexpr int kSlot = DH == 2 ? QB * FB * kWave * 16 : kFlag + 64;
    static_assert(BM <= kPagedTileMost, "the limit of rows counts on it");
    static_assert(DK % (32 * DH) == 0 && DV % (64 * CG) == 0 && KS >= DH && DH <= 2, "tile shape");
    static_assert(kFlag + 4 <= kSlot && kKeys == 8 * NW && 2 * (kPlanes - kLoad2) <= NB + 1,
                  "slots and loads");
};

template <class G, class T>
__global__ __launch_bounds__(G::NW* kWave) void k_absorbed(LatentArgs a, int32_t tiles) {
    constexpr int QB = G::QB, QS = G::QS, NB = G::NB, NW = G::NW, CG = G::CG, KS = G::KS, FB = G::FB;
    constexpr int kKeys = G::kKeys;
    using Pl = Planes<kKeys>;
    using Cr = Crossing<kKeys, G::BM>;
    __shared__ __align__(16) char tile0[G::kPlanes * Pl::kPlane];
    __shared__ __align__(16) char tile1[G::kPlanes * Pl::kPlane];
    __shared__ __align__(16) char slots[NW * G::kSlot];
    int64_t unit = xcd_block();
    if (unit >= (a.ranges ? a.ranges : a.seqs) * (int64_t)tiles) return;
    const int tile = tiles - 1 - (int)(unit % tiles);  // the longest first
    unit /= tiles;
    // a sequence, or a range of all of them
    int s = (int)unit, before = 0, pos = 0, end = 0, begin = 0;
    if (a.ranges) {
        const EvenSplit<kAbsorbedEvenSeqs> e(a, kKeys);
        begin = pos = (int)min(unit * e.per, (int64_t)e.total);
        end = min(pos + e.per, e.total);
        if (pos >= end) return;
        e.locate(pos, s, before);
    }
#pragma unroll 1
    for (;; ++s) {  // segments
        // Nothing that is made from the lane is kept from one segment to the next:
        // it would take the loop's registers.
        int zero_here = 0;
        asm volatile("" : "+s"(zero_here));
        const int tid = threadIdx.x + zero_here, lane = tid & (kWave - 1);
        const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
        const int team = w / CG, part = w % CG, kh = part / G::DH, dh = part % G::DH;
        TileJob job;
        job.sq = read_sequence(a, s);
        job.rows = job.sq.fresh * a.s.group;
        job.first = tile * G::BM;
        job.idle = job.sq.none || job.first >= job.rows;
        job.before = job.sq.length - job.sq.fresh + 1;
        job.k0 = 0;
        job.k1 = job.before + (min(job.first + G::BM, job.rows) - 1) / a.s.group;
        const bool late = pos > begin;
        bool split = false;
        if (a.ranges) {
            const int own =
                job.sq.none ? 0 : job.sq.bad ? 1 : (job.sq.length + kKeys - 1) / kKeys;
            split = pos > before || before + own > end;
            job.k0 = (pos - before) * kKeys;
            job.k1 = min(job.k1, (int)min((int64_t)(end - before) * kKeys, (int64_t)INT32_MAX));
            before += own;
            pos = before;
        }
        const auto segment = [&] {
            if (job.idle) return;
            const int n = lane & 15;
            const int row0 = job.first + 16 * QB * team;  // the team's first row
            TileRow r[QB];
#pragma unroll
            for (int b = 0; b < QB; ++b) r[b] = tile_row(a, job, row0 + 16 * b + n, 0);
            if (job.sq.bad) {
                if (part == 0)
#pragma unroll
                    for (int b = 0; b < QB; ++b) store_nan<T>(a, r[b]);
                return;
            }
            if (job.k0 >= job.k1) return;
            const Cr cross(job, job.first / a.s.group);
            const int lo = __builtin_amdgcn_readfirstlane(r[0].t);
            const int hi = __builtin_amdgcn_readlane(r[QB - 1].t, 15);
            const int mine = row0 < job.rows ? min(job.k1, job.before + hi) : 0;  // some row sees
            const int full = min(job.k1, job.before + lo);                       // all rows see

            const int32_t* pages = a.col + job.sq.page0;
            TileRows<Pl, 1> from;
            from.look_up(a, pages, lane, w, job.k0, job.k1);
            u32x4 q[QB][QS];
#pragma unroll
            for (int x = 0; x < QB; ++x)
#pragma unroll
                for (int t = 0; t < QS; ++t)
                    q[x][t] = load_query(a, r[x], 64 * (QS * dh + t) + 16 * (lane >> 4), 2 * a.key_dim);
            // this lane's row of a tile, and what it loads of plane g of it
            const char* row = nullptr;
            uint32_t byte = 0;
            const auto open_tile = [&](int t0) {
                const int l = from.anew(lane);
                byte = from.byte(l, w);
                row = from.latent(a, t0 + from.row(l, w), job.k1, 0) + byte;
            };
            const auto load_plane = [&](char* dst, int g) {
                load_to_lds(G::kWhole || 128 * g + (int)byte < 2 * a.key_dim
                                ? row + 128 * g
                                : reinterpret_cast<const char*>(g_zero),
                            dst + g * Pl::kPlane + w * 1024);
            };
            open_tile(job.k0);
#pragma unroll
            for (int g = 0; g < G::kPlanes; ++g) load_plane(tile0, g);
            from.look_up(a, pages, lane, w, job.k0 + kKeys, job.k1);
            if (a.s.c <= 0.f)
#pragma unroll
                for (int x = 0; x < QB; ++x)
#pragma unroll
                    for (int t = 0; t < QS; ++t) q[x][t] = sign_query<G>(a, q[x][t]);
            f32x4 o[QB][NB];
            float ref[QB], sum[QB];  // ref: of this lane's query, in the whole team; sum: its own
#pragma unroll
            for (int x = 0; x < QB; ++x) {
                ref[x] = -INFINITY;
                sum[x] = 0.f;
#pragma unroll
                for (int b = 0; b < NB; ++b) o[x][b] = f32x4{0, 0, 0, 0};
            }
            uint32_t wild = 0;  // see Crossing
            char* const mail = slots + w * G::kSlot;
            wait_for_loads();
            __syncthreads();

            // One tile of keys, staged in `rows`; the next one is loaded into `next`.
            const auto take = [&](char* rows, char* next, int t0) {
                // (past the end it loads zeros: the loads go between the products,
                // as memory takes them no faster)
                open_tile(t0 + kKeys);
                from.look_up(a, pages, lane, w, t0 + 2 * kKeys, job.k1);
                const bool active = t0 < mine;
                f32x4 sc[QB][KS];  // of the lane's query and its 4 keys of every block
                if (active) {
                    const int rb = Pl::row_base(16 * KS * kh, lane);
#pragma unroll
                    for (int x = 0; x < QB; ++x)
#pragma unroll
                        for (int b = 0; b < KS; ++b) sc[x][b] = f32x4{0, 0, 0, 0};
                    const auto products = [&](auto half) {
                        constexpr int kFrom = decltype(half)::value * QS;
                        // keys are read kAhead steps before their products, a plane of
                        // the next tile is asked for between; left to the compiler, every
                        // product waits for its own read
                        constexpr int kAhead = 2;
                        u32x4 k[kAhead + 1][KS];
                        const auto read = [&](int i) {
#pragma unroll
                            for (int b = 0; b < KS; ++b)
                                k[i % (kAhead + 1)][b] = Pl::row(rows, rb, 16 * b, kFrom + i);
                        };
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) read(i);
#pragma unroll
                        for (int i = 0; i < QS; ++i) {
                            __builtin_amdgcn_sched_barrier(0);
                            if (i + kAhead < QS) read(i + kAhead);
#pragma unroll
                            for (int g = 0; g < G::kLoad0; ++g)
                                if (g * QS / G::kLoad0 == i) load_plane(next, g);
#pragma unroll
                            for (int b = 0; b < KS; ++b)
#pragma unroll
                                for (int x = 0; x < QB; ++x)
                                    sc[x][b] = mfma32<T>(k[i % (kAhead + 1)][b], q[x][i], sc[x][b]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    };
                    if (G::DH == 1 || dh == 0) products(std::integral_constant<int, 0>{});
                    else products(std::integral_constant<int, G::DH - 1>{});
                } else {
#pragma unroll
                    for (int g = 0; g < G::kLoad0; ++g) load_plane(next, g);
                }
                if constexpr (G::DH == 2) {
                    // the other half's sums of the blocks whose weights it makes
                    char* const out = slots + (w ^ 1) * G::kSlot;
                    if (active)
#pragma unroll
                        for (int x = 0; x < QB; ++x)
#pragma unroll
                            for (int f = 0; f < FB; ++f)
                                *reinterpret_cast<f32x4*>(out + ((x * FB + f) * kWave + lane) * 16) =
                                    dh == 0 ? sc[x][FB + f] : sc[x][f];
                    __syncthreads();
                    if (active)
#pragma unroll
                        for (int x = 0; x < QB; ++x)
#pragma unroll
                            for (int f = 0; f < FB; ++f) {
                                const f32x4 y = *reinterpret_cast<const f32x4*>(
                                    mail + ((x * FB + f) * kWave + lane) * 16);
                                sc[x][f] = (dh == 0 ? sc[x][f] : sc[x][FB + f]) + y;
                            }
                }
                const int first = t0 + 16 * (KS * kh + FB * dh);  // the blocks' first key
                float top[QB], add[QB];
                const auto put_probs = [&] {
#pragma unroll
                    for (int x = 0; x < QB; ++x) {
                        add[x] = 0.f;
                        const float base = ref[x] == -INFINITY ? 0.f : ref[x];
#pragma unroll
                        for (int f = 0; f < FB; ++f) {
                            float p[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                p[j] = weight_of(sc[x][f][j], a.s.mag, base, kShift<T>);
                                add[x] += p[j];
                            }
                            *reinterpret_cast<u32x2*>(mail + ((x * FB + f) * kWave + lane) * 8) =
                                u32x2{pack2<T>(p[0], p[1]), pack2<T>(p[2], p[3])};
                        }
                    }
                };
#pragma unroll
                for (int g = G::kLoad0; g < G::kLoad1; ++g) load_plane(next, g);
                bool raise = false;
                if (active) {
#pragma unroll
                    for (int x = 0; x < QB; ++x) {
                        if (first + 16 * FB > full) {  // some row does not see some key
                            const int row = min(row0 + 16 * x + n, job.rows - 1);
                            const int sees = job.before + (int)a.group_div.div(row);
                            const Seen seen = Seen::first(min(job.k1, sees) - first);
#pragma unroll
                            for (int j = 0; j < 4 * FB; ++j)
                                sc[x][j >> 2][j & 3] = seen.pick(j, sc[x][j >> 2][j & 3], -INFINITY);
                        }
                        top[x] = sc[x][0][0];
#pragma unroll
                        for (int j = 1; j < 4 * FB; ++j) top[x] = fmaxf(top[x], sc[x][j >> 2][j & 3]);
                        top[x] *= a.s.mag;
                        raise |= passes(ref[x], top[x]);
                    }
                    put_probs();
                }
                const bool raised = __any(raise);
                if (lane == 0) *reinterpret_cast<int*>(mail + G::kFlag) = raised;
                __syncthreads();
                const int flag =
                    *reinterpret_cast<const int*>(slots + (lane % NW) * G::kSlot + G::kFlag);
#pragma unroll
                for (int g = G::kLoad1; g < G::kLoad2; ++g) load_plane(next, g);
                if (__any(flag != 0)) {  // hardly ever after the first tiles
                    if (active) {
#pragma unroll
                        for (int x = 0; x < QB; ++x) {
                            top[x] = quad_max(top[x]);
                            if (lane < 16)
                                *reinterpret_cast<float*>(mail + G::kTops + 64 * x + 4 * lane) = top[x];
                        }
                    }
                    __syncthreads();
                    if (active) {
#pragma unroll
                        for (int x = 0; x < QB; ++x) {
#pragma unroll
                            for (int c = 0; c < CG; ++c)
                                top[x] = fmaxf(top[x], *reinterpret_cast<const float*>(
                                                           slots + (team * CG + c) * G::kSlot +
                                                           G::kTops + 64 * x + 4 * n));
                            const float fix = move(ref[x], top[x]);
                            sum[x] *= fix;
#pragma unroll
                            for (int b = 0; b < NB; ++b) o[x][b] *= fix;
                        }
                        put_probs();
                    }
                    __syncthreads();
                }
                if (min(t0 + kKeys, job.k1) > job.before + job.first / a.s.group) {
                    const bool any = Cr::template clear<G, NW * kWave>(rows, G::kDv / 64);
                    wild |= (uint32_t)any << ((t0 - cross.from) / kKeys);
                    __syncthreads();
                }
                if (active) {
#pragma unroll
                    for (int x = 0; x < QB; ++x) sum[x] += add[x];
                    const char* vals = rows + part * (G::kDv / 64 / CG) * Pl::kPlane;
#pragma unroll
                    for (int j = 0; j < kKeys / 32; ++j) {
                        typename G::Probs pr[QB];
#pragma unroll
                        for (int x = 0; x < QB; ++x)
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                // block 2 j + b: where its weights were left
                                const int block = 2 * j + b, maker = block / FB, f = block % FB;
                                const u32x2 p = *reinterpret_cast<const u32x2*>(
                                    slots + (team * CG + maker) * G::kSlot +
                                    ((x * FB + f) * kWave + lane) * 8);
                                pr[x].w[2 * b] = p[0];
                                pr[x].w[2 * b + 1] = p[1];
                            }
                        const int vb = Pl::value_base(32 * j, lane);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const u32x4 v = Pl::value(vals, vb, b);
#pragma unroll
                            for (int g = G::kLoad2; g < G::kPlanes; ++g)
                                if (j == 0 && 2 * (g - G::kLoad2) == b) load_plane(next, g);
#pragma unroll
                            for (int x = 0; x < QB; ++x) o[x][b] = G::add_block(v, pr[x], o[x][b]);
                        }
                    }
                } else {
#pragma unroll
                    for (int g = G::kLoad2; g < G::kPlanes; ++g) load_plane(next, g);
                }
                wait_for_loads();
                __syncthreads();  // the next tile is there, this one's readers are done
            };
            for (int t0 = job.k0; t0 < job.k1; t0 += 2 * kKeys) {
                take(tile0, tile1, t0);
                if (t0 + kKeys < job.k1) take(tile1, tile0, t0 + kKeys);
            }
            auto* const wild_s = reinterpret_cast<unsigned long long*>(tile0);
            const bool crossed = job.k1 > job.before + job.first / a.s.group;
            if (crossed) Cr::gather(wild, wild_s);
#pragma unroll
            for (int x = 0; x < QB; ++x) {
                sum[x] = quad_sum(sum[x]);
                if (lane < 16) *reinterpret_cast<float*>(mail + G::kTops + 64 * x + 4 * lane) = sum[x];
            }
            const bool wrong = __any(from.wrong);
            if (lane == 0) *reinterpret_cast<int*>(mail + G::kFlag) = wrong;
            __syncthreads();
            if (row0 >= job.rows) return;
            const int flag = *reinterpret_cast<const int*>(slots + (lane % NW) * G::kSlot + G::kFlag);
            const bool any_wrong = __any(flag != 0);
            // the rows again: kept, they would take registers from the loop
            int again = row0;
            asm volatile("" : "+s"(again));
#pragma unroll
            for (int x = 0; x < QB; ++x) {
                r[x] = tile_row(a, job, again + 16 * x + n, 0);
                const int sees = job.before + r[x].t;
                if (!r[x].has || sees <= job.k0) continue;
                float l = 0.f;
#pragma unroll
                for (int c = 0; c < CG; ++c)
                    l += *reinterpret_cast<const float*>(slots + (team * CG + c) * G::kSlot +
                                                         G::kTops + 64 * x + 4 * n);
                if (any_wrong) l = NAN;
                const int64_t line = r[x].token * a.s.hq + r[x].hq;
                // where a part of a split sequence goes
                const int64_t at =
                    ((2 * unit + late) * tiles + tile) * G::BM + again - job.first + 16 * x + n;
                const float f = l == 0.f ? 0.f : 1.f / l;
                if (crossed)
                    cross.template add<T>(
                        wild_s, min(job.k1, sees), a.s.dim - part * (G::kDv / CG),
                        [&](int key) -> const char* {
                            const uint32_t pg = a.page_div.div(key), id = (uint32_t)pages[pg];
                            if (id >= (uint64_t)a.npages) return nullptr;
                            const uint32_t slot = key - pg * a.page_div.d;
                            return a.k + ((uint64_t)(id * a.k_page + slot * a.k_slot) << a.k_shift) +
                                   part * (2 * G::kDv / CG);
                        },
                        // (The element is one of the key's too: its score is an infinity or
                        // a NaN, and but for -infinity the row's sum is NaN anyway.)
                        [](int) { return 0.f; }, o[x]);
                char* row = !split ? a.out.base + r[x].token * a.out.row + r[x].hq * a.out.head
                                   : reinterpret_cast<char*>(a.part + at * a.s.dim);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int d = part * (G::kDv / CG) + 16 * b + 4 * (lane >> 4);
                    if (d >= a.s.dim) continue;
                    if (!split)
                        G::store_four(o[x][b] * f, row + 2 * d);
                    else
                        *reinterpret_cast<f32x4*>(row + 4 * d) = o[x][b];
                }
                if (part == 0 && lane < 16) {
                    if (split) {
                        a.part_ml[2 * at] = ref[x];
                        a.part_ml[2 * at + 1] = l;
                    } else if (a.lse) {
                        a.lse[line] =
                            l == 0.f ? -INFINITY : (ref[x] - kShift<T> + fast_log2(l)) * kLn2;
                    }
                }
            }
        };
        segment();
        if (pos >= end) return;
        __syncthreads();  // what is in LDS is used again
    }
}

// ---------------------------------------------------------------- expanded
// Keys and values of one head that k_expand made, of up to 64 MP and 64 VP
// elements, each as two numbers of the type that add up to it: rounded to one,
// a key's error would be that of the scores, and so of the log-sum-exp, and a
// value's as large as the result's own rounding. The keys' last part, of up to
// 64 elements, is the latent row's. A wavefront takes QB blocks of 16 rows.
// Bound by the products, 1.8 times the formula's for the second numbers: chunks of
// 2048 of two texts of up to 16384, 32 heads of 128 + 64 and 128, bfloat16, 1290 us,
// some 920 TFLOP/s with them; the matrix units are busy for half of the time, softmax
// and the exchange of tiles take the other.
template <class T, int MP_, int VP_, int NW_>
struct ExpandedGeo : Tile<T, 64, true> {
    static constexpr int NW = NW_, QB = 2, BM = NW * 16 * QB, kKeys = 8 * NW;
    static constexpr int MP = MP_, VP = VP_, QS = 2 * MP + 2, NB = 4 * VP;
    static constexpr int kLow = MP, kRope = 2 * MP, kValues = kRope + 1, kPlanes = kValues + 2 * VP;
    static_assert(kKeys % 32 == 0, "tile shape");
};

template <class G, class T>
__global__ __launch_bounds__(G::NW* kWave, 2) void k_expanded(LatentArgs a, int32_t tiles) {
    constexpr int QB = G::QB, QS = G::QS, NB = G::NB, NW = G::NW, kKeys = G::kKeys;
    using Pl = Planes<kKeys>;
    using Cr = Crossing<kKeys, G::BM>;
    __shared__ __align__(16) char tile0[G::kPlanes * Pl::kPlane];
    __shared__ __align__(16) char tile1[G::kPlanes * Pl::kPlane];
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
    const TileJob job = tile_job(a, s, tile, G::BM, piece);
    if (job.idle) return;
    const int n = lane & 15;
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
    if (tid == 0) wrong_s = 0;
    uint32_t wild = 0;  // see Crossing
    const Cr cross(job, job.first);
    const int lo = __builtin_amdgcn_readfirstlane(r[0].t);
    const int hi = __builtin_amdgcn_readlane(r[QB - 1].t, 15);
    const int mine = row0 < job.rows ? min(job.k1, job.before + hi) : 0;  // some row sees
    const int full = min(job.k1, job.before + lo);                       // all rows see

    u32x4 q[QB][QS];
    f32x4 o[QB][NB];
    float ref[QB], sum[QB];
    const int made = 2 * a.made_dim, values = 2 * a.s.dim;  // bytes
#pragma unroll
    for (int x = 0; x < QB; ++x) {
        ref[x] = -INFINITY;
        sum[x] = 0.f;
#pragma unroll
        for (int t = 0; t < QS; ++t) {
            const int at = 64 * t + 16 * (lane >> 4), rope = at - 128 * G::MP;
            q[x][t] = t < 2 * G::MP ? load_query(a, r[x], at, made)
                                    : load_query(a, r[x], made + rope, 2 * a.key_dim);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) o[x][b] = f32x4{0, 0, 0, 0};
    }
    if (a.s.c <= 0.f)
#pragma unroll
        for (int x = 0; x < QB; ++x)
#pragma unroll
            for (int t = 0; t < QS; ++t) q[x][t] = sign_query<G>(a, q[x][t]);
    const int32_t* pages = a.col + job.sq.page0;
    // the sequence's first row of made keys and values
    const int64_t made0 = h * a.made_rows +
                          (a.made_step ? s * a.made_step : job.sq.page0 * (int64_t)a.page_div.d);
    const char* made_k = a.made_k + made0 * 2 * made;
    const char* made_v = a.made_v + made0 * 2 * values;
    TileRows<Pl, 1> from;
    const uint32_t byte = from.byte(lane, w), trow = from.row(lane, w);
    // what this lane loads of plane g of a tile: its row's sources
    const char* zero = reinterpret_cast<const char*>(g_zero);
    const char *ksrc = zero, *vsrc = zero, *rsrc = zero;
    bool in = false;
    const auto open_tile = [&](int t0) {
        const int64_t key = t0 + (int)trow;
        in = key < job.k1;
        ksrc = made_k + key * 2 * made + byte;
        vsrc = made_v + key * 2 * values + byte;
        rsrc = from.latent(a, (int)key, job.k1, 0) + a.rope_at + byte;
    };
    const auto load_plane = [&](char* dst, int g) {
        char* to = dst + g * Pl::kPlane + w * 1024;
        if (g < G::kRope) {
            const bool low = g >= G::MP;
            const int at = 128 * (low ? g - G::MP : g);
            load_to_lds(in && at + (int)byte < made ? ksrc + (low ? made : 0) + at : zero, to);
        } else if (g == G::kRope) {
            load_to_lds(in && made + (int)byte < 2 * a.key_dim ? rsrc : zero, to);
        } else {
            const bool low = g >= G::kValues + G::VP;
            const int at = 128 * (low ? g - G::kValues - G::VP : g - G::kValues);
            load_to_lds(in && at + (int)byte < values ? vsrc + (low ? values : 0) + at : zero, to);
        }
    };
    from.look_up(a, pages, lane, w, job.k0, job.k1);
    __syncthreads();  // the flags
    open_tile(job.k0);
#pragma unroll
    for (int g = 0; g < G::kPlanes; ++g) load_plane(tile0, g);
    from.look_up(a, pages, lane, w, job.k0 + kKeys, job.k1);
    wait_for_loads();
    __syncthreads();

    const int rb = Pl::row_base(0, lane), vb = Pl::value_base(0, lane);
    // One tile of keys, staged in `rows`; the next one is loaded into `next`.
    const auto take = [&](char* rows, char* next, int t0) {
        char* vals = rows + G::kValues * Pl::kPlane;
        // (past the end it loads zeros)
        open_tile(t0 + kKeys);
        from.look_up(a, pages, lane, w, t0 + 2 * kKeys, job.k1);
        if (min(t0 + kKeys, job.k1) > job.before + job.first) {
            const bool any = Cr::template clear<G, NW * kWave>(vals, G::VP);
            wild |= (uint32_t)any << ((t0 - cross.from) / kKeys);
            __syncthreads();
        }
        // 32 keys, from staged row `at` on; the next tile is asked for during the first
        // step's products: the scores', and of several steps the results' too
        const auto step_of = [&](int at, auto loads) {
            constexpr bool kLoads = decltype(loads)::value;
            constexpr int kFirst = kKeys > 32 ? (G::kPlanes + 1) / 2 : G::kPlanes;
            const int t = t0 + at;
            if (t >= mine) {
                if (kLoads)
#pragma unroll
                    for (int g = 0; g < G::kPlanes; ++g) load_plane(next, g);
                return;
            }
            const char* krows = rows + at * 128;
            const char* vrows = vals + at * 128;
            f32x4 sc[QB][2];
#pragma unroll
            for (int x = 0; x < QB; ++x) sc[x][0] = sc[x][1] = f32x4{0, 0, 0, 0};
            // the keys' low parts first; read kAhead steps before their products, as in
            // k_absorbed
            constexpr int kSteps = 4 * G::MP + 2, kAhead = 2;
            u32x4 k[kAhead + 1][2];
            const auto step = [&](int i) {
                return i < 2 * G::MP ? i + 2 * G::MP : i < 4 * G::MP ? i - 2 * G::MP : i;
            };
            const auto read = [&](int i) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    k[i % (kAhead + 1)][b] = Pl::row(krows, rb, 16 * b, step(i));
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) read(i);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                if (i + kAhead < kSteps) read(i + kAhead);
                if (kLoads)
#pragma unroll
                    for (int g = 0; g < kFirst; ++g)
                        if (g * kSteps / kFirst == i) load_plane(next, g);
                const int part = step(i) < 2 * G::MP ? step(i) : step(i) - 2 * G::MP;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int x = 0; x < QB; ++x)
                        sc[x][b] = mfma32<T>(k[i % (kAhead + 1)][b], q[x][part], sc[x][b]);
            }
            __builtin_amdgcn_sched_barrier(0);
            bool raise = false;
            float top[QB];
#pragma unroll
            for (int x = 0; x < QB; ++x) {
                if (t + 32 > full)  // some row does not see some key
                    Softmax<G, T>::hide(sc[x], Seen::first(min(job.k1, job.before + r[x].t) - t));
                top[x] = sc[x][0][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) top[x] = fmaxf(top[x], sc[x][j >> 2][j & 3]);
                top[x] *= a.s.mag;
                raise |= passes(ref[x], top[x]);
            }
            if (__any(raise)) {  // hardly ever after the first tiles
#pragma unroll
                for (int x = 0; x < QB; ++x) {
                    const float fix = move(ref[x], quad_max(top[x]));
                    sum[x] *= fix;
#pragma unroll
                    for (int b = 0; b < NB; ++b) o[x][b] *= fix;
                }
            }
            typename G::Probs pr[QB];
#pragma unroll
            for (int x = 0; x < QB; ++x) {
                float p[8];
                const float base = ref[x] == -INFINITY ? 0.f : ref[x];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    p[j] = weight_of(sc[x][j >> 2][j & 3], a.s.mag, base, kShift<T>);
                    sum[x] += p[j];
                }
                G::pack_probs(p, pr[x]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const u32x4 low = Pl::value(vrows + G::VP * Pl::kPlane, vb, b);
                const u32x4 high = Pl::value(vrows, vb, b);
                if (kLoads)
#pragma unroll
                    for (int g = kFirst; g < G::kPlanes; ++g)
                        if ((g - kFirst) * NB / (G::kPlanes - kFirst + 1) == b) load_plane(next, g);
#pragma unroll
                for (int x = 0; x < QB; ++x) o[x][b] = G::add_block(low, pr[x], o[x][b]);
#pragma unroll
                for (int x = 0; x < QB; ++x) o[x][b] = G::add_block(high, pr[x], o[x][b]);
            }
        };
        step_of(0, std::true_type{});
#pragma unroll 1
        for (int at = 32; at < kKeys; at += 32) step_of(at, std::false_type{});
        wait_for_loads();
        __syncthreads();  // the next tile is there, this one's readers are done
    };
    for (int t0 = job.k0; t0 < job.k1; t0 += 2 * kKeys) {
        take(tile0, tile1, t0);
        if (t0 + kKeys < job.k1) take(tile1, tile0, t0 + kKeys);
    }
    if (from.wrong) wrong_s = 1;
    auto* const wild_s = reinterpret_cast<unsigned long long*>(tile0);
    const bool crossed = job.k1 > job.before + job.first;
    if (crossed) Cr::gather(wild, wild_s);
    else __syncthreads();
    if (row0 >= job.rows) return;
    // The score (before its factor's size) of the lane's query x and a key, without
    // the key's low parts: whether it is -infinity.
    const auto score_of = [&](int x, int key) {
        const uint32_t pg = a.page_div.div(key), id = (uint32_t)pages[pg];
        const char* row = id < (uint64_t)a.npages
                              ? a.k + ((uint64_t)(id * a.k_page + (key - pg * a.page_div.d) * a.k_slot)
                                       << a.k_shift)
                              : zero;
        float y = 0.f;
#pragma unroll 1
        for (int t = 0; t < QS; ++t) {
            u32x4 qt = q[x][0];
#pragma unroll
            for (int i = 1; i < QS; ++i) qt = i == t ? q[x][i] : qt;
            const int at = 64 * t + 16 * (lane >> 4), rope = at - 128 * G::MP;
            const char* from = rope < 0 ? made_k + (int64_t)key * 2 * made + at : row + a.rope_at + rope;
            const bool has = rope < 0 ? at < made : made + rope < 2 * a.key_dim;
            const u32x4 kt = *reinterpret_cast<const u32x4*>(has ? from : zero);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float q0, q1, k0, k1;
                unpack2<T>(qt[i], q0, q1);
                unpack2<T>(kt[i], k0, k1);
                y = fmaf(q1, k1, fmaf(q0, k0, y));
            }
        }
        y += __shfl_xor(y, 16, kWave);
        return y + __shfl_xor(y, 32, kWave);
    };
#pragma unroll
    for (int x = 0; x < QB; ++x) {
        const int sees = job.before + r[x].t;
        const float all = quad_sum(sum[x]);
        if (!r[x].has || sees <= job.k0) continue;
        const float l = wrong_s ? NAN : all;
        const int64_t line = r[x].token * a.s.hq + r[x].hq;
        const bool part = sees > a.piece;
        const int64_t at = (int64_t)piece * a.tokens * a.s.hq + line;
        const float f = l == 0.f ? 0.f : 1.f / l;
        if (crossed)
            cross.template add<T>(
                wild_s, min(job.k1, sees), a.s.dim,
                [&](int key) { return made_v + (int64_t)key * 2 * values; },
                [&](int key) { return score_of(x, key) == -INFINITY ? 0.f : 1.f; }, o[x]);
        char* row = part ? reinterpret_cast<char*>(a.part + at * a.s.dim)
                         : a.out.base + r[x].token * a.out.row + r[x].hq * a.out.head;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int d = 16 * b + 4 * (lane >> 4);
            if (d >= a.s.dim) continue;
            if (part)
                *reinterpret_cast<f32x4*>(row + 4 * d) = o[x][b];
            else
                G::store_four(o[x][b] * f, row + 2 * d);
        }
        if (lane < 16) {
            if (part) {
                a.part_ml[2 * at] = ref[x];
                a.part_ml[2 * at + 1] = l;
            } else if (a.lse) {
                a.lse[line] = l == 0.f ? -INFINITY : (ref[x] - kShift<T> + fast_log2(l)) * kLn2;
            }
        }
    }
}

// Every head's keys and values: C[row][m] = sum_x W[m][x] c[row][x], W the heads'
// key rows, then their value rows. A wavefront keeps 32 tokens' rows of c in
// registers (NS steps of 32 values of x), a work group of 8 of them takes `each`
// tiles of 128 rows of W through LDS, 128 values of x at a step: what has to come
// from memory per product is a fourth of what tiles of 128 x 128 read. Bound by the
// products and by what is written: 22.9 K tokens, 32 heads of 128 + 128 rows, x of 512:
// 321 us, 600 TFLOP/s and 0.75 GB (in tiles of 128 x 128, both through LDS, 487 us).
struct ExpandShape {
    int64_t rows;        // of made keys and values per head
    int32_t key_tiles;   // tiles of 128 of all heads' key rows
    int32_t value_tiles;
    int32_t each, ctiles;
    FastDiv key_div, value_div;  // rows of a head
};

// W's rows in LDS, as Planes, but read in another order: the operand of block 2 j + h
// has in place 4 q + r row 32 j + 8 q + 4 h + r, so that a lane's results of two blocks
// are 8 neighbours, and those of four lanes 64 bytes.
struct WRows {
    static constexpr int kPlane = 128 * 128;
    static constexpr __device__ __forceinline__ int swap(int r) {
        return ((r >> 1) & 1) | ((r >> 3) & 1) << 1 | ((r >> 4) & 1) << 2;
    }
    static __device__ __forceinline__ int base(int lane) {
        const int r = 8 * ((lane & 15) >> 2) + (lane & 3);
        return r * 128 + ((16 * (lane >> 4)) ^ (swap(r) << 4));
    }
    // block i of 8, step t of 4
    static __device__ __forceinline__ u32x4 row(const char* lds, int base, int i, int t) {
        const int r = 32 * (i >> 1) + 4 * (i & 1);  // (shares no bit with base's, nor with swap's)
        return *reinterpret_cast<const u32x4*>(lds + (base ^ (64 * (t & 1))) + r * 128 +
                                               (t >> 1) * kPlane);
    }
};

template <class T, int NS>
__global__ __launch_bounds__(512) void k_expand(ExpandArgs e, ExpandShape z) {
    constexpr int NW = 8, kRows = 32 * NW, kSteps = NS / 4;
    const LatentArgs& a = e.a;
    __shared__ __align__(16) char w0[2 * WRows::kPlane];
    __shared__ __align__(16) char w1[2 * WRows::kPlane];
    using G = Tile<T, 64, true>;
    const int tid = threadIdx.x, lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t unit = xcd_block();
    const int group = (int)(unit / z.ctiles);
    const int first = group * z.each;
    const int count = min(z.each, z.key_tiles + z.value_tiles - first);
    if (count <= 0) return;
    // this lane's two tokens: their latent rows, null where there is none
    const int64_t row0 = (unit - (int64_t)group * z.ctiles) * kRows + 32 * w;
    const char* from[2] = {nullptr, nullptr};
    bool none = false;  // a row that no sequence was found to need
    const auto take_row = [&](int x, const Sequence& sq, int64_t key) {
        if (key < 0 || key >= sq.length || sq.none) return false;
        const uint32_t pg = a.page_div.div((uint32_t)key);
        const uint32_t id = (uint32_t)a.col[sq.page0 + pg];
        const uint32_t slot = (uint32_t)key - pg * a.page_div.d;
        if (id < (uint64_t)a.npages)
            from[x] = a.k + ((uint64_t)(id * a.k_page + slot * a.k_slot) << a.k_shift);
        return true;
    };
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int64_t row = row0 + 16 * x + (lane & 15);
        if (row >= z.rows) continue;
        int64_t s, key;
        if (a.made_step) {
            s = row / a.made_step;
            key = row - s * a.made_step;
        } else {
            const int64_t entry = row / a.page_div.d;
            s = upper_index(a.rowptr, int64_t(0), a.seqs, entry);
            key = row - a.rowptr[s] * (int64_t)a.page_div.d;
        }
        none |= !take_row(x, read_sequence(a, s), key);
    }
    // A broken sequence's place in the table may be out of order, which misleads the search
    // for those of others. Most rows that nobody needs are just behind a text's end: only
    // where the table descends are all sequences asked for them.
    if (!a.made_step && __syncthreads_or(none)) {
        bool descends = false;
        for (int64_t s = tid; s < a.seqs; s += NW * kWave) descends |= a.rowptr[s] > a.rowptr[s + 1];
        if (__syncthreads_or(descends)) {
#pragma unroll 1
            for (int64_t s = 0; s < a.seqs; ++s) {
                const Sequence sq = read_sequence(a, s);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int64_t row = row0 + 16 * x + (lane & 15);
                    if (row < z.rows && !from[x])
                        take_row(x, sq, row - sq.page0 * (int64_t)a.page_div.d);
                }
            }
        }
    }
    if (!__syncthreads_or(from[0] || from[1])) return;
    const char* zero = reinterpret_cast<const char*>(g_zero);
    u32x4 c[2][NS];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int t = 0; t < NS; ++t) {
            const int at = 64 * t + 16 * (lane >> 4);
            c[x][t] = *reinterpret_cast<const u32x4*>(
                from[x] && at < 2 * e.latent_dim ? from[x] + at : zero);
        }
    // W's tile t of this work group: its side, first row, rows of a head and of all
    struct Side {
        bool keys;
        int m0, per, all;
    };
    const auto side = [&](int t) {
        Side x;
        x.keys = first + t < z.key_tiles;
        x.m0 = 128 * (x.keys ? first + t : first + t - z.key_tiles);
        x.per = x.keys ? a.made_dim : a.s.dim;
        x.all = a.s.hq * x.per;
        return x;
    };
    const char* wsrc[2];  // this lane's rows of blocks of 8 rows 2 w and 2 w + 1
    const auto open = [&](int t) {
        const Side x = side(t);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * (2 * w + i) + (lane >> 3), m = x.m0 + r;
            wsrc[i] = nullptr;
            if (m < x.all) {
                const int head = (int)(x.keys ? z.key_div : z.value_div).div(m);
                const AttnRows& y = x.keys ? e.wk : e.wv;
                wsrc[i] = y.base + head * y.row + (m - head * x.per) * y.head;
            }
        }
    };
    const auto load = [&](char* to, int step) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * (2 * w + i) + (lane >> 3);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int at = 256 * step + 128 * g + 16 * ((lane & 7) ^ WRows::swap(r));
                load_to_lds(wsrc[i] && at < 2 * e.latent_dim ? wsrc[i] + at : zero,
                            to + g * WRows::kPlane + (2 * w + i) * 1024);
            }
        }
    };
    f32x4 acc[8][2];  // blocks of 16 rows of W, of 16 tokens
    const int wb = WRows::base(lane);
    // tile t, whose step `at` is in `rows`; the next one is loaded into `next`
    const auto take = [&](const char* rows, char* next, int t, auto at) {
        constexpr int kAt = decltype(at)::value;
        if constexpr (kAt == 0)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = f32x4{0, 0, 0, 0};
        if (kAt + 1 < kSteps) {
            load(next, kAt + 1);
        } else if (t + 1 < count) {
            open(t + 1);
            load(next, 0);
        }
        // operands are read kAhead before their products, as in k_absorbed
        constexpr int kAhead = 4;
        u32x4 y[kAhead + 1];
#pragma unroll
        for (int n = -kAhead; n < 32; ++n) {
            __builtin_amdgcn_sched_barrier(0);
            const int r = n + kAhead;
            if (r < 32) y[r % (kAhead + 1)] = WRows::row(rows, wb, r % 8, r / 8);
            if (n < 0) continue;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                acc[n % 8][x] = mfma32<T>(y[n % (kAhead + 1)], c[x][4 * kAt + n / 8], acc[n % 8][x]);
        }
        __builtin_amdgcn_sched_barrier(0);
        wait_for_loads();
        __syncthreads();
        if constexpr (kAt + 1 == kSteps) {  // (after the wait, which would be theirs too)
            const Side d = side(t);
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 8 neighbours of each token's row
                const int m = d.m0 + 32 * j + 8 * (lane >> 4);
                if (m >= d.all) continue;
                const int head = (int)(d.keys ? z.key_div : z.value_div).div(m);
                char* to = (d.keys ? a.made_k : a.made_v) +
                           ((int64_t)head * z.rows * 2 * d.per + m - head * d.per) * 2;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!from[x]) continue;
                    char* row = to + (row0 + 16 * x + (lane & 15)) * 4 * d.per;
                    // rounded, and what that leaves (nothing where it is not finite)
                    uint32_t high[4], low[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const f32x4& y = acc[2 * j + h / 2][x];
                        const float y0 = y[2 * (h & 1)], y1 = y[2 * (h & 1) + 1];
                        high[h] = pack2<T>(y0, y1);
                        float r0, r1;
                        unpack2<T>(high[h], r0, r1);
                        low[h] = pack2<T>(__builtin_isfinite(r0) ? y0 - r0 : 0.f,
                                          __builtin_isfinite(r1) ? y1 - r1 : 0.f);
                    }
                    *reinterpret_cast<u32x4*>(row) = u32x4{high[0], high[1], high[2], high[3]};
                    *reinterpret_cast<u32x4*>(row + 2 * d.per) = u32x4{low[0], low[1], low[2], low[3]};
                }
            }
        }
    };
    open(0);
    load(w0, 0);
    wait_for_loads();
    __syncthreads();
    using I0 = std::integral_constant<int, 0>;
    if constexpr (kSteps == 1) {
        for (int t = 0; t < count; t += 2) {
            take(w0, w1, t, I0{});
            if (t + 1 < count) take(w1, w0, t + 1, I0{});
        }
    } else {
        for (int t = 0; t < count; ++t) {
            take(w0, w1, t, I0{});
            take(w1, w0, t, std::integral_constant<int, 1>{});
            if constexpr (kSteps == 4) {
                take(w0, w1, t, std::integral_constant<int, 2>{});
                take(w1, w0, t, std::integral_constant<int, 3>{});
            }
        }
    }
}

template <class F>
void with_latent_type(int type, F&& f) {
    if (type == SPGEMM_TYPE_BF16) f((__bf16*)nullptr);
    else f((_Float16*)nullptr);
}
template <int N>
using Int = std::integral_constant<int, N>;
// f(geometry, type) of a call: the smallest widths that hold it.
template <class F>
void with_absorbed(const LatentArgs& a, F&& f) {
    with_latent_type(a.s.type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const auto width = [&](auto dk, auto dv, auto dh) {
            constexpr int K = decltype(dk)::value, V = decltype(dv)::value, D = decltype(dh)::value;
            if (a.key_dim == K) f((AbsorbedGeo<T, K, V, 2, D, true>*)nullptr, t);
            else f((AbsorbedGeo<T, K, V, 2, D, false>*)nullptr, t);
        };
        if (a.s.dim <= 128 && a.key_dim <= 192) width(Int<192>{}, Int<128>{}, Int<1>{});
        else if (a.s.dim <= 256 && a.key_dim <= 320) width(Int<320>{}, Int<256>{}, Int<1>{});
        else width(Int<576>{}, Int<512>{}, Int<2>{});
    });
}
template <class F>
void with_expanded(const LatentArgs& a, F&& f) {
    with_latent_type(a.s.type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const auto width = [&](auto planes) {
            constexpr int P = decltype(planes)::value;
            // Tiles of 256 rows where they fill the compute units: chunks of 2048 in 2
            // texts and 32 heads take 1590 us in them, 1836 in tiles of 128; chunks
            // of up to 500 in 6 texts and 9 heads 51 and 46 us. (Rows fit 31 bits.)
            const int64_t tall = a.s.hq * (a.seqs + a.tokens / 256);
            if (a.max_new >= 256 && a.max_new <= 1 << 30 && tall >= 256)
                f((ExpandedGeo<T, P, P, 8>*)nullptr, t);
            else f((ExpandedGeo<T, P, P, 4>*)nullptr, t);
        };
        if (a.s.dim <= 64 && a.made_dim <= 64) width(Int<1>{});
        else width(Int<2>{});
    });
}

}  // namespace

int latent_tile_rows(const LatentArgs& a, bool absorbed) {
    int bm = 0;
    const auto get = [&](auto* g, auto*) { bm = std::remove_pointer_t<decltype(g)>::BM; };
    if (absorbed) with_absorbed(a, get);
    else with_expanded(a, get);
    return bm;
}

void latent_attention(const LatentArgs& a, bool absorbed, hipStream_t st) {
    const int rows = latent_tile_rows(a, absorbed);
    const int32_t tiles = (int32_t)ceil_div((int64_t)a.max_new * a.s.group, rows);
    if (absorbed) {
        const dim3 grid = grid_2d(xcd_grid((a.ranges ? a.ranges : a.seqs) * (int64_t)tiles));
        with_absorbed(a, [&](auto* geo, auto* t) {
            using G = std::remove_pointer_t<decltype(geo)>;
            auto run = k_absorbed<G, std::remove_pointer_t<decltype(t)>>;
            hipLaunchKernelGGL(run, grid, dim3(G::NW * kWave), 0, st, a, tiles);
        });
    } else {
        const dim3 grid = grid_2d(xcd_grid(a.seqs * a.s.hkv * a.npieces * tiles));
        with_expanded(a, [&](auto* geo, auto* t) {
            using G = std::remove_pointer_t<decltype(geo)>;
            auto run = k_expanded<G, std::remove_pointer_t<decltype(t)>>;
            hipLaunchKernelGGL(run, grid, dim3(G::NW * kWave), 0, st, a, tiles);
        });
    }
    SG_LAUNCH_CHECK();
    if (a.npieces == 1 && a.ranges == 0) return;
    with_latent_type(a.s.type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (a.seqs <= 256) join_parts<T, 256>(a, tiles, rows, kAbsorbedKeys, kShift<T>, st);
        else join_parts<T, kAbsorbedEvenSeqs>(a, tiles, rows, kAbsorbedKeys, kShift<T>, st);
    });
}

void latent_expand(const ExpandArgs& e, hipStream_t st) {
    const LatentArgs& a = e.a;
    ExpandShape z;
    z.rows = a.made_rows;
    z.key_tiles = (int32_t)ceil_div((int64_t)a.s.hq * a.made_dim, 128);
    z.value_tiles = (int32_t)ceil_div((int64_t)a.s.hq * a.s.dim, 128);
    z.key_div = FastDiv((uint32_t)a.made_dim);
    z.value_div = FastDiv((uint32_t)a.s.dim);
    const int64_t ctiles = ceil_div(z.rows, 256), wtiles = z.key_tiles + z.value_tiles;
    if (ctiles == 0) return;
    if (ctiles > INT32_MAX) throw OverflowError("rows of made keys");
    // One work group per compute unit is there at once; looking its tokens up and
    // reading them takes as long as 1.2 tiles (26 of 23 thousand cycles): so many
    // tiles each as end first. 22.9 K tokens, 64 tiles of W: 8 each, 3 rounds, 321 us;
    // 5 each, 5 rounds, 340.
    int64_t best = INT64_MAX;
    for (int each = 1; each <= std::min<int64_t>(wtiles, 64); ++each) {
        const int64_t rounds = ceil_div(ctiles * ceil_div(wtiles, each), 256);
        const int64_t cost = rounds * (5 * each + 6);
        if (cost < best) {
            best = cost;
            z.each = each;
        }
    }
    z.ctiles = (int32_t)ctiles;
    const dim3 grid = grid_2d(xcd_grid(ctiles * ceil_div(wtiles, z.each)));
    with_latent_type(a.s.type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const auto run = e.latent_dim <= 128   ? k_expand<T, 4>
                         : e.latent_dim <= 256 ? k_expand<T, 8>
                                               : k_expand<T, 16>;
        hipLaunchKernelGGL(run, grid, dim3(512), 0, st, e, z);
    });
    SG_LAUNCH_CHECK();
}

}  // namespace sg
