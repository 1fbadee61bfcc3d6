// Attention of new tokens over a quantised paged cache. The cache's values are
// exact in bfloat16, and so are its products: a query of any type enters them
// as NP bfloat16 parts that add up to it (8, 11 and 24 bits: 1, 2 and 3 parts),
// and so do the probabilities, with 8, 16 or 24 bits. Single precision runs at a
// third of the bfloat16 rate that way, five times its own.
#include "attention_join.h"
#include "mx.h"

namespace sg {

namespace {

constexpr int kWaves = 4;

template <class T>
constexpr int kParts = std::is_same<T, __bf16>::value ? 1 : sizeof(T) == 2 ? 2 : 3;

// The upper 16 bits of a float as bfloat16 (rounded toward 0, so that what is
// left has the same sign and the parts add up).
__device__ __forceinline__ float bf16_cut(float x) {
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xffff0000u);
}
// NP words of bfloat16 pairs that add up to a and b, the largest first.
template <int NP>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&w)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        if (i == NP - 1) {
            w[i] = pack2<__bf16>(a, b);
        } else {
            const float x = bf16_cut(a), y = bf16_cut(b);
            w[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, y),
                                         __builtin_bit_cast(uint32_t, x), 0x07060302u);
            a -= x;
            b -= y;
        }
    }
}

// The tile of bfloat16 keys and values, with queries, weights and results of
// type T.
template <class T, int DP, bool FULL>
struct MxGeo : Tile<__bf16, DP, FULL> {
    using Base = Tile<__bf16, DP, FULL>;
    static constexpr int NP = kParts<T>;
    struct Probs { u32x4 w[NP]; };
    static __device__ __forceinline__ void pack_probs(const float (&p)[Base::VK], Probs& out) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[NP];
            split2<NP>(p[2 * i], p[2 * i + 1], w);
#pragma unroll
            for (int x = 0; x < NP; ++x) out.w[x][i] = w[x];
        }
    }
    static __device__ __forceinline__ f32x4 add_block(u32x4 v, const Probs& p, f32x4 o) {
#pragma unroll
        for (int x = NP - 1; x >= 0; --x) o = mfma32<__bf16>(v, p.w[x], o);
        return o;
    }
    static __device__ __forceinline__ float prob_of(const Probs& p, int key) {
        float sum = 0.f;
#pragma unroll
        for (int x = NP - 1; x >= 0; --x)
            sum += Base::prob_of(typename Base::Probs{{p.w[x][0], p.w[x][1], p.w[x][2], p.w[x][3]}}, key);
        return sum;
    }
    static __device__ __forceinline__ void store_four(f32x4 v, char* at) {
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<u32x2*>(at) = u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
        else
            *reinterpret_cast<f32x4*>(at) = v;
    }
    // 8 values of a query row, from the d-th on, as step `step` of its parts.
    // (An infinity or a NaN is its first part alone.)
    static __device__ __forceinline__ void load_query(const char* row, int d, int dim, int step,
                                                      typename Base::RowFrag (&q)[NP]) {
        const bool in = FULL || d < dim;
        if constexpr (NP == 1) {
            q[0].w[step] = in ? *reinterpret_cast<const u32x4*>(row + 2 * d) : u32x4{0, 0, 0, 0};
        } else {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
            if (in) {
                if constexpr (sizeof(T) == 2) {
                    const u32x4 w = *reinterpret_cast<const u32x4*>(row + 2 * d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) unpack2<T>(w[i], x[2 * i], x[2 * i + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const f32x4 y = *reinterpret_cast<const f32x4*>(row + 4 * d + 16 * j);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[4 * j + i] = y[i];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[NP];
                split2<NP>(x[2 * i], x[2 * i + 1], w);
                const bool a = __builtin_isfinite(x[2 * i]), b = __builtin_isfinite(x[2 * i + 1]);
                if (!a || !b) {  // (cut, a NaN could become an infinity)
                    const uint32_t whole = pack2<__bf16>(x[2 * i], x[2 * i + 1]);
                    w[0] = (a ? w[0] & 0xffffu : whole & 0xffffu) |
                           (b ? w[0] & 0xffff0000u : whole & 0xffff0000u);
#pragma unroll
                    for (int p = 1; p < NP; ++p)
                        w[p] = (a ? w[p] & 0xffffu : 0u) | (b ? w[p] & 0xffff0000u : 0u);
                }
#pragma unroll
                for (int p = 0; p < NP; ++p) q[p].w[step][i] = w[p];
            }
        }
    }
};

// How single wavefronts read codes: lane l takes kRun codes of key l % 16 (and
// of that plus 16), from value 4 kRun t + kRun (l / 16) on for load t, which is
// within one block. kRun * bits are 16 bytes where the row is long enough.
template <int BITS, int DP>
struct MxRuns {
    static constexpr int kRun = BITS == 8 ? 16 : DP >= 128 ? 32 : 16;
    static constexpr int kLoads = DP / (4 * kRun);
    static constexpr int kWords = kRun * BITS / 32;
    static constexpr int kSteps = kRun / 8;  // products per load
    static_assert(kLoads * kSteps == DP / 32, "every product has its codes");
    static __device__ __forceinline__ int first(int t) {
        return 4 * kRun * t + kRun * (lane_id() >> 4);
    }
    struct Codes {
        uint32_t w[kLoads][kWords];
        uint32_t scale[kLoads];
    };
    template <bool FULL>
    static __device__ __forceinline__ void load(const char* codes, const uint8_t* scales, int dim,
                                                Codes& c) {
#pragma unroll
        for (int t = 0; t < kLoads; ++t) {
            const int d = first(t);
            if (FULL || d < dim) {
                const char* at = codes + d * BITS / 8;
                if constexpr (kWords == 4) {
                    const u32x4 x = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
                    for (int i = 0; i < 4; ++i) c.w[t][i] = x[i];
                } else {
                    const u32x2 x = *reinterpret_cast<const u32x2*>(at);
                    c.w[t][0] = x[0];
                    c.w[t][1] = x[1];
                }
                c.scale[t] = scales[d / SPGEMM_MX_BLOCK];
            } else {
#pragma unroll
                for (int i = 0; i < kWords; ++i) c.w[t][i] = 0;
                c.scale[t] = 127;
            }
        }
    }
    static __device__ __forceinline__ u32x4 decode(const Codes& c, int t, int u) {
        return mx_decode8<BITS>(&c.w[t][u * BITS / 4], mx_scale(c.scale[t]));
    }
};

// o += w times the 4 values from value d of a cached row on.
template <int BITS>
__device__ __forceinline__ f32x4 add_codes(const char* codes, const uint8_t* scales, int d, float w,
                                           f32x4 o) {
    uint32_t c[2] = {0, 0};
    if constexpr (BITS == 8)
        c[0] = *reinterpret_cast<const uint32_t*>(codes + d);
    else
        c[0] = *reinterpret_cast<const uint16_t*>(codes + d / 2);
    const u32x4 x = mx_decode8<BITS>(c, mx_scale(scales[d / SPGEMM_MX_BLOCK]));
    float y[4];
    unpack2<__bf16>(x[0], y[0], y[1]);
    unpack2<__bf16>(x[1], y[2], y[3]);
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = fmaf(w, y[r], o[r]);
    return o;
}

// Work groups of k_mx that a compute unit holds at once. (A third of heads of 128
// leaves 168 registers and spills: 325 us for 282 in 8 bits, 351 for 221 in 4.)
template <int DP>
constexpr int kMxResident = DP <= 64 ? 3 : DP <= 128 ? 2 : 1;

// Few rows per sequence and key head: one wavefront takes 16 rows and one range
// or piece of the keys, straight from memory, in one pass with a running maximum
// and sum. Codes of a tile of 32 keys are turned into operands in registers (keys)
// and into rows in LDS (values, read back transposed), and the next tile's are
// under way from then on. Bound by the codes' and scales' bytes, once each: a new
// token of 64 texts of up to 16384, 64 / 8 heads of 128, 8 bits, 1.14 GB, takes
// 265 us with the join (4.3 TB/s); 4 of 32 / 8 heads, 4 bits, 0.59 GB, 163 us
// (3.6 TB/s, the vector unit half busy, most of it with codes). A second tile under
// way, in 40 more registers, gained nothing (282 and 231 us for 282 and 221).
template <int BITS, class G, class T>
__global__ __launch_bounds__(kWaves* kWave, kMxResident<G::kDim>) void k_mx(MxArgs a, int32_t tiles) {
    using R = MxRuns<BITS, G::kDim>;
    constexpr int NP = G::NP, KT = G::KT;
    static_assert(KT == kMxKeys, "the host cuts keys by whole tiles");
    __shared__ __align__(16) char stage[kWaves][KT * G::kRowBytes];
    const int lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    char* vrows = stage[w];
    int64_t unit = xcd_block() * kWaves + w;
    if (unit >= (a.ranges ? a.ranges : a.seqs * a.npieces) * a.s.hkv * tiles) return;
    const int tile = (int)(unit % tiles);
    unit /= tiles;
    int range = 0, piece = 0, s = 0, h;
    int pos = 0, end = 0, before = 0;  // tiles of all sequences' keys, of a range
    // The heads of the same keys run side by side: a line of the cache's codes or
    // scales often holds several heads' and is then read once per chiplet.
    h = (int)(unit % a.s.hkv);
    unit /= a.s.hkv;
    if (a.ranges) {
        range = (int)unit;
        const EvenSplit<kMxEvenSeqs> e(a, KT);
        pos = (int)min((int64_t)range * e.per, (int64_t)e.total);
        end = min(pos + e.per, e.total);
        if (pos >= end) return;
        e.locate(pos, s, before);
    } else {
        piece = (int)(unit % a.npieces);
        s = (int)(unit / a.npieces);
    }
    const int begin = pos;
#pragma unroll 1
    for (;; ++s) {  // segments
        TileJob job = tile_job(a, s, tile, 16, piece);
        const bool late = pos > begin;
        bool split = false;
        if (a.ranges) {
            const int own = job.sq.none ? 0 : job.sq.bad ? 1 : (job.sq.length + KT - 1) / KT;
            split = pos > before || before + own > end;
            const int last = job.before + (min(job.first + 16, job.rows) - 1) / a.s.group;
            job.k0 = (pos - before) * KT;
            job.k1 = min(last, (int)min((int64_t)(end - before) * KT, (int64_t)INT32_MAX));
            before += own;
            pos = before;
        }
        const auto segment = [&] {
            if (job.idle) return;
            const int n = lane & 15;
            const TileRow r = tile_row(a, job, job.first + n, h);
            if (job.sq.bad) {
                if (piece == 0) store_nan<T>(a, r);
                return;
            }
            if (job.k0 >= job.k1) return;
            const int lo = __builtin_amdgcn_readfirstlane(r.t);

            typename G::RowFrag q[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) G::zero_row(q[p]);
            if (r.has) {
                const char* row = a.q.base + r.token * a.q.row + r.hq * a.q.head;
#pragma unroll
                for (int t = 0; t < R::kLoads; ++t)
#pragma unroll
                    for (int u = 0; u < R::kSteps; ++u)
                        G::load_query(row, R::first(t) + 8 * u, a.s.dim, t * R::kSteps + u, q);
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) G::sign_row(q[p], a.s.c);
            const char* kb = a.k + h * a.k_head;
            const char* vb = a.v + h * a.v_head;
            const uint8_t* ksb = a.ks + h * a.ks_head;
            const uint8_t* vsb = a.vs + h * a.vs_head;
            const int32_t* pages = a.col + job.sq.page0;
            bool wrong = false;  // a page outside the cache
            struct Place {
                uint32_t id[2], slot[2];  // of this lane's two keys
            };
            // keys past the end repeat the last one (also where a whole tile is past it:
            // a load under a branch would make every wait the wait for all loads)
            const uint32_t each = a.page_div.d == 1 ? ~0u : 0u;  // (of one slot: no branch either)
            const auto place = [&](int t0) {
                Place x;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t key = (uint32_t)min(t0 + 16 * j + n, job.k1 - 1);
                    const uint32_t pg = (__umulhi(key, a.page_div.mul) >> a.page_div.shift) | (key & each);
                    x.id[j] = (uint32_t)pages[pg];
                    x.slot[j] = key - pg * a.page_div.d;
                }
                return x;
            };
            const auto checked = [&](Place& x) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (x.id[j] >= (uint64_t)a.npages) {
                        wrong = true;
                        x.id[j] = 0;
                    }
            };
            typename R::Codes k[2], v[2];
            const auto load = [&](const Place& x) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    R::template load<G::kFull>(
                        kb + ((uint64_t)(x.id[j] * a.k_page + x.slot[j] * a.k_slot) << a.k_shift),
                        ksb + ((uint64_t)(x.id[j] * a.ks_page + x.slot[j] * a.ks_slot) << a.ks_shift),
                        a.s.dim, k[j]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    R::template load<G::kFull>(
                        vb + ((uint64_t)(x.id[j] * a.v_page + x.slot[j] * a.v_slot) << a.v_shift),
                        vsb + ((uint64_t)(x.id[j] * a.vs_page + x.slot[j] * a.vs_slot) << a.vs_shift),
                        a.s.dim, v[j]);
                }
            };
            Place now = place(job.k0), next = place(job.k0 + KT);
            checked(now);
            load(now);

            typename G::AccB o;
#pragma unroll
            for (int b = 0; b < G::NB; ++b) o.o[b] = f32x4{0, 0, 0, 0};
            Softmax<G, T> sm;
            const int vbase = G::value_base(0);
#pragma unroll 1
            for (int t0 = job.k0; t0 < job.k1; t0 += KT) {
                const int left = job.k1 - t0;
                f32x4 sc[1][G::KSUB];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f32x4 x{0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < R::kLoads; ++t)
#pragma unroll
                        for (int u = 0; u < R::kSteps; ++u) {
                            const u32x4 y = R::decode(k[j], t, u);
#pragma unroll
                            for (int p = NP - 1; p >= 0; --p)
                                x = mfma32<__bf16>(y, q[p].w[t * R::kSteps + u], x);
                        }
                    sc[0][j] = x;
                }
                // a key that a row does not see must not reach it as 0 times an
                // infinity or a NaN: its row is staged as 0 and added on its own below
                const bool crosses = t0 + KT > job.before + lo;
                uint32_t wild = 0;
                wave_lds_sync();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    u32x4 y[R::kLoads * R::kSteps];
                    bool off = false;
#pragma unroll
                    for (int t = 0; t < R::kLoads; ++t)
#pragma unroll
                        for (int u = 0; u < R::kSteps; ++u) y[t * R::kSteps + u] = R::decode(v[j], t, u);
                    if (crosses) {
#pragma unroll
                        for (const u32x4& x : y) {
                            const uint32_t words[4] = {x[0], x[1], x[2], x[3]};
                            off |= G::words_wild(words);
                        }
                        uint64_t is = __ballot(off);
                        is |= is >> 32;
                        is |= is >> 16;
                        wild |= (uint32_t)(is & 0xffff) << (16 * j);
                    }
                    // 0 weight times what the row that they repeat holds may be NaN
                    if (left < KT || wild) {
                        const bool zero = 16 * j + n >= left || (wild >> (16 * j + n) & 1);
#pragma unroll
                        for (u32x4& x : y) x = zero ? u32x4{0, 0, 0, 0} : x;
                    }
#pragma unroll
                    for (int t = 0; t < R::kLoads; ++t)
#pragma unroll
                        for (int u = 0; u < R::kSteps; ++u)
                            *reinterpret_cast<u32x4*>(
                                vrows + G::stage_at(16 * j + n, 2 * (R::first(t) + 8 * u))) =
                                y[t * R::kSteps + u];
                }
                wave_lds_sync();
                const Place here = now;
                // (the pages first: loads end in the order that they began in)
                now = next;
                checked(now);
                next = place(t0 + 2 * KT);
                load(now);
                sm.hide(sc[0], Seen::first(min(left, job.before + r.t - t0)));
                typename G::Probs pr[1];
                bool far;
                const float fix = sm.template weigh<true>(sc, a.s.mag, pr, far);
                if (__any(fix != 1.f)) G::scale_acc(o, fix);
#pragma unroll
                for (int i = 0; i < G::NB; ++i)
                    o.o[i] = G::add_block(G::value_frag(vrows, vbase, i), pr[0], o.o[i]);
                for (; wild; wild &= wild - 1) {
                    const int key = __builtin_ctz(wild);
                    const uint32_t id = __shfl(key < 16 ? here.id[0] : here.id[1], key & 15, kWave);
                    const uint32_t slot = __shfl(key < 16 ? here.slot[0] : here.slot[1], key & 15, kWave);
                    const float p = G::prob_of(pr[0], key);
                    if (t0 + key >= min(job.k1, job.before + r.t)) continue;
                    const char* codes = vb + ((uint64_t)(id * a.v_page + slot * a.v_slot) << a.v_shift);
                    const uint8_t* scales =
                        vsb + ((uint64_t)(id * a.vs_page + slot * a.vs_slot) << a.vs_shift);
#pragma unroll
                    for (int i = 0; i < G::NB; ++i) {
                        const int d = 16 * i + 4 * (lane >> 4);
                        if (G::kFull || d < a.s.dim) o.o[i] = add_codes<BITS>(codes, scales, d, p, o.o[i]);
                    }
                }
            }
            sm.finish(a.s.mag);
            if (__any(wrong)) sm.l = NAN;
            if (!a.ranges)
                store_row<G, T>(a, job, r, piece, o, sm);
            else if (r.has && job.before + r.t > job.k0)
                store_row_at<G, T>(
                    a, r, !split,
                    ((((int64_t)2 * range + late) * a.s.hkv + h) * tiles + tile) * 16 + n, o, sm);
        };
        segment();
        if (pos >= end) return;
    }
}

// Many rows: a work group of 4 wavefronts takes 4 * 16 * QB rows, a wavefront
// 16 * QB of them, and BK keys at a time are turned into bfloat16 rows in LDS
// for all of them. Bound by the softmax and the turning of codes on the vector unit
// (52 % busy) beside the products (35 %), with two wavefronts per SIMD: chunks of
// 2048 of two texts of up to 32768, 32 / 8 heads of 128, 1500 us, 787 TFLOP/s. Tiles
// of 256 rows, whose codes are turned half as often, take 1611 us with one work
// group per compute unit, and a second buffer for one barrier a tile instead of two
// 1526.
template <class G, class T>
struct MxWide {
    static constexpr int QB = G::kDim <= 128 && G::NP == 1 ? 2 : 1;  // 16-row blocks per wavefront
    static constexpr int BM = kWaves * 16 * QB;
    static_assert(BM <= kPagedTileMost, "the limit of rows counts on it");
    static constexpr int BK = G::kDim <= 128 ? 64 : 32;
    static constexpr int NS = G::NP == 1 && BK > G::KT ? 2 : 1;  // tiles per step of the softmax
};

template <int BITS, class G, class T>
__global__ __launch_bounds__(kWaves* kWave, G::kDim <= 128 ? 2 : 1) void k_mx_wide(MxArgs a,
                                                                                   int32_t tiles) {
    using W = MxWide<G, T>;
    constexpr int NT = kWaves * kWave, BK = W::BK, QB = W::QB, NS = W::NS, NP = G::NP;
    // 16-byte pieces of codes
    constexpr int kCodes = 128 / BITS, kPieces = G::kDim / kCodes;
    constexpr int kStep = NT / kPieces < BK ? NT / kPieces : BK, kLoads = BK / kStep;
    static_assert(BK % (NS * G::KT) == 0 && BK % kStep == 0, "tile shape");
    __shared__ __align__(16) char rows[2][BK * G::kRowBytes];  // k, v
    __shared__ uint32_t off[2][4][BK];  // of this tile and the next: codes and scales of k and v
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

    typename G::RowFrag q[QB][NP];
    typename G::AccB o[QB];
    Softmax<G, T> sm[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
#pragma unroll
        for (int i = 0; i < G::NB; ++i) o[b].o[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < NP; ++p) G::zero_row(q[b][p]);
        if (r[b].has) {
            const char* row = a.q.base + r[b].token * a.q.row + r[b].hq * a.q.head;
#pragma unroll
            for (int t = 0; t < G::QS; ++t)
                G::load_query(row, 32 * t + 8 * (lane >> 4), a.s.dim, t, q[b]);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) G::sign_row(q[b][p], a.s.c);
    }
    const char* kb = a.k + h * a.k_head;
    const char* vb = a.v + h * a.v_head;
    const uint8_t* ksb = a.ks + h * a.ks_head;
    const uint8_t* vsb = a.vs + h * a.vs_head;
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
            off[par][2][tid] = id * a.ks_page + slot * a.ks_slot;
            off[par][3][tid] = id * a.vs_page + slot * a.vs_slot;
        }
    };
    u32x4 fly[2][kLoads];
    uint32_t fly_s[2][kLoads];
    const int prow = tid / kPieces, pd = tid % kPieces * kCodes;  // this thread's pieces
    const bool inside = (G::kFull || pd < a.s.dim) && prow < kStep;
    const auto load_rows = [&](int t0, int par) {
        const int left = job.k1 - t0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int p = i * kStep + prow;
            fly[0][i] = fly[1][i] = u32x4{0, 0, 0, 0};  // past the end and the row's width
            fly_s[0][i] = fly_s[1][i] = 127;
            if (inside && p < left) {
                fly[0][i] = *reinterpret_cast<const u32x4*>(
                    kb + ((uint64_t)off[par][0][p] << a.k_shift) + pd * BITS / 8);
                fly[1][i] = *reinterpret_cast<const u32x4*>(
                    vb + ((uint64_t)off[par][1][p] << a.v_shift) + pd * BITS / 8);
                fly_s[0][i] = ksb[((uint64_t)off[par][2][p] << a.ks_shift) + pd / SPGEMM_MX_BLOCK];
                fly_s[1][i] = vsb[((uint64_t)off[par][3][p] << a.vs_shift) + pd / SPGEMM_MX_BLOCK];
            }
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
        // some row may not see some key: a value row with an infinity or
        // a NaN is staged as 0, so that 0 times it stays 0, and is added
        // on its own below for the rows that see it
        const bool crosses = t0 + BK > job.before + job.first / a.s.group;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int p = i * kStep + prow;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                u32x4 y[kCodes / 8];
                bool is = false;
#pragma unroll
                for (int u = 0; u < kCodes / 8; ++u) {
                    const uint32_t c[4] = {fly[x][i][0], fly[x][i][1], fly[x][i][2], fly[x][i][3]};
                    y[u] = mx_decode8<BITS>(c + u * BITS / 4, mx_scale(fly_s[x][i]));
                    if (x == 1 && crosses) {
                        const uint32_t words[4] = {y[u][0], y[u][1], y[u][2], y[u][3]};
                        is |= G::words_wild(words);
                    }
                }
                if (x == 1 && crosses) {
                    const uint64_t b = __ballot(is);
                    const int lane0 = lane / kPieces * kPieces;  // of this row's pieces
                    const uint64_t whole = (1ull << kPieces) - 1;
                    if (b >> lane0 & whole) {
#pragma unroll
                        for (int u = 0; u < kCodes / 8; ++u) y[u] = u32x4{0, 0, 0, 0};
                        if (lane == lane0) atomicOr(&wild_s[par], 1ull << p);
                    }
                }
                if (prow < kStep)
#pragma unroll
                    for (int u = 0; u < kCodes / 8; ++u)
                        *reinterpret_cast<u32x4*>(rows[x] + G::stage_at(p, 2 * (pd + 8 * u))) = y[u];
            }
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
                        for (int x = 0; x < QB; ++x) {
                            f32x4 y{0, 0, 0, 0};
#pragma unroll
                            for (int p = NP - 1; p >= 0; --p) y = G::dot(k, q[x][p], y);
                            sc[x][i][b] = y;
                        }
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
            // weights again, after those of the others (as in k_paged_wide).
            constexpr bool kAgain = G::kFull && NP == 1;
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
                    const char* codes = vb + ((uint64_t)off[par][1][first + key] << a.v_shift);
                    const uint8_t* scales = vsb + ((uint64_t)off[par][3][first + key] << a.vs_shift);
#pragma unroll
                    for (int x = 0; x < QB; ++x) {
                        const float p = G::prob_of(pr[x][i], key);
                        if (t0 + first + key >= job.before + r[x].t) continue;
#pragma unroll
                        for (int b = 0; b < G::NB; ++b) {
                            const int d = 16 * b + 4 * (lane >> 4);
                            if (G::kFull || d < a.s.dim)
                                o[x].o[b] = add_codes<BITS>(codes, scales, d, p, o[x].o[b]);
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

// f(geometry, type, bits) of a call.
template <class T, int BITS, class F>
void with_mx_dim(int dim, F&& f) {
    const auto go = [&](auto dp, auto full) {
        f((MxGeo<T, decltype(dp)::value, decltype(full)::value>*)nullptr, (T*)nullptr,
          std::integral_constant<int, BITS>{});
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    using I256 = std::integral_constant<int, 256>;
    if (dim == 64) go(I64{}, std::true_type{});
    else if (dim < 64) go(I64{}, std::false_type{});
    else if (dim == 128) go(I128{}, std::true_type{});
    else if (dim < 128) go(I128{}, std::false_type{});
    else if (dim == 256) go(I256{}, std::true_type{});
    else go(I256{}, std::false_type{});
}
template <class F>
void with_mx(const AttnShape& s, int format, F&& f) {
    const auto type = [&](auto bits) {
        constexpr int B = decltype(bits)::value;
        if (s.type == SPGEMM_TYPE_BF16) with_mx_dim<__bf16, B>(s.dim, f);
        else if (s.type == SPGEMM_TYPE_F16) with_mx_dim<_Float16, B>(s.dim, f);
        else with_mx_dim<float, B>(s.dim, f);
    };
    if (format == SPGEMM_MX_E4M3) type(std::integral_constant<int, 8>{});
    else type(std::integral_constant<int, 4>{});
}

}  // namespace

// Whether a sequence's rows of a key head are worth keys in LDS for all of them. k_mx cuts
// ragged texts evenly but turns the codes anew for every 16 rows, k_mx_wide turns them
// once for 128 (64) and cuts by the longest text, which is all that the host knows of them:
// between 16 and some 64 rows the texts decide which is better, and the limit lies between.
// us by k_mx and k_mx_wide, 4 heads (8 where texts are of one length), heads of 128:
//   8 bits, bf16, 16 rows   64 texts to 8192 85, 142   64 of 3000 63, 64    200 to 400 49, 30
//                 32 rows                    120, 145  64 of 6000 365, 203             74, 32
//   4 bits, bf16, 32 rows                    82, 140              208, 191             69, 31
//   8 bits, fp32, 32 rows                    127, 211             369, 299             79, 42
//   8 bits, fp16, 64 rows (64 to 16 K, 8 heads) 967, 648          686, 295             101, 39
// and of 256:
//   8 bits, bf16, 48 rows   64 to 8192 405, 436        64 of 3000 285, 173  200 to 400 124, 84
//                 64 rows              524, 445                   353, 177             146, 88
bool mx_wide(const AttnShape& s, int64_t rows) { return rows > (s.dim > 128 ? 48 : 16); }

int mx_tile_rows(const AttnShape& s, int64_t rows) {
    if (!mx_wide(s, rows)) return 16;
    return s.dim <= 128 && s.type == SPGEMM_TYPE_BF16 ? 128 : 64;
}

void mx_attention(const MxArgs& a, hipStream_t st) {
    const int64_t rows = (int64_t)a.max_new * a.s.group;
    const int64_t tiles = ceil_div(rows, mx_tile_rows(a.s, rows));
    if (a.seqs == 0 || a.tokens == 0 || tiles == 0) return;
    const int64_t units = (a.ranges ? a.ranges : a.seqs * a.npieces) * a.s.hkv * tiles;
    with_mx(a.s, a.format, [&](auto* geo, auto* t, auto bits) {
        using G = std::remove_pointer_t<decltype(geo)>;
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int B = decltype(bits)::value;
        if (mx_wide(a.s, rows)) {
            auto run = k_mx_wide<B, G, T>;
            hipLaunchKernelGGL(run, grid_2d(xcd_grid(units)), dim3(kWaves * kWave), 0, st, a,
                               (int32_t)tiles);
        } else {
            auto run = k_mx<B, G, T>;
            hipLaunchKernelGGL(run, grid_2d(xcd_grid(ceil_div(units, kWaves))),
                               dim3(kWaves * kWave), 0, st, a, (int32_t)tiles);
        }
        SG_LAUNCH_CHECK();
        if (a.ranges)
            join_parts<T, kMxEvenSeqs>(a, (int32_t)tiles, 16, G::KT, kProbShift<T>, st);
        else if (a.npieces > 1)
            paged_join(a, st);
    });
}

}  // namespace sg
