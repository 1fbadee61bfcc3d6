// One wavefront's share of softmax attention over a list of gathered keys:
// the tile operations that the attention kernels are put together from.
//
// A tile is 16 query rows (the query heads that share one key head, or
// neighbouring tokens too) against KT keys that lie anywhere in memory. Both
// products run on the matrix units with the keys on the side that needs no
// transpose of the probabilities:
//
//   S^T = K Q^T     A operand: K rows (lane l: key l%16), B operand: Q rows
//   O^T += V^T P^T  A operand: V^T (lane l: an index of the head dimension),
//                   B operand: P^T (lane l: query l%16)
//
// A 16x16 result holds, in lane l and register r, row 4*(l/16)+r of column
// l%16. So S^T leaves 4 keys of one query in each lane, which is what the B
// operand of the second product wants if its inner index numbers the keys as
// (4*(l/16)+r of the tile's first 16, then of its second 16): the
// probabilities never leave the lane, and a query's running maximum, sum and
// rescaling are one value per lane. V^T is not loaded transposed: each lane
// takes 16 bytes of each of its 8 keys' rows (16 lanes read a whole row), and
// the 8x8 block is turned over in registers with byte permutes; the c-th of
// the lane's 8 head-dimension indices goes into the c-th product.
#pragma once

#include "common.h"

namespace sg {

using f32x4 = float __attribute__((ext_vector_type(4)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f16x8 = _Float16 __attribute__((ext_vector_type(8)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using f16x2 = _Float16 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = (float)(1.44269504088896340736 - (double)kLog2e);
constexpr float kLn2 = 0.69314718055994530942f;

// exp2 and log2 of the vector unit (1 ulp; results below the smallest normal
// number become 0, which is far below the rounding of any sum they enter)
__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_log2(float x) { return __builtin_amdgcn_logf(x); }

// Two floats rounded to nearest even and packed, the first in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same<T, __bf16>::value)
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
    else
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}
template <class T>
__device__ __forceinline__ void unpack2(uint32_t x, float& a, float& b) {
    if constexpr (std::is_same<T, __bf16>::value) {
        a = __builtin_bit_cast(float, x << 16);
        b = __builtin_bit_cast(float, x & 0xffff0000u);
    } else {
        const f16x2 h = __builtin_bit_cast(f16x2, x);
        a = (float)h[0];
        b = (float)h[1];
    }
}

template <class T>
__device__ __forceinline__ f32x4 mfma32(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (std::is_same<T, __bf16>::value)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Largest / sum over the four lanes that hold one query (l%16 alike), by the
// vector unit's exchanges of 16 and of 32 lanes.
template <class Op>
__device__ __forceinline__ float quad_reduce(float x, Op op) {
    const uint32_t a = __builtin_bit_cast(uint32_t, x);
    const auto h = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    x = op(__builtin_bit_cast(float, (uint32_t)h[0]), __builtin_bit_cast(float, (uint32_t)h[1]));
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto f = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return op(__builtin_bit_cast(float, (uint32_t)f[0]), __builtin_bit_cast(float, (uint32_t)f[1]));
}
__device__ __forceinline__ float quad_max(float x) {
    return quad_reduce(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float quad_sum(float x) {
    return quad_reduce(x, [](float a, float b) { return a + b; });
}

// exp(scale * s - lse), with c + c_low = scale * log2(e). In single precision
// the roundings of c and of lse * log2(e), which would weigh |lse| times a
// rounding, are carried along; in the 16-bit types they are below the weight's
// own rounding unless |lse| passes 2^13. lse's rounding remains, |lse| times
// 2^-24, which of large scores is more than 1: a weight above 1 is taken as 1, so
// that none passes its type's range (minimum() keeps a NaN). An infinite lse (no
// row, or one that sees nothing) gives 0.
template <class T>
__device__ __forceinline__ float weight(float s, float c, float c_low, float lse) {
    const float a = lse == -INFINITY ? INFINITY : lse * kLog2e;
    float x = fmaf(s, c, -a);
    if constexpr (sizeof(T) == 4) {
        const float low = fmaf(lse, kLog2eLow, fmaf(lse, kLog2e, -a));
        x += a == INFINITY ? 0.f : fmaf(s, c_low, -low);
    }
    return __builtin_elementwise_minimum(fast_exp2(x), 1.f);
}

// Unsigned division of n < 2^31 by a divisor fixed at launch: with
// s = ceil(log2 d) and mul = floor(2^(31+s) / d) + 1, the error of
// mul * n / 2^(31+s) is below n * d / (d * 2^(31+s)) < 1 / d.
struct FastDiv {
    uint32_t d = 1, mul = 0, shift = 0;
    __host__ __device__ FastDiv() = default;
    __host__ explicit FastDiv(uint32_t d_) : d(d_) {
        if (d <= 1) return;
        uint32_t s = 0;
        while ((1ull << s) < d) ++s;
        mul = (uint32_t)((1ull << (31 + s)) / d + 1);
        shift = s - 1;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return d == 1 ? n : __umulhi(n, mul) >> shift;
    }
};

// The tile geometry for element type T and a head dimension padded to DP.
// FULL: the head dimension is DP itself, so that no chunk needs a check.
template <class T, int DP, bool FULL>
struct Tile {
    static constexpr bool kFull = FULL;
    static constexpr bool k16 = sizeof(T) == 2;
    static constexpr int KT = k16 ? 32 : 16;     // keys per tile
    static constexpr int KSUB = KT / 16;         // 16-key results of S^T
    static constexpr int VK = KT / 4;            // keys per lane
    static constexpr int QS = DP * (int)sizeof(T) / 64;  // 64-byte steps of a row
    static constexpr int CHL = k16 && DP >= 128 ? 8 : 4;  // head-dimension values per V chunk
    static constexpr int U = DP / (16 * CHL);    // V chunks per lane and key
    static constexpr int VW = CHL * (int)sizeof(T) / 4;   // words per V chunk

    struct RowFrag { u32x4 w[QS]; };        // a row as A or B operand of S^T
    struct Acc { f32x4 o[U][CHL]; };        // O^T
    struct Probs { uint32_t w[4]; };        // P^T as B operand (floats' bits if T is float)
    struct VBlock { uint32_t w[VK][VW]; };  // one V chunk of the lane's keys

    // The 16-byte pieces 4*t + l/16 of a row; pieces from row_bytes on are 0.
    static __device__ __forceinline__ void load_row(const char* row, int row_bytes, RowFrag& f) {
        const int at = 16 * (lane_id() >> 4);
#pragma unroll
        for (int t = 0; t < QS; ++t) {
            if (FULL || 64 * t + at < row_bytes)
                f.w[t] = *reinterpret_cast<const u32x4*>(row + 64 * t + at);
            else
                f.w[t] = u32x4{0, 0, 0, 0};
        }
    }
    // A query row for scores with the factor |c|, or 1 if c is 0 (see Softmax):
    // 0 times each value then, which is NaN for an infinity or a NaN.
    static __device__ __forceinline__ void sign_row(RowFrag& f, float c) {
        if (__builtin_expect(c > 0.f, 1)) return;
        if (c < 0.f) {
            const uint32_t flip = k16 ? 0x80008000u : 0x80000000u;
#pragma unroll
            for (int t = 0; t < QS; ++t) f.w[t] ^= flip;
        } else {
#pragma unroll
            for (int t = 0; t < QS; ++t)
                f.w[t] = u32x4{times0(f.w[t][0]), times0(f.w[t][1]), times0(f.w[t][2]),
                               times0(f.w[t][3])};
        }
    }
    static __device__ __forceinline__ uint32_t times0(uint32_t w) {
        if constexpr (k16) {
            float a, b;
            unpack2<T>(w, a, b);
            return pack2<T>(a * 0.f, b * 0.f);
        } else {
            return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, w) * 0.f);
        }
    }
    static __device__ __forceinline__ void zero_row(RowFrag& f) {
#pragma unroll
        for (int t = 0; t < QS; ++t) f.w[t] = u32x4{0, 0, 0, 0};
    }

    // c + A B^T over the head dimension, and over 64 bytes of it.
    static __device__ __forceinline__ f32x4 dot_step(u32x4 a, u32x4 b, f32x4 c) {
        if constexpr (k16) {
            return mfma32<T>(a, b, c);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, (uint32_t)a[j]),
                                                         __builtin_bit_cast(float, (uint32_t)b[j]),
                                                         c, 0, 0, 0);
            return c;
        }
    }
    static __device__ __forceinline__ f32x4 dot(const RowFrag& a, const RowFrag& b, f32x4 c) {
#pragma unroll
        for (int t = 0; t < QS; ++t) c = dot_step(a.w[t], b.w[t], c);
        return c;
    }
    // A B^T with the bits that the column pass gets, which takes rows of 1024
    // bytes by halves.
    static __device__ __forceinline__ f32x4 dot_halves(const RowFrag& a, const RowFrag& b) {
        f32x4 c[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int t = 0; t < QS; ++t) {
            const int half = kRowBytes == 1024 && t >= QS / 2;
            c[half] = dot_step(a.w[t], b.w[t], c[half]);
        }
        return kRowBytes == 1024 ? c[0] + c[1] : c[0];
    }
    // a . b of this lane's own row, summed as dot_halves() sums it.
    static __device__ __forceinline__ float dot_own(const RowFrag& a, const RowFrag& b) {
        const f32x4 all = dot_halves(a, b);
        const int n = lane_id() & 15;
        const float lo = n & 1 ? all[1] : all[0], hi = n & 1 ? all[3] : all[2];
        return __shfl(n & 2 ? hi : lo, 16 * (n >> 2) + n, kWave);
    }

    // The position in the tile of this lane's j-th key of P^T and V.
    static __device__ __forceinline__ int key_of(int j) {
        return 4 * (lane_id() >> 4) + (j & 3) + 16 * (j >> 2);
    }

    // Bytes from a row's start to this lane's chunk u, and whether the row has it.
    static __device__ __forceinline__ int chunk_at(int u) {
        return 4 * VW * (16 * u + (lane_id() & 15));
    }
    static __device__ __forceinline__ void load_chunk(const char* row, int u, int row_bytes,
                                                      uint32_t (&w)[VW]) {
        const int at = chunk_at(u);
        if (FULL || at < row_bytes) {
            if constexpr (VW == 4) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(row + at);
                w[0] = x[0]; w[1] = x[1]; w[2] = x[2]; w[3] = x[3];
            } else {
                const u32x2 x = *reinterpret_cast<const u32x2*>(row + at);
                w[0] = x[0]; w[1] = x[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < VW; ++i) w[i] = 0;
        }
    }

    static __device__ __forceinline__ void zero_acc(Acc& a) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < CHL; ++c) a.o[u][c] = f32x4{0, 0, 0, 0};
    }
    static __device__ __forceinline__ void scale_acc(Acc& a, float f) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < CHL; ++c) a.o[u][c] *= f;
    }

    // Whether words of the type's values hold an infinity or a NaN.
    template <int N>
    static __device__ __forceinline__ bool words_wild(const uint32_t (&w)[N]) {
        bool wild = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (k16) {
                constexpr uint32_t e = std::is_same<T, __bf16>::value ? 0x7f80u : 0x7c00u;
                wild |= (w[i] & e) == e || ((w[i] >> 16) & e) == e;
            } else {
                wild |= (w[i] & 0x7f800000u) == 0x7f800000u;
            }
        }
        return wild;
    }

    struct AccB;
    static __device__ __forceinline__ void scale_acc(AccB& a, float f) {
#pragma unroll
        for (int b = 0; b < DP / 16; ++b) a.o[b] *= f;
    }

    // P^T from the lane's KT/4 probabilities (in key_of order), rounded to T: the
    // matrix units take both factors in one type, and a second product with what
    // the rounding leaves would double the work on O. Each weight is off by up to
    // half a step, as the result itself is by its own rounding: the error against
    // 64 bits is 1.2 to 1.4 times that of the result's rounding alone.
    static __device__ __forceinline__ void pack_probs(const float (&p)[VK], Probs& out) {
        if constexpr (k16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) out.w[i] = pack2<T>(p[2 * i], p[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) out.w[i] = __builtin_bit_cast(uint32_t, p[i]);
        }
    }

    // O^T += V^T P^T for word i of chunk u: the accumulators o[u][c] of the
    // kPerWord values c that the word holds; w: the word of each of the
    // lane's keys.
    static constexpr int kPerWord = k16 ? 2 : 1;
    static __device__ __forceinline__ void accumulate_word(const uint32_t (&w)[VK], const Probs& p,
                                                           f32x4 (&o)[kPerWord]) {
        if constexpr (k16) {
            const u32x4 b{p.w[0], p.w[1], p.w[2], p.w[3]};
            u32x4 lo, hi;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x05040100u);
                hi[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], 0x07060302u);
            }
            o[0] = mfma32<T>(lo, b, o[0]);
            o[1] = mfma32<T>(hi, b, o[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, w[j]),
                                                            __builtin_bit_cast(float, p.w[j]),
                                                            o[0], 0, 0, 0);
        }
    }
    static __device__ __forceinline__ void accumulate(const VBlock& v, const Probs& p, int u,
                                                      Acc& a) {
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            uint32_t w[VK];
#pragma unroll
            for (int j = 0; j < VK; ++j) w[j] = v.w[j][i];
            f32x4 o[kPerWord];
#pragma unroll
            for (int c = 0; c < kPerWord; ++c) o[c] = a.o[u][kPerWord * i + c];
            accumulate_word(w, p, o);
#pragma unroll
            for (int c = 0; c < kPerWord; ++c) a.o[u][kPerWord * i + c] = o[c];
        }
    }
    // The weight that this lane's query gives to `key` of the tile.
    static __device__ __forceinline__ float prob_of(const Probs& p, int key) {
        const int j = (key & 3) + 4 * (key >> 4);
        const int i = k16 ? j >> 1 : j;
        const u32x4 all{p.w[0], p.w[1], p.w[2], p.w[3]};
        const uint32_t mine = all[i];
        const uint32_t w = __shfl(mine, 16 * ((key >> 2) & 3) + (lane_id() & 15), kWave);
        if constexpr (k16) {
            float x, y;
            unpack2<T>(w, x, y);
            return j & 1 ? y : x;
        } else {
            return __builtin_bit_cast(float, w);
        }
    }
    // O^T += V^T P^T for chunk u where v holds infinities or NaN and not every
    // query sees every key: such keys count as 0 in the product and are added
    // on their own in the lanes whose query sees them. row(key): a pointer to
    // the key's row, sees(key): whether this lane's query does.
    template <class Row, class Sees>
    static __device__ __forceinline__ void add_wild_keys(VBlock& v, const Probs& p, int u,
                                                         int row_bytes, Row&& row, Sees&& sees,
                                                         Acc& a) {
        uint32_t keys = wild_keys(v);
#pragma unroll
        for (int j = 0; j < VK; ++j)
            if (keys >> key_of(j) & 1)
#pragma unroll
                for (int i = 0; i < VW; ++i) v.w[j][i] = 0;
#pragma unroll 1
        for (; keys; keys &= keys - 1) {
            const int key = __builtin_ctz(keys);
            const char* at = row(key);
            const float w = prob_of(p, key);
            if (sees(key)) add_wild(at, w, u, row_bytes, a);
        }
    }
    // Not 0 (a NaN) if the chunk holds an infinity or a NaN: 0 times all of it.
    static __device__ __forceinline__ float chunk_zero(const uint32_t (&w)[VW], float z) {
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            if constexpr (std::is_same<T, __bf16>::value)
                z = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w[i]),
                                                    bf16x2{(__bf16)0.f, (__bf16)0.f}, z, false);
            else if constexpr (k16)
                z = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w[i]),
                                           f16x2{(_Float16)0.f, (_Float16)0.f}, z, false);
            else
                z = fmaf(__builtin_bit_cast(float, w[i]), 0.f, z);
        }
        return z;
    }
    // The keys (bits) whose chunk holds an infinity or a NaN.
    static __device__ __forceinline__ uint32_t wild_keys(const VBlock& v) {
        uint32_t keys = 0;
#pragma unroll
        for (int j = 0; j < VK; ++j) {
            const uint64_t b = __ballot(words_wild(v.w[j]));
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (b >> (16 * x) & 0xffff) keys |= 1u << (4 * x + (j & 3) + 16 * (j >> 2));
        }
        return keys;
    }

    // Rows staged in LDS, so that one trip to memory serves both operands.
    // The 16-byte pieces of a row are exchanged by the bits b0.. of its
    // number: by (b0, b1, b3, b2 ^ b4), which differs over 16 rows in
    // sequence (the same piece of each is read at once) and in its upper two
    // bits over every fourth and every eighth row (64 bytes of four such rows
    // are); for rows of 128 bytes, two to a line of the banks, by (b1, b2, b3).
    static constexpr int kDim = DP;
    static constexpr int kRowBytes = DP * (int)sizeof(T);
    static constexpr __device__ __forceinline__ int stage_x(int r) {
        return kRowBytes < 256 ? ((r >> 1) & 7) << 4
                               : ((r & 3) | ((r >> 3) & 1) << 2 | (((r >> 2) ^ (r >> 4)) & 1) << 3)
                                     << 4;
    }
    static __device__ __forceinline__ int stage_at(int r, int byte) {
        return r * kRowBytes + (byte ^ stage_x(r));
    }
    // stage_at(r | dr, byte | dbyte) from at = stage_at(r, byte), for constants
    // that share no bit with r and byte (the exchange is linear in the bits).
    static __device__ __forceinline__ int stage_more(int at, int dr, int dbyte) {
        return (at ^ dbyte ^ stage_x(dr)) + dr * kRowBytes;
    }
    // Where this lane's pieces of rows first + l % 16 and its chunks of rows
    // first + key_of(j) begin, for a tile whose first row is `first`; dr: a
    // constant, 0 or 16, more rows.
    static __device__ __forceinline__ int row_base(int first) {
        return stage_at(first + (lane_id() & 15), 16 * (lane_id() >> 4));
    }
    static __device__ __forceinline__ int chunk_base(int first) {
        return stage_at(first + 4 * (lane_id() >> 4), chunk_at(0));
    }
    static __device__ __forceinline__ void staged_row(const char* lds, int base, int dr,
                                                      RowFrag& f) {
#pragma unroll
        for (int t = 0; t < QS; ++t)
            f.w[t] = *reinterpret_cast<const u32x4*>(lds + stage_more(base, dr, 64 * t));
    }
    // dot() of two staged rows, of STEPS steps of 64 bytes from the bases on.
    template <int STEPS>
    static __device__ __forceinline__ f32x4 dot_staged(const char* a, int abase, const char* b,
                                                       int bbase) {
        f32x4 c{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < STEPS; ++t)
            c = dot_step(*reinterpret_cast<const u32x4*>(a + stage_more(abase, 0, 64 * t)),
                         *reinterpret_cast<const u32x4*>(b + stage_more(bbase, 0, 64 * t)), c);
        return c;
    }
    static __device__ __forceinline__ void stage_chunk(char* lds, int base, int j, int u,
                                                       const uint32_t (&w)[VW]) {
        char* at = lds + stage_more(base, (j & 3) + 16 * (j >> 2), 64 * VW * u);
        if constexpr (VW == 4)
            *reinterpret_cast<u32x4*>(at) = u32x4{w[0], w[1], w[2], w[3]};
        else
            *reinterpret_cast<u32x2*>(at) = u32x2{w[0], w[1]};
    }
    // The lane's chunks of a tile's rows.
    static __device__ __forceinline__ void stage_tile(char* lds, int base, const VBlock (&x)[U]) {
#pragma unroll
        for (int j = 0; j < VK; ++j)
#pragma unroll
            for (int u = 0; u < U; ++u) stage_chunk(lds, base, j, u, x[u].w[j]);
    }
    // Its keys from the `left`-th on as 0: 0 weight times what the row that
    // they repeat holds may be NaN.
    static __device__ __forceinline__ void clear_past(VBlock (&x)[U], int left) {
#pragma unroll
        for (int j = 0; j < VK; ++j)
            if (key_of(j) >= left)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < VW; ++i) x[u].w[j][i] = 0;
    }
    static __device__ __forceinline__ void staged_chunk(const char* lds, int base, int dr, int j,
                                                        int u, uint32_t (&w)[VW]) {
        const char* at = lds + stage_more(base, dr + (j & 3) + 16 * (j >> 2), 64 * VW * u);
        if constexpr (VW == 4) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(at);
            w[0] = x[0]; w[1] = x[1]; w[2] = x[2]; w[3] = x[3];
        } else {
            const u32x2 x = *reinterpret_cast<const u32x2*>(at);
            w[0] = x[0]; w[1] = x[1];
        }
    }

    // V^T from LDS, by blocks of 16 indices of the head dimension: lane l has
    // index 16 b + l%16 of its keys, turned over on the way by the transposing
    // read (16 lanes name 4 rows of 16 values and each gets a column).
    static constexpr int NB = DP / 16;
    struct AccB { f32x4 o[NB]; };  // register r of block b: index 16 b + 4 (l/16) + r
    static __device__ __forceinline__ int value_base(int first) {
        const int l = lane_id() & 15, quad = lane_id() >> 4;
        return k16 ? stage_at(first + 4 * quad + (l >> 2), 8 * (l & 3))
                   : stage_at(first + 4 * quad, 4 * l);
    }
    static __device__ __forceinline__ u32x4 value_frag(const char* lds, int base, int b) {
        if constexpr (k16) {
            using s16x4 = short __attribute__((ext_vector_type(4)));
            using lds_s16x4 = __attribute__((address_space(3))) s16x4;
            const u32x2 lo = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                           (lds_s16x4*)(lds + stage_more(base, 0, 32 * b))));
            const u32x2 hi = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                           (lds_s16x4*)(lds + stage_more(base, 16, 32 * b))));
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
        } else {
            u32x4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[r] = *reinterpret_cast<const uint32_t*>(lds + stage_more(base, r, 64 * b));
            return x;
        }
    }
    // v with 0 in place of the lane's keys j that on(j) denies.
    template <class On>
    static __device__ __forceinline__ u32x4 keep(u32x4 v, On&& on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (k16)
                v[i] &= (on(2 * i) ? 0xffffu : 0u) | (on(2 * i + 1) ? 0xffff0000u : 0u);
            else
                v[i] = on(i) ? v[i] : 0u;
        }
        return v;
    }
    static __device__ __forceinline__ f32x4 add_block(u32x4 v, const Probs& p, f32x4 o) {
        if constexpr (k16) {
            return mfma32<T>(v, u32x4{p.w[0], p.w[1], p.w[2], p.w[3]}, o);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                o = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, (uint32_t)v[r]),
                                                         __builtin_bit_cast(float, p.w[r]), o, 0, 0,
                                                         0);
            return o;
        }
    }
    // o += w times 4 values of type T.
    static __device__ __forceinline__ f32x4 add_four(const char* at, float w, f32x4 o) {
        if constexpr (k16) {
            const u32x2 x = *reinterpret_cast<const u32x2*>(at);
            float y[4];
            unpack2<T>(x[0], y[0], y[1]);
            unpack2<T>(x[1], y[2], y[3]);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = fmaf(w, y[r], o[r]);
        } else {
            const f32x4 y = *reinterpret_cast<const f32x4*>(at);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = fmaf(w, y[r], o[r]);
        }
        return o;
    }
    static __device__ __forceinline__ void store_four(f32x4 v, char* at) {
        if constexpr (k16)
            *reinterpret_cast<u32x2*>(at) = u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
        else
            *reinterpret_cast<f32x4*>(at) = v;
    }

    // Element index of the accumulator's first value in register r of chunk
    // u; the CHL values o[u][0..CHL)[r] follow one another.
    static __device__ __forceinline__ int dim_of(int u, int r) {
        return CHL * (16 * u + 4 * (lane_id() >> 4) + r);
    }
    // Register r of chunk u, times f, rounded to T and stored at row + dim_of.
    static __device__ __forceinline__ void store_out(const Acc& a, int u, int r, float f, char* row,
                                                     int row_bytes) {
        const int at = dim_of(u, r) * (int)sizeof(T);
        if (!FULL && at >= row_bytes) return;
        if constexpr (k16) {
            uint32_t w[VW];
#pragma unroll
            for (int i = 0; i < VW; ++i)
                w[i] = pack2<T>(a.o[u][2 * i][r] * f, a.o[u][2 * i + 1][r] * f);
            if constexpr (VW == 4)
                *reinterpret_cast<u32x4*>(row + at) = u32x4{w[0], w[1], w[2], w[3]};
            else
                *reinterpret_cast<u32x2*>(row + at) = u32x2{w[0], w[1]};
        } else {
            *reinterpret_cast<f32x4*>(row + at) =
                f32x4{a.o[u][0][r] * f, a.o[u][1][r] * f, a.o[u][2][r] * f, a.o[u][3][r] * f};
        }
    }
    // Chunk u of the row at `row`, times w.
    static __device__ __forceinline__ void add_wild(const char* row, float w, int u, int row_bytes,
                                                    Acc& a) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int at = dim_of(u, r) * (int)sizeof(T);
            if (!FULL && at >= row_bytes) continue;
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                const uint32_t y = *reinterpret_cast<const uint32_t*>(row + at + 4 * i);
                if constexpr (k16) {
                    float y0, y1;
                    unpack2<T>(y, y0, y1);
                    a.o[u][2 * i][r] = fmaf(w, y0, a.o[u][2 * i][r]);
                    a.o[u][2 * i + 1][r] = fmaf(w, y1, a.o[u][2 * i + 1][r]);
                } else {
                    a.o[u][i][r] = fmaf(w, __builtin_bit_cast(float, y), a.o[u][i][r]);
                }
            }
        }
    }
    // The same values as floats at dst (a row of the head dimension's floats).
    static __device__ __forceinline__ void store_part(const Acc& a, int u, int r, float f,
                                                      float* dst, int dim) {
        const int at = dim_of(u, r);
        if (!FULL && at >= dim) return;
#pragma unroll
        for (int c = 0; c < CHL; c += 4)
            *reinterpret_cast<f32x4*>(dst + at + c) =
                f32x4{a.o[u][c][r] * f, a.o[u][c + 1][r] * f, a.o[u][c + 2][r] * f,
                      a.o[u][c + 3][r] * f};
    }
};

// Half precision keeps only 2^-24 absolutely: probabilities are held times
// 2^14 there, so that the many small ones of a long row keep their 11 bits
// (the largest is 2^14, a quarter of the type's range). The sum carries the
// same factor.
template <class T>
constexpr float kProbShift = std::is_same<T, _Float16>::value ? 14.f : 0.f;

// The keys of a tile that this lane's query sees: bit (j & 3) + 16 * (j >> 2)
// for the lane's j-th key.
struct Seen {
    uint32_t bits;
    // from a tile's keys as bits 0 to 31
    static __device__ __forceinline__ Seen keys(uint32_t all) {
        return {all >> (4 * (lane_id() >> 4))};
    }
    static __device__ __forceinline__ Seen first(int n) {
        return keys(n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1);
    }
    // x if the lane's j-th key is seen, else y (by bits: whatever x holds)
    __device__ __forceinline__ float pick(int j, float x, float y) const {
        const int at = (j & 3) + 16 * (j >> 2);
        const uint32_t on = (uint32_t)((int32_t)(bits << (31 - at)) >> 31);
        return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & on) |
                                             (__builtin_bit_cast(uint32_t, y) & ~on));
    }
};

// The running maximum (base 2) and sum of a softmax, of this lane's query;
// the sum covers this lane's keys only until finish().
template <class G, class T>
struct Softmax {
    // Single precision keeps m before its factor until finish(): the largest
    // weight is 1 to the last bit then, and a row's only key gives its value
    // unchanged. 16 bits round that difference away, unless m is far from 0:
    // from 2^12 on its own rounding, and that of the shift minus it, up to
    // 2^-24 of it each, are not small beside a weight's, and from about 2^24 on 2
    // to the power of them, which is what the largest weight becomes, passes the
    // types' ranges at either end. There the products are rounded as the
    // maximum's was, which makes it 1 again and takes two instructions a weight
    // for one.
    static constexpr bool kLate = sizeof(T) == 4;
    static constexpr float kFar = 4096.f;
    float m = -INFINITY, l = 0.f;

    // Takes NS tiles' scores before their factor c > 0 (a negative one's sign
    // goes into q, and 0 makes q 0; -infinity for a key that does not count)
    // and leaves the weights; returns the factor of what was summed before.
    // far: whether this lane's query is so; without EXACT it is left at that.
    template <bool EXACT, int NS>
    __device__ __forceinline__ float weigh(const f32x4 (&s)[NS][G::KSUB], float c,
                                           typename G::Probs (&out)[NS], bool& far) {
        float top = s[0][0][0];
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int j = 0; j < G::VK; ++j) top = fmaxf(top, s[i][j >> 2][j & 3]);
        const float mn = fmaxf(m, kLate ? quad_max(top) : quad_max(top) * c);
        const float ms = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: weights 0, not NaN
        const float fix = fast_exp2(kLate ? (m - ms) * c : m - ms);
        m = mn;
        far = !kLate && fabsf(ms) >= kFar;
        const float base = kProbShift<T> - ms;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float p[G::VK];
#pragma unroll
            for (int j = 0; j < G::VK; ++j) {
                const float x = s[i][j >> 2][j & 3];
                p[j] = kLate ? (x - ms) * c : fmaf(x, c, base);
            }
            if (EXACT && __builtin_expect(__any(far), 0)) {
#pragma clang fp contract(off)
#pragma unroll
                for (int j = 0; j < G::VK; ++j) {
                    const float apart = s[i][j >> 2][j & 3] * c - ms + kProbShift<T>;
                    p[j] = far ? apart : p[j];
                }
            }
#pragma unroll
            for (int j = 0; j < G::VK; ++j) {
                p[j] = fast_exp2(p[j]);
                sum += p[j];
            }
            G::pack_probs(p, out[i]);
        }
        l = l * fix + sum;
        return fix;
    }
    // After weigh<false> where some query was far: its weights EXACT, from the
    // scores that it had (other queries' results keep their bits). old: l before.
    template <int NS>
    __device__ __forceinline__ void weigh_far(const f32x4 (&s)[NS][G::KSUB], float c, float old,
                                              float fix, typename G::Probs (&out)[NS]) {
        const float near = l;
        bool far;
        l = old * fix;
        (void)weigh<true>(s, c, out, far);
        l = far ? l : near;
    }
    // weigh() of one tile's keys that are seen, and o rescaled.
    __device__ __forceinline__ void step(f32x4 (&s)[1][G::KSUB], Seen seen, float c,
                                         typename G::Acc& o, typename G::Probs (&out)[1]) {
        hide(s[0], seen);
        bool far;
        const float fix = weigh<true>(s, c, out, far);
        if (__any(fix != 1.f)) G::scale_acc(o, fix);
    }
    static __device__ __forceinline__ void hide(f32x4 (&s)[G::KSUB], Seen seen) {
#pragma unroll
        for (int j = 0; j < G::VK; ++j)
            s[j >> 2][j & 3] = seen.pick(j, s[j >> 2][j & 3], -INFINITY);
    }
    __device__ __forceinline__ void finish(float c) {
        l = quad_sum(l);
        if (sizeof(T) == 4) m *= c;
    }
    __device__ __forceinline__ float factor() const { return l == 0.f ? 0.f : 1.f / l; }
    __device__ __forceinline__ float lse() const {
        return l == 0.f ? -INFINITY : (m - kProbShift<T> + fast_log2(l)) * kLn2;
    }
};

// Joins `count` partial results of dim floats, `step` floats apart, by one
// wavefront: the four rows of 16 lanes take every fourth piece, four values a
// lane, so that a long chain of pieces is a quarter as long and its loads
// wide; they are added up at the end, in the same order every time.
struct JoinedRow {
    static constexpr int kParts = 4;  // of 64 values
    f32x4 x[kParts];
    // weight(i): the factor of piece i
    template <class Weight>
    __device__ __forceinline__ JoinedRow(const float* part, int64_t step, int count, int dim,
                                         Weight&& weight) {
        const int at = 4 * (lane_id() & 15);
#pragma unroll
        for (int j = 0; j < kParts; ++j) x[j] = f32x4{0, 0, 0, 0};
#pragma unroll 2
        for (int i = lane_id() >> 4; i < count; i += 4) {
            const float w = weight(i);
            const float* src = part + i * step;
#pragma unroll
            for (int j = 0; j < kParts; ++j)
                if (64 * j + at < dim)
                    x[j] += *reinterpret_cast<const f32x4*>(src + 64 * j + at) * w;
        }
#pragma unroll
        for (int j = 0; j < kParts; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) x[j][r] = quad_sum(x[j][r]);
    }
    // The values times f, rounded to T.
    template <class T>
    __device__ __forceinline__ void store(char* row, float f, int dim) const {
        const int j = lane_id() >> 4, at = 64 * j + 4 * (lane_id() & 15);
        if (at >= dim) return;
        const f32x4 y = (j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3]) * f;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<u32x2*>(row + 2 * at) = u32x2{pack2<T>(y[0], y[1]),
                                                            pack2<T>(y[2], y[3])};
        else
            *reinterpret_cast<f32x4*>(row + 4 * at) = y;
    }
};
// The largest maximum and the sum of softmax partials (maximum, sum) `step`
// pairs apart, by one wavefront.
__device__ __forceinline__ void join_sums(const float* ml, int64_t step, int count, float& m,
                                          float& l) {
    m = -INFINITY;
    for (int i = lane_id(); i < count; i += kWave) m = fmaxf(m, ml[2 * i * step]);
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
    m = m == -INFINITY ? 0.f : m;
    l = 0.f;
    for (int i = lane_id(); i < count; i += kWave)
        l += ml[2 * i * step + 1] * fast_exp2(ml[2 * i * step] - m);
    l = wave_reduce_sum(l);
}

// Calls f(Tag<T, DP, FULL>) for the run-time element type and head dimension.
template <class T, int DP, bool FULL>
struct TileTag {
    using Elem = T;
    using Geo = Tile<T, DP, FULL>;
};
template <class T, class F>
void with_dim(int dim, F&& f) {
    if (dim == 64) f(TileTag<T, 64, true>{});
    else if (dim < 64) f(TileTag<T, 64, false>{});
    else if (dim == 128) f(TileTag<T, 128, true>{});
    else if (dim < 128) f(TileTag<T, 128, false>{});
    else if (dim == 256) f(TileTag<T, 256, true>{});
    else f(TileTag<T, 256, false>{});
}

}  // namespace sg
