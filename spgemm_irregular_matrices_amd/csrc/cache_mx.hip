// Writing new tokens into a quantised cache, and reading a cache back.
#include "mx.h"

namespace sg {

namespace {

constexpr int kWaves = 4;
constexpr int kEach = 8;   // values per lane and step
constexpr int kSteps = 4;  // steps per wavefront, all under way at once: keys and values in turn
constexpr int kSides = 2;

// Largest index s in [0, n) with a[s] <= x (ascending; 0 if there is none), 64 lanes at a time.
__device__ __forceinline__ int64_t wave_upper_index(const int64_t* a, int64_t n, int64_t x) {
    int64_t lo = 0;
    while (n > 1) {
        const int64_t step = (n + kWave - 1) / kWave;
        const int64_t at = lane_id() * step;
        const uint64_t below = __ballot(at < n && a[lo + at] <= x);
        const int64_t first = below ? (63 - __builtin_clzll(below)) * step : 0;
        lo += first;
        n = min(step, n - first);
    }
    return lo;
}

// Where a new token lies in the cache.
struct Slot {
    bool row;   // the token is a row of a sequence
    bool there; // and has a place
    uint32_t id, slot;
};
__device__ __forceinline__ Slot find_slot(const MxRowsArgs& a, int64_t token) {
    Slot x{false, false, 0, 0};
    Sequence sq;
    int64_t s = wave_upper_index(a.q_rowptr, a.seqs, token);
    if (!find_sequence(a, token, s, sq)) return x;
    x.row = true;
    if (sq.bad) return x;
    const uint32_t at = (uint32_t)(sq.length - sq.fresh + (int)(token - sq.q0));
    const uint32_t pg = a.page_div.div(at);
    x.id = __builtin_amdgcn_readfirstlane(a.col[sq.page0 + pg]);  // (all lanes have the same)
    x.slot = __builtin_amdgcn_readfirstlane(at - pg * a.page_div.d);
    x.there = x.id < (uint64_t)a.npages;
    return x;
}

// This lane's values of a pair of steps: head, first value. (Whether a step is of
// keys or of values is known where the kernel is compiled, and a token's place is
// the same in all lanes: addresses but for these are made once, in scalars. By
// lanes, the vector unit was 87 % busy with them: 15 K tokens were written and read
// in 26 + 22 us for 22 + 15.)
struct Part {
    bool has;
    int h, d;
};
__device__ __forceinline__ Part part_of(const MxRowsArgs& a, FastDiv per_head, int part, int pair) {
    const int x = (part * (kSteps / kSides) + pair) * kWave + lane_id();
    Part p;
    p.h = (int)per_head.div(x);
    p.has = p.h < a.s.hkv;
    p.d = kEach * (x - p.h * (int)per_head.d);
    return p;
}
// Of one side of the cache or of the rows: where a token's begin, and its heads' stride.
struct Side {
    char* at;
    int64_t head;
};
__device__ __forceinline__ Side codes_of(const MxRowsArgs& a, const Slot& t, bool value) {
    const uint32_t place = value ? t.id * a.v_page + t.slot * a.v_slot : t.id * a.k_page + t.slot * a.k_slot;
    return {const_cast<char*>(value ? a.v : a.k) + ((uint64_t)place << (value ? a.v_shift : a.k_shift)),
            value ? a.v_head : a.k_head};
}
__device__ __forceinline__ Side scales_of(const MxRowsArgs& a, const Slot& t, bool value) {
    const uint32_t place =
        value ? t.id * a.vs_page + t.slot * a.vs_slot : t.id * a.ks_page + t.slot * a.ks_slot;
    return {(char*)const_cast<uint8_t*>(value ? a.vs : a.ks) +
                ((uint64_t)place << (value ? a.vs_shift : a.ks_shift)),
            value ? a.vs_head : a.ks_head};
}
__device__ __forceinline__ Side rows_of(const MxRowsArgs& a, int64_t token, bool value) {
    const AttnRows& r = value ? a.rv : a.rk;
    return {r.base + token * r.row, r.head};
}
// This wavefront's token and part of it.
__device__ __forceinline__ int64_t token_of(int32_t parts, int& part) {
    const int64_t unit = grid_block() * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t token = parts == 1 ? unit : unit / parts;
    part = (int)(unit - token * parts);
    return token;
}

template <class T>
__device__ __forceinline__ void load_values(const char* at, float (&x)[kEach]) {
    if constexpr (sizeof(T) == 2) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2<T>(w[i], x[2 * i], x[2 * i + 1]);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x4 y = reinterpret_cast<const f32x4*>(at)[j];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * j + i] = y[i];
        }
    }
}

// Largest of the four lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xb1, 0xf, 0xf, true));  // lanes 1, 0, 3, 2
    return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4e, 0xf, 0xf, true));  // 2, 3, 0, 1
}

// One wavefront takes kSteps * 64 pieces of 8 values of one token. Its rows are
// on their way before it looks its token's place up. Bound by bytes where tokens are
// many (15 K, 8 heads of 128, half to 4 bits, 78 MB: 22 us), by the chain of loads to
// the place where they are few (one token: 3 us).
template <class T, int BITS>
__global__ __launch_bounds__(kWaves* kWave) void k_mx_write(MxRowsArgs a, int32_t parts,
                                                            FastDiv per_head) {
    int part;
    const int64_t token = token_of(parts, part);
    if (token >= a.tokens) return;
    float x[kSteps][kEach];
    Part p[kSteps / kSides];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        Part& y = p[i / kSides];
        if (i % kSides == 0) y = part_of(a, per_head, part, i / kSides);
        if (!y.has) continue;
        const Side r = rows_of(a, token, i % kSides);
        load_values<T>(r.at + y.h * r.head + y.d * (int)sizeof(T), x[i]);
    }
    const Slot at = find_slot(a, token);
    if (!at.there) return;
    constexpr float kMost = BITS == 8 ? 1.75f : 1.5f;  // of 2^kTop
    constexpr int kTop = BITS == 8 ? 8 : 2;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const Part& y = p[i / kSides];
        if (!y.has) continue;  // (whole blocks: head_dim is a multiple of 32)
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            top = max(top, __builtin_bit_cast(uint32_t, x[i][j]) & 0x7fffffffu);
        top = block_max(top);
        // a = 2^(exponent - 127) * (1 + fraction); a subnormal one is far below 2^-117
        constexpr uint32_t kFraction = (uint32_t)((kMost - 1.f) * 8388608.f);
        const int e = (int)(top >> 23) - kTop + ((top & 0x7fffffu) > kFraction ? 1 : 0);
        const bool wild = top >= 0x7f800000u;
        const uint32_t byte = wild ? 255u : (uint32_t)max(e, 127 - 117);
        const float scale = mx_scale(wild ? 127u : byte);
        uint32_t w[2] = {0, 0};
        if constexpr (BITS == 8) {
            using s16x2 = short __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s16x2 c{0, 0};
                c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[i][4 * j], x[i][4 * j + 1], scale, false);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[i][4 * j + 2], x[i][4 * j + 3], scale, true);
                w[j] = wild ? 0u : __builtin_bit_cast(uint32_t, c);
            }
        } else {
            uint32_t c = 0;
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[i][0], x[i][1], scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[i][2], x[i][3], scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[i][4], x[i][5], scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[i][6], x[i][7], scale, 3);
            w[0] = wild ? 0u : c;
        }
        const Side c = codes_of(a, at, i % kSides), z = scales_of(a, at, i % kSides);
        char* codes = c.at + y.h * c.head + y.d * BITS / 8;
        if constexpr (BITS == 8)
            *reinterpret_cast<u32x2*>(codes) = u32x2{w[0], w[1]};
        else
            *reinterpret_cast<uint32_t*>(codes) = w[0];
        if ((lane_id() & 3) == 0)
            z.at[y.h * z.head + y.d / SPGEMM_MX_BLOCK] = (char)byte;
    }
}

// The reverse, split alike; bound by bytes: 921 MB of 8-bit texts read and written as
// bfloat16 take 178 us, 5.2 TB/s.
template <class T, int BITS>
__global__ __launch_bounds__(kWaves* kWave) void k_mx_read(MxRowsArgs a, int32_t parts,
                                                              FastDiv per_head) {
    int part;
    const int64_t token = token_of(parts, part);
    if (token >= a.tokens) return;
    const Slot at = find_slot(a, token);
    if (!at.row) return;
    uint32_t w[kSteps][BITS / 4], scale[kSteps];
    Part p[kSteps / kSides];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        Part& y = p[i / kSides];
        if (i % kSides == 0) y = part_of(a, per_head, part, i / kSides);
        scale[i] = 255;
#pragma unroll
        for (int j = 0; j < BITS / 4; ++j) w[i][j] = 0;
        if (!y.has || !at.there) continue;
        const Side c = codes_of(a, at, i % kSides), z = scales_of(a, at, i % kSides);
        const char* codes = c.at + y.h * c.head + y.d * BITS / 8;
        if constexpr (BITS == 8) {
            const u32x2 y = *reinterpret_cast<const u32x2*>(codes);
            w[i][0] = y[0];
            w[i][1] = y[1];
        } else {
            w[i][0] = *reinterpret_cast<const uint32_t*>(codes);
        }
        scale[i] = (uint8_t)z.at[y.h * z.head + y.d / SPGEMM_MX_BLOCK];
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const Part& y = p[i / kSides];
        if (!y.has) continue;
        const Side r = rows_of(a, token, i % kSides);
        char* row = r.at + y.h * r.head + y.d * (int)sizeof(T);
        if constexpr (std::is_same<T, __bf16>::value) {
            *reinterpret_cast<u32x4*>(row) = mx_decode8<BITS>(w[i], mx_scale(scale[i]));
        } else {
            float f[kEach];
            mx_decode8_float<BITS>(w[i], mx_scale(scale[i]), f);
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<u32x4*>(row) = u32x4{pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]),
                                                       pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7])};
            } else {
                reinterpret_cast<f32x4*>(row)[0] = f32x4{f[0], f[1], f[2], f[3]};
                reinterpret_cast<f32x4*>(row)[1] = f32x4{f[4], f[5], f[6], f[7]};
            }
        }
    }
}

template <class F>
void with_bits(int type, int format, F&& f) {
    const auto go = [&](auto bits) {
        if (type == SPGEMM_TYPE_BF16) f((__bf16*)nullptr, bits);
        else if (type == SPGEMM_TYPE_F16) f((_Float16*)nullptr, bits);
        else f((float*)nullptr, bits);
    };
    if (format == SPGEMM_MX_E4M3) go(std::integral_constant<int, 8>{});
    else go(std::integral_constant<int, 4>{});
}

template <class Kernel>
void launch_rows(Kernel run, const MxRowsArgs& a, hipStream_t st) {
    if (a.tokens == 0 || a.seqs == 0) return;
    const int per_head = a.s.dim / kEach;
    const int parts = (int)ceil_div((int64_t)a.s.hkv * per_head, kSteps / kSides * kWave);
    hipLaunchKernelGGL(run, grid_2d(ceil_div(a.tokens * parts, kWaves)), dim3(kWaves * kWave), 0, st,
                       a, parts, FastDiv((uint32_t)per_head));
    SG_LAUNCH_CHECK();
}

}  // namespace

void mx_write(const MxRowsArgs& a, hipStream_t st) {
    with_bits(a.s.type, a.format, [&](auto* t, auto bits) {
        launch_rows(k_mx_write<std::remove_pointer_t<decltype(t)>, decltype(bits)::value>, a, st);
    });
}
void mx_read(const MxRowsArgs& a, hipStream_t st) {
    with_bits(a.s.type, a.format, [&](auto* t, auto bits) {
        launch_rows(k_mx_read<std::remove_pointer_t<decltype(t)>, decltype(bits)::value>, a, st);
    });
}

}  // namespace sg
