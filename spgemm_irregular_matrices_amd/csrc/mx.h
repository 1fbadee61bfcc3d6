// Quantised caches (include/spgemm_cache.h): blocks of 32 values with a power
// of two as scale, codes of 8 or 4 bits. The codes' conversions are single
// instructions that take the scale as a float whose exponent they use.
#pragma once

#include "../../include/spgemm_cache.h"
#include "attention_paged.h"

namespace sg {

struct MxArgs : PagedArgs {  // k, v and their strides: the codes'
    const uint8_t* ks = nullptr;
    const uint8_t* vs = nullptr;
    uint32_t ks_page = 0, ks_slot = 0, vs_page = 0, vs_slot = 0;
    uint32_t ks_shift = 0, vs_shift = 0;
    int64_t ks_head = 0, vs_head = 0;  // bytes
    int format = 0;
};
// dim values of the new tokens' rows: k, v of `rows`; in: to the cache
struct MxRowsArgs : MxArgs {
    AttnRows rk, rv;
};
constexpr int kMxEvenSeqs = 256;  // sequences that are cut evenly
constexpr int kMxKeys = 32;  // keys per tile of single wavefronts
void mx_write(const MxRowsArgs& a, hipStream_t st);
void mx_read(const MxRowsArgs& a, hipStream_t st);
void mx_attention(const MxArgs& a, hipStream_t st);
bool mx_wide(const AttnShape& s, int64_t rows);
int mx_tile_rows(const AttnShape& s, int64_t rows);

// A scale's byte as the conversions take it (0 is 2^-127, 255 NaN).
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __builtin_bit_cast(float, byte << 23);
}

// 8 codes as 8 bfloat16 values: exact, but for those past its range.
template <int BITS>
__device__ __forceinline__ u32x4 mx_decode8(const uint32_t* w, float scale) {
    u32x4 x;
    if constexpr (BITS == 8) {
        x[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, false));
        x[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, true));
        x[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, false));
        x[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, true));
    } else {
        x[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 0));
        x[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 1));
        x[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 2));
        x[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 3));
    }
    return x;
}

// 8 codes as floats: exact, but for those past the type's range.
template <int BITS>
__device__ __forceinline__ void mx_decode8_float(const uint32_t* w, float scale, float (&x)[8]) {
    using f32x2 = float __attribute__((ext_vector_type(2)));
    f32x2 y[4];
    if constexpr (BITS == 8) {
        y[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], scale, false);
        y[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], scale, true);
        y[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], scale, false);
        y[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], scale, true);
    } else {
        y[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], scale, 0);
        y[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], scale, 1);
        y[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], scale, 2);
        y[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], scale, 3);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = y[i][0];
        x[2 * i + 1] = y[i][1];
    }
}

}  // namespace sg
