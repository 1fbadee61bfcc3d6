// Checks of arguments that the attention entry points share, and what their
// launches are described by.
#pragma once

#include <algorithm>
#include <cmath>
#include <new>

#include "attention.h"

namespace sg {

inline int type_size(int32_t t) { return t == SPGEMM_TYPE_F32 ? 4 : 2; }

inline bool desc_valid(const spgemm_attention_desc* d) {
    if (!d || d->type < SPGEMM_TYPE_BF16 || d->type > SPGEMM_TYPE_F32) return false;
    if (d->heads_q < 1 || d->heads_kv < 1 || d->heads_q > SPGEMM_ATTENTION_MAX_HEADS ||
        d->heads_q % d->heads_kv != 0)
        return false;
    if (d->head_dim < 1 || d->head_dim > SPGEMM_ATTENTION_MAX_HEAD_DIM ||
        d->head_dim * type_size(d->type) % 16 != 0)
        return false;
    return std::isfinite(d->scale) && std::fabs(d->scale) < 1e30;
}

inline AttnShape make_shape(const spgemm_attention_desc* d) {
    AttnShape s;
    s.type = d->type;
    s.hq = d->heads_q;
    s.hkv = d->heads_kv;
    s.group = s.hq / s.hkv;
    s.dim = d->head_dim;
    s.scale = (float)d->scale;
    s.c = (float)(d->scale * 1.4426950408889634);
    s.c_low = (float)(d->scale * 1.4426950408889634 - (double)s.c);
    s.mag = s.c == 0.f ? 1.f : std::fabs(s.c);
    return s;
}

// A stride over a dimension of n places, in bytes: 0 where it is never used.
// -1 if it is not a stride this library takes.
constexpr int64_t kMaxStride = int64_t(1) << 40;
inline int64_t stride_bytes(int64_t stride, int64_t n, int size) {
    if (n <= 1) return 0;
    if (stride < 0 || stride > kMaxStride || stride * size % 16 != 0) return -1;
    return stride * size;
}

inline bool rows_valid(const spgemm_rows* x, int64_t n, int32_t heads, const spgemm_attention_desc* d,
                bool output, AttnRows* r) {
    if (!x) return false;
    if (n == 0) return true;  // no element: nothing of it is used
    const int size = type_size(d->type);
    r->base = static_cast<char*>(x->data);
    r->row = stride_bytes(x->stride_row, n, size);
    r->head = stride_bytes(x->stride_head, heads, size);
    if (!r->base || reinterpret_cast<uintptr_t>(r->base) % 16 != 0 || r->row < 0 || r->head < 0)
        return false;
    if (!output) return true;
    // rows of an output do not overlap: one dimension's stride passes the
    // whole of the other
    const int64_t line = (int64_t)d->head_dim * size;
    const __int128 heads_span = (__int128)r->head * (heads - 1) + line;
    const __int128 rows_span = (__int128)r->row * (n - 1) + line;
    const bool rows_out = (heads == 1 || r->head >= line) && (n == 1 || r->row >= heads_span);
    const bool heads_out = (n == 1 || r->row >= line) && (heads == 1 || r->head >= rows_span);
    return rows_out || heads_out;
}

// The largest power of two that divides every (nonzero) stride, and whether
// the extent in units of it fits 32 bits.
inline bool gather_unit(const int64_t* strides, const int64_t* counts, int n, uint32_t* shift) {
    int64_t all = int64_t(1) << 30;
    for (int i = 0; i < n; ++i) all |= strides[i];
    *shift = (uint32_t)__builtin_ctzll((unsigned long long)all);
    __int128 span = 0;
    for (int i = 0; i < n; ++i)
        if (counts[i] > 1) span += (__int128)(strides[i] >> *shift) * (counts[i] - 1);
    return span <= 0xffffffffLL;
}

// Carves a workspace into 256-byte aligned parts.
struct Carver {
    char* base;
    int64_t used = 0;
    float* take(__int128 floats) {
        const int64_t at = used;
        const __int128 end = (__int128)at + (floats * 4 + 255) / 256 * 256;
        if (end > ((__int128)1 << 60)) throw OverflowError("workspace size");
        used = (int64_t)end;
        return base && floats > 0 ? reinterpret_cast<float*>(base + at) : nullptr;
    }
};

inline bool workspace_valid(const void* ws, int64_t bytes, int64_t need) {
    return need == 0 || (ws && reinterpret_cast<uintptr_t>(ws) % 256 == 0 && bytes >= need);
}

inline bool batch_sizes_valid(const spgemm_paged_batch* b) {
    return b && b->pages && b->pages->nrows >= 0 && b->tokens >= 0 && b->max_new >= 0 &&
           b->max_length >= 0;
}
constexpr int64_t kMaxTokens = int64_t(1) << 30;
// A tile's rows are counted in 32 bits, those of its last one past the end too.
constexpr int64_t kMaxPairs = (int64_t(1) << 31) - kPagedTileMost;
inline bool batch_sizes_fit(const spgemm_paged_batch* b, const spgemm_attention_desc* d) {
    return b->pages->nrows < kMaxTokens && b->tokens <= kMaxTokens &&
           b->max_length <= kMaxTokens && b->tokens * d->heads_q <= kMaxPairs;
}

template <class F>
int guarded(F&& f) {
    try {
        return f();
    } catch (const OomError&) {
        return SPGEMM_ERR_OUT_OF_MEMORY;
    } catch (const OverflowError&) {
        return SPGEMM_ERR_OVERFLOW;
    } catch (const HipError& e) {
        return e.code == hipErrorOutOfMemory ? SPGEMM_ERR_OUT_OF_MEMORY : SPGEMM_ERR_HIP;
    } catch (const std::bad_alloc&) {
        return SPGEMM_ERR_OUT_OF_MEMORY;
    } catch (...) {
        return SPGEMM_ERR_HIP;
    }
}

}  // namespace sg
