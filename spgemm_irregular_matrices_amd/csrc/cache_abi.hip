// Argument checks and the C ABI of include/spgemm_cache.h.
#include <algorithm>

#include "attention_checks.h"
#include "latent.h"
#include "mx.h"
#include "overlap.h"

using namespace sg;

namespace {

// ---------------------------------------------------------------- batches
// What every call over a paged cache checks of its batch and cache: OK with
// *empty set where there is nothing to do.
int paged_checks(const spgemm_paged_batch* b, const AttnShape& s, int64_t npages, int64_t page_size,
                 PagedArgs* a, bool* empty) {
    const spgemm_csr* pg = b->pages;
    if (pg->nnz < 0 || npages < 0 || page_size < 1 || pg->ncols != npages)
        return SPGEMM_ERR_INVALID_ARG;
    if (pg->nnz > 0x7fffffffLL || npages > 0x7fffffffLL || page_size > kMaxTokens)
        return SPGEMM_ERR_OVERFLOW;
    *empty = a->seqs == 0 || a->tokens == 0 || a->max_new == 0;
    if (*empty) return SPGEMM_OK;
    if (!pg->rowptr || (pg->nnz > 0 && !pg->col) || !b->q_rowptr || !b->lengths)
        return SPGEMM_ERR_INVALID_ARG;
    a->npages = npages;
    a->page_div = FastDiv((uint32_t)page_size);
    a->group_div = FastDiv((uint32_t)s.group);
    a->room = pg->nnz;
    a->rowptr = pg->rowptr;
    a->col = pg->col;
    a->q_rowptr = b->q_rowptr;
    a->lengths = b->lengths;
    return SPGEMM_OK;
}

void batch_shape(const spgemm_paged_batch* b, const AttnShape& s, PagedArgs* a) {
    a->s = s;
    a->seqs = b->pages->nrows;
    a->tokens = b->tokens;
    a->max_new = (int32_t)std::min(b->max_new, b->tokens);
    a->max_length = (int32_t)b->max_length;
}

// Pieces of the keys, so that `target` units (wavefronts with keys of their own,
// or work groups) are there, with at least `least` keys and a multiple of
// `step` keys each.
void cut_pieces(PagedArgs* a, int64_t tile, int64_t target, int64_t least, int64_t step) {
    const int64_t rows = (int64_t)a->max_new * a->s.group;
    const int64_t whole_tiles = a->seqs * ceil_div(rows, tile);
    const int64_t tiles = std::min(whole_tiles, a->seqs + a->tokens * a->s.group / tile);
    const int64_t units = std::max<int64_t>(a->s.hkv * tiles, 1);
    const int64_t most = std::max<int64_t>(ceil_div(a->max_length, least), 1);
    const int64_t want = std::min(std::max<int64_t>(target / units, 1), most);
    a->piece = (int32_t)std::max<int64_t>(
        ceil_div(ceil_div(a->max_length, want), step) * step, step);
    a->npieces = (int32_t)std::max<int64_t>(ceil_div(a->max_length, a->piece), 1);
}

// tile_rows: rows of a tile, heads: key heads whose ranges are apart.
int64_t carve_parts(void* ws, PagedArgs* a, int64_t tile_rows = 1, int64_t heads = 1) {
    const int64_t tiles = ceil_div((int64_t)a->max_new * a->s.group, tile_rows);
    Carver c{static_cast<char*>(ws)};
    if (a->ranges > 0) {
        const __int128 rows = (__int128)2 * a->ranges * tiles * tile_rows * heads;
        a->part = c.take(rows * a->s.dim);
        a->part_ml = c.take(rows * 2);
    } else if (a->npieces > 1) {
        const __int128 rows = (__int128)a->npieces * a->tokens * a->s.hq;
        a->part = c.take(rows * a->s.dim);
        a->part_ml = c.take(rows * 2);
    }
    return c.used;
}

// ---------------------------------------------------------------- quantised
bool mx_desc_valid(const spgemm_attention_desc* d) {
    return desc_valid(d) && d->head_dim % SPGEMM_MX_BLOCK == 0;
}

// One tensor of bytes: its strides in units of 1 << shift. align: of data and
// strides.
int mx_bytes(const spgemm_mx_bytes& x, const spgemm_mx_cache* cache, int heads, int align,
             const char** base, int64_t* head, uint32_t* page, uint32_t* slot, uint32_t* shift) {
    const int64_t counts[2] = {cache->npages, cache->page_size};
    const auto bytes = [&](int64_t stride, int64_t n) -> int64_t {
        if (n <= 1) return 0;
        return stride < 0 || stride > kMaxStride || stride % align != 0 ? -1 : stride;
    };
    const int64_t s[3] = {bytes(x.stride_page, counts[0]), bytes(x.stride_slot, counts[1]),
                          bytes(x.stride_head, heads)};
    if (s[0] < 0 || s[1] < 0 || s[2] < 0) return SPGEMM_ERR_INVALID_ARG;
    *base = static_cast<const char*>(x.data);
    if (cache->npages > 0 && (!*base || reinterpret_cast<uintptr_t>(*base) % align != 0))
        return SPGEMM_ERR_INVALID_ARG;
    if (!gather_unit(s, counts, 2, shift)) return SPGEMM_ERR_OVERFLOW;
    *page = (uint32_t)(s[0] >> *shift);
    *slot = (uint32_t)(s[1] >> *shift);
    *head = s[2];
    return SPGEMM_OK;
}

int mx_cache(const spgemm_mx_cache* c, const AttnShape& s, MxArgs* a) {
    a->format = c->format;
    const char *ks = nullptr, *vs = nullptr;
    int rc = mx_bytes(c->k_codes, c, s.hkv, 16, &a->k, &a->k_head, &a->k_page, &a->k_slot, &a->k_shift);
    if (rc == SPGEMM_OK)
        rc = mx_bytes(c->v_codes, c, s.hkv, 16, &a->v, &a->v_head, &a->v_page, &a->v_slot, &a->v_shift);
    if (rc == SPGEMM_OK)
        rc = mx_bytes(c->k_scales, c, s.hkv, 1, &ks, &a->ks_head, &a->ks_page, &a->ks_slot,
                      &a->ks_shift);
    if (rc == SPGEMM_OK)
        rc = mx_bytes(c->v_scales, c, s.hkv, 1, &vs, &a->vs_head, &a->vs_page, &a->vs_slot,
                      &a->vs_shift);
    a->ks = reinterpret_cast<const uint8_t*>(ks);
    a->vs = reinterpret_cast<const uint8_t*>(vs);
    return rc;
}

bool mx_format_valid(const spgemm_mx_cache* c) {
    return c && (c->format == SPGEMM_MX_E4M3 || c->format == SPGEMM_MX_E2M1) && c->reserved == 0;
}

// Whether no two places of a cache share a byte, in one of its tensors or in two.
bool cache_apart(const spgemm_mx_cache* c, int heads, int codes, int scales) {
    const auto places = [&](const spgemm_mx_bytes& x, int width) {
        return Places{(int64_t) reinterpret_cast<intptr_t>(x.data), width,
                      {x.stride_page, x.stride_slot, x.stride_head}, {c->npages, c->page_size, heads}};
    };
    const Places all[4] = {places(c->k_codes, codes), places(c->v_codes, codes),
                           places(c->k_scales, scales), places(c->v_scales, scales)};
    for (const Places& p : all)
        if (!places_apart(p)) return false;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (places_meet(all[i], all[j])) return false;
    return true;
}

// Writing and reading: everything but the direction.
template <class Run>
int mx_rows(const spgemm_attention_desc* desc, const spgemm_rows* k, const spgemm_rows* v,
            const spgemm_mx_cache* cache, const spgemm_paged_batch* batch, bool output, Run&& run) {
    if (!desc || !batch_sizes_valid(batch) || !mx_format_valid(cache)) return SPGEMM_ERR_INVALID_ARG;
    spgemm_attention_desc d = *desc;
    d.heads_q = d.heads_kv;
    d.scale = 0.;
    if (!mx_desc_valid(&d)) return SPGEMM_ERR_INVALID_ARG;
    if (!batch_sizes_fit(batch, &d)) return SPGEMM_ERR_OVERFLOW;
    return guarded([&]() -> int {
        MxRowsArgs a;
        batch_shape(batch, make_shape(&d), &a);
        if (!rows_valid(k, a.tokens, a.s.hkv, &d, output, &a.rk) ||
            !rows_valid(v, a.tokens, a.s.hkv, &d, output, &a.rv))
            return SPGEMM_ERR_INVALID_ARG;
        bool empty = false;
        int rc = paged_checks(batch, a.s, cache->npages, cache->page_size, &a, &empty);
        if (rc != SPGEMM_OK || empty) return rc;
        rc = mx_cache(cache, a.s, &a);
        if (rc != SPGEMM_OK) return rc;
        const int codes = cache->format == SPGEMM_MX_E4M3 ? a.s.dim : a.s.dim / 2;
        const int scales = a.s.dim / SPGEMM_MX_BLOCK;
        if (!output && cache->npages > 0 && !cache_apart(cache, a.s.hkv, codes, scales))
            return SPGEMM_ERR_INVALID_ARG;
        run(a);
        return SPGEMM_OK;
    });
}

// How keys are cut. Many rows: in pieces, as for a cache of 16-bit values. Few:
// evenly over the wavefronts that are there at once, whatever the texts' lengths
// (64 ragged texts of up to 16384 tokens, 8 bits: 291 us, in pieces of each text
// 437), where EvenSplit takes so many texts and each wavefront has few of them. A
// range may be one tile: one token over 1000 takes 15.7 us then, with two tiles at
// least 16.3, with four 19.0 (absorbed, 5 texts of up to 3000: 23.5, 27.2, 29.3).
void mx_pieces(PagedArgs* a) {
    const int64_t rows = (int64_t)a->max_new * a->s.group;
    const int64_t tile = mx_tile_rows(a->s, rows);
    const int64_t each = a->s.dim <= 128 ? 2 : 1;
    if (mx_wide(a->s, rows)) {
        const bool ragged = rows > tile && a->tokens * 4 < a->seqs * a->max_new * 3;
        cut_pieces(a, tile, each * (ragged ? 512 : 256), 256, 64);
    } else {
        const int64_t tiles = std::max<int64_t>(ceil_div(rows, tile), 1);
        const int64_t most = a->seqs * ceil_div(a->max_length, kMxKeys);
        if (a->seqs <= kMxEvenSeqs && a->seqs * a->s.hkv * tiles < each * 2048 &&
            most > a->seqs && most < INT32_MAX / 2) {
            a->piece = std::max(a->max_length, 1);
            a->ranges = (int32_t)std::max<int64_t>(std::min(most, each * 1024 / (a->s.hkv * tiles)), 1);
        } else {
            cut_pieces(a, tile, each * 1024, 64, 32);
        }
    }
}

// ---------------------------------------------------------------- latent
bool latent_desc_valid(const spgemm_latent_desc* d, bool absorbed) {
    if (!d || (d->type != SPGEMM_TYPE_BF16 && d->type != SPGEMM_TYPE_F16)) return false;
    if (d->heads < 1 || d->heads > SPGEMM_ATTENTION_MAX_HEADS) return false;
    if (d->latent_dim < 32 || d->latent_dim > SPGEMM_LATENT_MAX_DIM || d->latent_dim % 32 != 0)
        return false;
    if (d->rope_dim < 0 || d->rope_dim > SPGEMM_LATENT_MAX_ROPE || d->rope_dim % 8 != 0)
        return false;
    const auto head = [](int32_t n) {
        return n >= 16 && n <= SPGEMM_LATENT_MAX_HEAD && n % 16 == 0;
    };
    if (!absorbed && (!head(d->key_dim) || !head(d->value_dim))) return false;
    return std::isfinite(d->scale) && std::fabs(d->scale) < 1e30;
}

// A tensor's description as the shared checks take it.
spgemm_attention_desc rows_desc(const spgemm_latent_desc* d, int heads_q, int heads_kv, int dim) {
    return {d->type, heads_q, heads_kv, dim, d->scale};
}

// What a call is launched with, from sizes alone.
void latent_shape(const spgemm_latent_desc* d, const spgemm_paged_batch* b, bool absorbed,
                  LatentArgs* a) {
    const spgemm_attention_desc r =
        rows_desc(d, d->heads, absorbed ? 1 : d->heads, absorbed ? d->latent_dim : d->value_dim);
    batch_shape(b, make_shape(&r), a);
    a->key_dim = (absorbed ? d->latent_dim : d->key_dim) + d->rope_dim;
    a->made_dim = absorbed ? 0 : d->key_dim;
    a->rope_at = 2 * d->latent_dim;
    const int64_t tile = latent_tile_rows(*a, absorbed);
    if (absorbed) {
        // One work group per compute unit is there at once, and a text by itself is as
        // slow as it is long: all keys are cut evenly over them, by what a wavefront can look
        // over. (128 heads: 300 texts up to 512 tokens, one of 32 K, take 178 us, in a work
        // group a text 1563; 64 up to 1000, one of 32 K, 4 new tokens each, 212 and 1549; 300
        // up to 4096 374 and 397; 600 of 2048 each, which end together anyway, 640 and 563;
        // 1100 up to 512, one of 32 K, are not cut: 1710.) Where they are many, only if most
        // have as many new tokens as the longest chunk, whose tiles are everybody's: a range's
        // empty tiles leave compute units idle (300 of 2000, half with 4 new tokens and half
        // with one, 1087 us cut evenly, 825 not).
        const int64_t tiles = std::max<int64_t>(ceil_div((int64_t)a->max_new * a->s.group, tile), 1);
        const bool alike = 5 * a->tokens >= 4 * a->seqs * a->max_new;
        const bool even = a->seqs <= kAbsorbedEvenSeqs && (a->seqs * tiles < 512 || (tiles <= 64 && alike));
        const int64_t most = a->seqs * ceil_div(a->max_length, kAbsorbedKeys);
        a->piece = std::max(a->max_length, 1);
        if (even && most > a->seqs && most < INT32_MAX / 2)
            a->ranges = (int32_t)std::max<int64_t>(std::min(most, 256 / tiles), 1);
    } else {
        // one work group of 256 rows per compute unit or two of 128 are there at once, in
        // six rounds, since the texts differ; of 1024 keys at least, which suits many short
        // texts (20 of 700 with 300 new tokens each, 16 heads: 239 us, of 256 at least 339)
        // better than single ones (one of 1000 with 100: 78 and 52)
        cut_pieces(a, tile, (tile == 256 ? 6 : 12) * 256, 1024, 64);
    }
}

// Rows of made keys: one per place of the table, or per sequence and place,
// whichever are fewer.
void made_rows(const spgemm_paged_batch* b, int64_t page_size, LatentArgs* a) {
    const __int128 by_table = (__int128)b->pages->nnz * page_size;
    const __int128 by_length = (__int128)a->seqs * a->max_length;
    a->made_step = by_table <= by_length ? 0 : a->max_length;
    const __int128 rows = std::min(by_table, by_length);
    if (rows > ((__int128)1 << 40)) throw OverflowError("rows of made keys");
    a->made_rows = (int64_t)rows;
}

int64_t carve_made(void* ws, LatentArgs* a) {
    Carver c{static_cast<char*>(ws)};
    a->made_k = reinterpret_cast<char*>(c.take((__int128)a->made_rows * a->s.hq * a->made_dim));
    a->made_v = reinterpret_cast<char*>(c.take((__int128)a->made_rows * a->s.hq * a->s.dim));
    const int64_t used = c.used;
    return used + carve_parts(ws ? static_cast<char*>(ws) + used : nullptr, a);
}

int latent_cache(const spgemm_latent_cache* c, LatentArgs* a) {
    const int64_t counts[2] = {c->npages, c->page_size};
    const int64_t s[2] = {stride_bytes(c->stride_page, counts[0], 2),
                          stride_bytes(c->stride_slot, counts[1], 2)};
    if (s[0] < 0 || s[1] < 0) return SPGEMM_ERR_INVALID_ARG;
    a->k = static_cast<const char*>(c->data);
    if (c->npages > 0 && (!a->k || reinterpret_cast<uintptr_t>(a->k) % 16 != 0))
        return SPGEMM_ERR_INVALID_ARG;
    if (!gather_unit(s, counts, 2, &a->k_shift)) return SPGEMM_ERR_OVERFLOW;
    a->k_page = (uint32_t)(s[0] >> a->k_shift);
    a->k_slot = (uint32_t)(s[1] >> a->k_shift);
    return SPGEMM_OK;
}

// Both forms; w_k and w_v only of the expanded one.
int latent_call(const spgemm_latent_desc* desc, const spgemm_rows* q, const spgemm_rows* w_k,
                const spgemm_rows* w_v, const spgemm_latent_cache* cache,
                const spgemm_paged_batch* batch, const spgemm_rows* out, float* lse, bool absorbed,
                void* workspace, int64_t workspace_bytes, hipStream_t st) {
    if (!latent_desc_valid(desc, absorbed) || !batch_sizes_valid(batch) || !cache)
        return SPGEMM_ERR_INVALID_ARG;
    const int dim = absorbed ? desc->latent_dim : desc->key_dim;
    const spgemm_attention_desc dq = rows_desc(desc, desc->heads, 1, dim + desc->rope_dim);
    const spgemm_attention_desc dout =
        rows_desc(desc, desc->heads, 1, absorbed ? desc->latent_dim : desc->value_dim);
    if (!batch_sizes_fit(batch, &dq)) return SPGEMM_ERR_OVERFLOW;
    return guarded([&]() -> int {
        ExpandArgs e;
        LatentArgs& a = e.a;
        latent_shape(desc, batch, absorbed, &a);
        if (!rows_valid(q, a.tokens, a.s.hq, &dq, false, &a.q) ||
            !rows_valid(out, a.tokens, a.s.hq, &dout, true, &a.out))
            return SPGEMM_ERR_INVALID_ARG;
        if (!absorbed) {
            const spgemm_attention_desc dw = rows_desc(desc, 1, 1, desc->latent_dim);
            if (!rows_valid(w_k, a.s.hq, desc->key_dim, &dw, false, &e.wk) ||
                !rows_valid(w_v, a.s.hq, desc->value_dim, &dw, false, &e.wv))
                return SPGEMM_ERR_INVALID_ARG;
        }
        bool empty = false;
        int rc = paged_checks(batch, a.s, cache->npages, cache->page_size, &a, &empty);
        if (rc != SPGEMM_OK || empty) return rc;
        rc = latent_cache(cache, &a);
        if (rc != SPGEMM_OK) return rc;
        a.lse = lse;
        e.latent_dim = desc->latent_dim;
        if (!absorbed) made_rows(batch, cache->page_size, &a);
        const int64_t need = absorbed ? carve_parts(workspace, &a, latent_tile_rows(a, true))
                                      : carve_made(workspace, &a);
        if (!workspace_valid(workspace, workspace_bytes, need)) return SPGEMM_ERR_INVALID_ARG;
        if (!absorbed) latent_expand(e, st);
        latent_attention(a, absorbed, st);
        return SPGEMM_OK;
    });
}

}  // namespace

extern "C" {

SPGEMM_API int spgemm_mx_write(const spgemm_attention_desc* desc, const spgemm_rows* k,
                               const spgemm_rows* v, const spgemm_mx_cache* cache,
                               const spgemm_paged_batch* batch, void* stream) {
    return mx_rows(desc, k, v, cache, batch, false,
                   [&](const MxRowsArgs& a) { mx_write(a, (hipStream_t)stream); });
}

SPGEMM_API int spgemm_mx_read(const spgemm_attention_desc* desc, const spgemm_mx_cache* cache,
                              const spgemm_paged_batch* batch, const spgemm_rows* k,
                              const spgemm_rows* v, void* stream) {
    return mx_rows(desc, k, v, cache, batch, true,
                   [&](const MxRowsArgs& a) { mx_read(a, (hipStream_t)stream); });
}

SPGEMM_API int spgemm_mx_attention_workspace(const spgemm_attention_desc* desc,
                                             const spgemm_paged_batch* batch, int64_t* bytes) {
    if (!mx_desc_valid(desc) || !batch_sizes_valid(batch) || !bytes) return SPGEMM_ERR_INVALID_ARG;
    if (!batch_sizes_fit(batch, desc)) return SPGEMM_ERR_OVERFLOW;
    return guarded([&]() -> int {
        MxArgs a;
        batch_shape(batch, make_shape(desc), &a);
        mx_pieces(&a);
        *bytes = carve_parts(nullptr, &a, mx_tile_rows(a.s, (int64_t)a.max_new * a.s.group), a.s.hkv);
        return SPGEMM_OK;
    });
}

SPGEMM_API int spgemm_mx_attention(const spgemm_attention_desc* desc, const spgemm_rows* q,
                                   const spgemm_mx_cache* cache, const spgemm_paged_batch* batch,
                                   const spgemm_rows* out, float* lse, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    if (!mx_desc_valid(desc) || !batch_sizes_valid(batch) || !mx_format_valid(cache))
        return SPGEMM_ERR_INVALID_ARG;
    if (!batch_sizes_fit(batch, desc)) return SPGEMM_ERR_OVERFLOW;
    return guarded([&]() -> int {
        MxArgs a;
        batch_shape(batch, make_shape(desc), &a);
        mx_pieces(&a);
        if (!rows_valid(q, a.tokens, a.s.hq, desc, false, &a.q) ||
            !rows_valid(out, a.tokens, a.s.hq, desc, true, &a.out))
            return SPGEMM_ERR_INVALID_ARG;
        bool empty = false;
        int rc = paged_checks(batch, a.s, cache->npages, cache->page_size, &a, &empty);
        if (rc != SPGEMM_OK || empty) return rc;
        rc = mx_cache(cache, a.s, &a);
        if (rc != SPGEMM_OK) return rc;
        a.lse = lse;
        const int tile = mx_tile_rows(a.s, (int64_t)a.max_new * a.s.group);
        if (!workspace_valid(workspace, workspace_bytes, carve_parts(workspace, &a, tile, a.s.hkv)))
            return SPGEMM_ERR_INVALID_ARG;
        mx_attention(a, (hipStream_t)stream);
        return SPGEMM_OK;
    });
}

SPGEMM_API int spgemm_latent_attention_workspace(const spgemm_latent_desc* desc,
                                                 const spgemm_paged_batch* batch, int64_t* bytes) {
    if (!latent_desc_valid(desc, true) || !batch_sizes_valid(batch) || !bytes)
        return SPGEMM_ERR_INVALID_ARG;
    const spgemm_attention_desc r = rows_desc(desc, desc->heads, 1, desc->latent_dim);
    if (!batch_sizes_fit(batch, &r)) return SPGEMM_ERR_OVERFLOW;
    return guarded([&]() -> int {
        LatentArgs a;
        latent_shape(desc, batch, true, &a);
        *bytes = carve_parts(nullptr, &a, latent_tile_rows(a, true));
        return SPGEMM_OK;
    });
}

SPGEMM_API int spgemm_latent_attention(const spgemm_latent_desc* desc, const spgemm_rows* q,
                                       const spgemm_latent_cache* cache,
                                       const spgemm_paged_batch* batch, const spgemm_rows* out,
                                       float* lse, void* workspace, int64_t workspace_bytes,
                                       void* stream) {
    return latent_call(desc, q, nullptr, nullptr, cache, batch, out, lse, true, workspace,
                       workspace_bytes, (hipStream_t)stream);
}

SPGEMM_API int spgemm_latent_expanded_workspace(const spgemm_latent_desc* desc,
                                                const spgemm_latent_cache* cache,
                                                const spgemm_paged_batch* batch, int64_t* bytes) {
    if (!latent_desc_valid(desc, false) || !batch_sizes_valid(batch) || !cache || !bytes ||
        cache->page_size < 1 || batch->pages->nnz < 0)
        return SPGEMM_ERR_INVALID_ARG;
    const spgemm_attention_desc r = rows_desc(desc, desc->heads, 1, desc->value_dim);
    if (!batch_sizes_fit(batch, &r) || cache->page_size > kMaxTokens ||
        batch->pages->nnz > 0x7fffffffLL)
        return SPGEMM_ERR_OVERFLOW;
    return guarded([&]() -> int {
        LatentArgs a;
        latent_shape(desc, batch, false, &a);
        made_rows(batch, cache->page_size, &a);
        *bytes = carve_made(nullptr, &a);
        return SPGEMM_OK;
    });
}

SPGEMM_API int spgemm_latent_expanded(const spgemm_latent_desc* desc, const spgemm_rows* q,
                                      const spgemm_rows* w_k, const spgemm_rows* w_v,
                                      const spgemm_latent_cache* cache,
                                      const spgemm_paged_batch* batch, const spgemm_rows* out,
                                      float* lse, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
    return latent_call(desc, q, w_k, w_v, cache, batch, out, lse, false, workspace, workspace_bytes,
                       (hipStream_t)stream);
}

}  // extern "C"
