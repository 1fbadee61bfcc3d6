/*
 * spgemm_cache.h -- C ABI of key/value caches that take less memory than
 * those of spgemm_attention.h, and of the attention that reads them, on the
 * MI355X (gfx950): paged caches in 8 or 4 bits a value, and paged caches of
 * one latent vector a token that all heads share.
 *
 * Conventions are those of spgemm_attention.h: its descriptions, batches,
 * page tables, alignment, checks of a batch on the device, infinities and
 * NaN, workspaces, graphs and statuses hold here too.
 */
#ifndef SPGEMM_CACHE_H
#define SPGEMM_CACHE_H

#include "spgemm_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Quantised caches. The head_dim values of one token and head are cut into
 * blocks of 32. A block holds a power of two and a floating code per value:
 *
 *   value = code * 2^(scale - 127)      scale: a byte; 255 stands for NaN
 *
 * with codes of 8 bits (sign, 4 of exponent with bias 7, 3 of fraction: to 448,
 * 0x7f and 0xff are NaN) or of 4 (sign, 2 of exponent with bias 1, 1 of
 * fraction: 0, 0.5, 1, 1.5, 2, 3, 4, 6; two to a byte, the first in its low
 * half). All values are exact in bfloat16 and float, up to those past their
 * ranges. What is written is, for a block with largest magnitude a,
 *
 *   e = the smallest integer with a <= M * 2^e, M = 448 or 6, but at least -117
 *   code_i = x_i / 2^e, rounded to the nearest code, of two to the even one
 *
 * so that nothing saturates and every value is rounded once; a block that
 * holds an infinity or a NaN becomes NaN whole. Scales of any byte are read.
 * ------------------------------------------------------------------------ */
#define SPGEMM_MX_BLOCK 32

typedef enum {
    SPGEMM_MX_E4M3 = 0, /* 8 bits a value */
    SPGEMM_MX_E2M1 = 1  /* 4 bits a value */
} spgemm_mx_format;

/* Bytes of every slot and head: byte b of head h in slot s of page p is at
 * data[p * stride_page + s * stride_slot + h * stride_head + b]. */
typedef struct {
    void* data;
    int64_t stride_page;
    int64_t stride_slot;
    int64_t stride_head;
} spgemm_mx_bytes;

/* A quantised paged cache: head_dim bytes of codes (half as many in 4 bits)
 * and head_dim / 32 scales for the key and for the value of every slot and
 * head. head_dim is a multiple of 32. Codes' data and strides are multiples of
 * 16 bytes; scales have any. A cache whose places overlap (a stride that does
 * not pass what smaller ones reach, or a byte that two of the four tensors have)
 * is read, and refused where it is written. Tensors may lie between each other's
 * places, as parts of one allocation do; where their strides are so unlike that
 * telling them apart takes thousands of steps, they count as overlapping. */
typedef struct {
    int32_t format;    /* spgemm_mx_format                                     */
    int32_t reserved;  /* 0                                                    */
    int64_t npages;
    int64_t page_size; /* slots per page, at least 1; any number               */
    spgemm_mx_bytes k_codes, k_scales, v_codes, v_scales;
} spgemm_mx_cache;

/* Quantise the batch's new tokens into the cache: row q_rowptr[s] + t of k and
 * v (heads_kv heads, batch->tokens rows, any of the three types) goes to place
 * length - n + t of sequence s, n its new tokens. Other places keep what they
 * hold. Nothing of a sequence that breaks the batch's rules is written, nor a
 * token whose page is outside the cache. (Two rows for one place: which of
 * them it holds afterwards, code by code, is not said.) heads_q and scale of
 * `desc` are not read. Asynchronous on `stream`, without workspace. Errors:
 * INVALID_ARG, OVERFLOW (as spgemm_paged_attention), HIP. */
SPGEMM_API int spgemm_mx_write(const spgemm_attention_desc* desc, const spgemm_rows* k,
                               const spgemm_rows* v, const spgemm_mx_cache* cache,
                               const spgemm_paged_batch* batch, void* stream);

/* The reverse: row q_rowptr[s] + t of k and v becomes the value of place
 * length - n + t of sequence s, rounded to the type (a whole text is read by n
 * = length). Rows of sequences that break the rules, and of tokens whose page
 * is outside the cache, become NaN as those of spgemm_paged_attention do; rows
 * of no sequence stay as they were. Errors: as spgemm_mx_write. */
SPGEMM_API int spgemm_mx_read(const spgemm_attention_desc* desc, const spgemm_mx_cache* cache,
                              const spgemm_paged_batch* batch, const spgemm_rows* k,
                              const spgemm_rows* v, void* stream);

/* spgemm_paged_attention over a quantised cache: the formula with the cache's
 * values for k and v. They enter the products as they are; queries do too (in
 * two or three bfloat16 parts where they are half or float), and the
 * probabilities with 8 (bfloat16), 16 (half) or 24 (float) significant bits.
 * (A value past bfloat16's range enters as what the conversion makes of it, an
 * infinity or NaN.)
 * Errors and broken batches: as there. */
SPGEMM_API int spgemm_mx_attention_workspace(const spgemm_attention_desc* desc,
                                             const spgemm_paged_batch* batch, int64_t* bytes);
SPGEMM_API int spgemm_mx_attention(const spgemm_attention_desc* desc, const spgemm_rows* q,
                                   const spgemm_mx_cache* cache, const spgemm_paged_batch* batch,
                                   const spgemm_rows* out, float* lse, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Latent caches. A token holds one vector c_j of latent_dim values and one
 * r_j of rope_dim values (keys' part that depends on the position), next to
 * each other, for all heads together.
 * ------------------------------------------------------------------------ */
#define SPGEMM_LATENT_MAX_DIM 512
#define SPGEMM_LATENT_MAX_ROPE 64
#define SPGEMM_LATENT_MAX_HEAD 128

typedef struct {
    int32_t type;        /* bfloat16 or half                                   */
    int32_t heads;       /* at most 65536                                      */
    int32_t latent_dim;  /* 32 to 512, a multiple of 32                        */
    int32_t rope_dim;    /* 0 to 64, a multiple of 8                           */
    int32_t key_dim;     /* the expanded form's values of a head's key beside the
                            rope_dim ones and of its value: 16 to 128, multiples
                            of 16; the absorbed form does not read them        */
    int32_t value_dim;
    double scale;        /* factor of the scores; magnitude below 1e30         */
} spgemm_latent_desc;

/* Value x of c (x < latent_dim) or r (x - latent_dim) in slot s of page p is at
 * data[p * stride_page + s * stride_slot + x]; rows are 16-byte aligned. */
typedef struct {
    const void* data;
    int64_t npages;
    int64_t page_size;
    int64_t stride_page;
    int64_t stride_slot;
} spgemm_latent_cache;

/* Absorbed form: queries in the latents' space. For the batch's new tokens
 * (rows and what they see as in spgemm_paged_attention) and every head,
 *
 *   s_j = scale * (q . [c_j, r_j])    o = sum_j softmax(s)_j c_j
 *
 * with q [tokens, heads, latent_dim + rope_dim] and out [tokens, heads,
 * latent_dim]; lse (may be NULL) as there. Probabilities are rounded to the
 * type before the second product, the result once. (Both forms. An infinite
 * value whose probability that rounds to 0 gives NaN or itself. Sums are held
 * times up to 2^8 before the result's division: bfloat16 values past 2^119 may
 * overflow them.) Errors and broken batches: as spgemm_paged_attention. */
SPGEMM_API int spgemm_latent_attention_workspace(const spgemm_latent_desc* desc,
                                                 const spgemm_paged_batch* batch, int64_t* bytes);
SPGEMM_API int spgemm_latent_attention(const spgemm_latent_desc* desc, const spgemm_rows* q,
                                       const spgemm_latent_cache* cache,
                                       const spgemm_paged_batch* batch, const spgemm_rows* out,
                                       float* lse, void* workspace, int64_t workspace_bytes,
                                       void* stream);

/* Expanded form: every head's keys and values are made from the latents,
 *
 *   k_hj = [W_k,h c_j, r_j]   v_hj = W_v,h c_j
 *   s_j = scale * (q_h . k_hj)    o_h = sum_j softmax(s)_j v_hj
 *
 * with w_k [heads, key_dim, latent_dim] and w_v [heads, value_dim, latent_dim]
 * given as spgemm_rows (row: the head, head: the key's or value's index), q
 * [tokens, heads, key_dim + rope_dim] and out [tokens, heads, value_dim]. The
 * products with the weights are kept in the workspace for every cached token of
 * the batch, as two numbers of the type each (the rounded product, and what
 * that leaves, rounded): that is for chunks of many new tokens; a few are the
 * absorbed form's, with W_k and W_v multiplied into q and out. A product past
 * the type's range is infinite. The workspace grows with the smaller of the page
 * table's room * page_size and sequences * max_length, times the call's heads (4
 * bytes a value: 17 GB for 128 heads of 128 + 128 over 128 K tokens); a caller
 * bounds it by calls for groups of heads, whose q, w_k, w_v and out are slices of
 * the whole ones. Errors and broken batches:
 * as spgemm_paged_attention; the workspace call needs the cache's page size. */
SPGEMM_API int spgemm_latent_expanded_workspace(const spgemm_latent_desc* desc,
                                                const spgemm_latent_cache* cache,
                                                const spgemm_paged_batch* batch, int64_t* bytes);
SPGEMM_API int spgemm_latent_expanded(const spgemm_latent_desc* desc, const spgemm_rows* q,
                                      const spgemm_rows* w_k, const spgemm_rows* w_v,
                                      const spgemm_latent_cache* cache,
                                      const spgemm_paged_batch* batch, const spgemm_rows* out,
                                      float* lse, void* workspace, int64_t workspace_bytes,
                                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPGEMM_CACHE_H */
