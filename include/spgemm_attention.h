/*
 * spgemm_attention.h -- C ABI of softmax attention over sparse structure on
 * the MI355X (gfx950): attention whose mask is the structure of a CSR matrix,
 * its gradients, and attention of new tokens over a paged key/value cache.
 *
 * With query rows q_i, key rows k_j and value rows v_j of one head, and M_i
 * the columns that row i of the mask stores,
 *
 *   s_ij  = scale * (q_i . k_j)                      for j in M_i
 *   lse_i = log(sum_{j in M_i} exp(s_ij))
 *   p_ij  = exp(s_ij - lse_i)
 *   o_i   = sum_{j in M_i} p_ij v_j
 *
 * that is: a product of two dense matrices sampled at the mask's entries, a
 * softmax along the sparse rows, and the product of the resulting sparse
 * matrix with a dense one. All heads share the mask. heads_q is a multiple
 * of heads_kv; query head h reads key head h / (heads_q / heads_kv).
 *
 * Conventions, beside those of spgemm.h (device pointers on the current HIP
 * device, hipStream_t as void*, statuses, no C++ exception)
 *   - A tensor of rows is given as spgemm_rows: element (t, h, x) is at
 *     data[t * stride_row + h * stride_head + x]. Strides count elements, are
 *     not negative, and together with `data` keep every row 16-byte aligned;
 *     head_dim * (bytes of the type) is a multiple of 16 too. Rows of an
 *     output tensor must not overlap. Anything else is INVALID_ARG. (That an
 *     output shares no memory with another tensor of the call is the caller's
 *     to see to.)
 *   - Types: bfloat16, IEEE half or float for every tensor of a call alike;
 *     log-sum-exps are always float, [rows, heads_q] without gaps. Scores,
 *     softmax statistics and all sums are held in 32 bits. The probabilities
 *     (and their gradients in the backward pass) are rounded to the tensors'
 *     type before they enter the second product, results once at the end.
 *   - Calls with the same arguments give the same bits: no sum depends on
 *     the order in which work groups run.
 *   - An infinity or a NaN reaches the results whose formula has it, and no
 *     others: not those of a row that does not store the key that holds it,
 *     nor of a token that may not see it.
 *   - Attention calls neither allocate nor wait: they are asynchronous on
 *     `stream`, take their workspace from the caller, and may be captured
 *     into a HIP graph. A workspace belongs to one call at a time; two
 *     graphs that may run at once need one each.
 */
#ifndef SPGEMM_ATTENTION_H
#define SPGEMM_ATTENTION_H

#include "spgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SPGEMM_TYPE_BF16 = 0,
    SPGEMM_TYPE_F16 = 1,
    SPGEMM_TYPE_F32 = 2
} spgemm_type;

#define SPGEMM_ATTENTION_MAX_HEAD_DIM 256
#define SPGEMM_ATTENTION_MAX_HEADS 65536

/* What the tensors of one call have in common. */
typedef struct {
    int32_t type;      /* spgemm_type                                          */
    int32_t heads_q;   /* a multiple of heads_kv, at most 65536                */
    int32_t heads_kv;
    int32_t head_dim;  /* 1 to 256, a multiple of 8 (of 4 for floats)          */
    double scale;      /* factor of the scores; magnitude below 1e30           */
} spgemm_attention_desc;

/* A [rows, heads, head_dim] tensor (see above). */
typedef struct {
    void* data;
    int64_t stride_row;
    int64_t stride_head;
} spgemm_rows;

typedef struct spgemm_attention_plan_s* spgemm_attention_plan;

/* Create a plan for one mask: checks it, copies its columns, cuts its long
 * rows into pieces of similar work and, if `backward` is not 0, does the same
 * for its transpose. mask->val is not read and may be NULL. Columns need not
 * be sorted (but only rows whose columns ascend can share work with their
 * neighbours); a column that a row stores twice counts as two keys. The mask's
 * arrays are not used after the call, which blocks until the plan is ready.
 * A plan never changes afterwards: any number of calls, on any streams, may
 * use it at once, and it must outlive them and the graphs that captured
 * them. Errors: INVALID_ARG, INDEX_RANGE (row pointers or columns),
 * OVERFLOW (2^31 - 1 or more rows, columns over INT32_MAX, 2^31 or more
 * entries), OUT_OF_MEMORY, HIP. */
SPGEMM_API int spgemm_attention_plan_create(spgemm_attention_plan* out, const spgemm_csr* mask,
                                            int32_t backward, void* stream);

/* Wait for the device and free the plan. NULL is a no-op. */
SPGEMM_API void spgemm_attention_plan_destroy(spgemm_attention_plan plan);

/* Bytes of workspace (256-byte aligned device memory) that
 * spgemm_attention_forward, or with `backward` not 0
 * spgemm_attention_backward, needs; 0 is possible. Errors: INVALID_ARG,
 * NOT_READY (backward of a plan without it). */
SPGEMM_API int spgemm_attention_workspace(spgemm_attention_plan plan,
                                          const spgemm_attention_desc* desc, int32_t backward,
                                          int64_t* bytes);

/* o and lse of every row of the mask, from q (mask rows) and k, v (mask
 * columns). A row without entries, or all of whose scores are -infinity,
 * gets o = 0 and lse = -infinity. Rows of k and v that no entry names are
 * not read. `lse` may be NULL. Errors: INVALID_ARG (also a workspace that is
 * too small, or a plan of another device), OVERFLOW (k or v spans so many
 * bytes that a row's offset in units of the strides' common power of two
 * does not fit 32 bits; at 16 bytes that is 64 GiB), HIP. */
SPGEMM_API int spgemm_attention_forward(spgemm_attention_plan plan,
                                        const spgemm_attention_desc* desc, const spgemm_rows* q,
                                        const spgemm_rows* k, const spgemm_rows* v,
                                        const spgemm_rows* out, float* lse, void* workspace,
                                        int64_t workspace_bytes, void* stream);

/* Gradients of a scalar with respect to q, k and v, given its gradient dout
 * with respect to o, and o and lse as the forward call left them. The
 * probabilities are recomputed from q, k and lse (a float: of scores past 10^4
 * its rounding, 2^-24 of it, is the larger part of a probability's relative
 * error; none is taken as more than 1):
 *
 *   delta_i = dout_i . o_i          ds_ij = p_ij (dout_i . v_j - delta_i)
 *   dq_i = scale * sum_{j in M_i} ds_ij k_j
 *   dk_j = scale * sum_{i: j in M_i} ds_ij q_i      dv_j = sum p_ij dout_i
 *
 * with dk and dv summed over the query heads of each key head too. Gradients
 * are written, not added to; rows without entries get 0. `lse` is needed.
 * Errors: as spgemm_attention_forward, and NOT_READY (the plan was created
 * without `backward`). OVERFLOW counts q and dout as well. */
SPGEMM_API int spgemm_attention_backward(spgemm_attention_plan plan,
                                         const spgemm_attention_desc* desc, const spgemm_rows* q,
                                         const spgemm_rows* k, const spgemm_rows* v,
                                         const spgemm_rows* out, const float* lse,
                                         const spgemm_rows* dout, const spgemm_rows* dq,
                                         const spgemm_rows* dk, const spgemm_rows* dv,
                                         void* workspace, int64_t workspace_bytes, void* stream);

/* A paged cache: token x of head h in slot s of page p is at
 * k[p * k_stride_page + s * k_stride_slot + h * k_stride_head + x], and
 * likewise for v. Alignment and strides as for spgemm_rows. */
typedef struct {
    const void* k;
    const void* v;
    int64_t npages;
    int64_t page_size;  /* slots per page, at least 1; any number             */
    int64_t k_stride_page, k_stride_slot, k_stride_head;
    int64_t v_stride_page, v_stride_slot, v_stride_head;
} spgemm_paged_cache;

/* A batch of sequences, each with new tokens at the end of its cached ones.
 * All arrays are device arrays and are read when the kernels run, so that a
 * captured call follows their later values. */
typedef struct {
    /* Row s lists sequence s's pages in order: nrows = sequences, ncols =
     * cache pages; nnz is the room of `col`, which may be larger than
     * rowptr[nrows]. val is not read. */
    const spgemm_csr* pages;
    const int64_t* q_rowptr;  /* sequences + 1: sequence s's new tokens are the
                                 rows [q_rowptr[s], q_rowptr[s + 1]) of q     */
    const int64_t* lengths;   /* cached tokens of each sequence, its new ones
                                 (written to the cache before) among them     */
    int64_t tokens;           /* rows of q and out                            */
    int64_t max_new;          /* bounds on the new tokens and the length of   */
    int64_t max_length;       /* any sequence, for the launch's shape         */
} spgemm_paged_batch;

/* Workspace of spgemm_paged_attention for these sizes (pointers in `batch`
 * are not read; only its sizes and pages->nrows are). Errors: INVALID_ARG,
 * OVERFLOW. */
SPGEMM_API int spgemm_paged_attention_workspace(const spgemm_attention_desc* desc,
                                                const spgemm_paged_batch* batch, int64_t* bytes);

/* o and lse of new tokens over their sequence's cache. The t-th of n new
 * tokens of a sequence of length L sees the cached tokens 0 to L - n + t; what
 * the cache holds in any other place (later tokens, the rest of the last
 * page, other pages) does not reach its result, NaN and infinities included.
 * Rows of out and lse outside [q_rowptr[0], q_rowptr[nrows]) stay as they
 * were. The batch is checked where it is read: a sequence whose length is
 * below its number of new tokens, above max_length or above its pages' room,
 * that has more than max_new new tokens, or that needs a page outside [0,
 * npages), gets NaN in those of its first max_new rows that exist (a page
 * that only some of its tokens need: in those tokens' rows at least); no
 * memory outside the arrays is touched. A sequence is judged by its own
 * entries alone: another's broken row pointer or start costs it nothing, but
 * what a row holds that two sequences name is not said. `lse` may be NULL. Errors:
 * INVALID_ARG, OVERFLOW (as spgemm_attention_forward; tokens, max_length or
 * the page size over 2^30, 2^30 or more sequences, more than 2^31 - 128 pairs
 * of token and query head, 2^31 or more pages or entries of their table), HIP. */
SPGEMM_API int spgemm_paged_attention(const spgemm_attention_desc* desc, const spgemm_rows* q,
                                      const spgemm_paged_cache* cache,
                                      const spgemm_paged_batch* batch, const spgemm_rows* out,
                                      float* lse, void* workspace, int64_t workspace_bytes,
                                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPGEMM_ATTENTION_H */
