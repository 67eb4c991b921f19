/*
 * ar_ops.h -- C ABI of the operators around the all-reduce of a decode step
 * (same library as ar.h: libtda_ar.so).
 *
 * One tensor-parallel rank's layer of a decode step is: say where the new
 * tokens go (ar_kv_plan, once a step), write their K and V rows to the cache
 * (ar_kv4_append), attend over the cache (ar_kv4_attend), project, all-reduce
 * the partial sums (ar_allreduce), and add the residual, normalise and round
 * to 8 bits for the next product (ar_add_norm_fp8).
 *
 * Conventions, beside ar.h's codes:
 *   - Every pointer is a device address on the current device, owned by the
 *     caller.  Nothing is allocated.  Strides count elements.
 *   - `stream` may be any stream of the current device, the default streams
 *     included: no kernel here waits for another launch.  Every call may be
 *     captured in a CUDA graph.
 *   - The host checks what it can see (sizes, NULL and misaligned pointers,
 *     types) and returns AR_EINVAL or AR_ETOOBIG with nothing enqueued; what
 *     only the device sees (lengths, page ids, slots) is checked in the kernels,
 *     which stay inside the buffers and say what was wrong as each call states.
 *
 * The 4-bit paged cache ("pool"): [pages][kv_heads][page / 16][18 * head_dim]
 * bytes, contiguous, 16-byte aligned.  The last axis is one tile: 16 consecutive
 * tokens of one head, K and V and their scales side by side, D = head_dim and
 * G = D / 32 groups:
 *   [0, 8D)     K nibbles  [token 16][t 4][group G][i 8], channel 32*group + 8*t + i
 *   [8D, 16D)   V nibbles  [half 2][g 8][t 4][group G][odd 2][i 4], token 8*half + 2*t + odd,
 *               channel 32*group + 4*g + i
 *   [16D, 17D)  K scales   bfloat16 [token 16][group G]
 *   [17D, 18D)  V scales   the same
 * Of a byte's two nibbles the low one comes first.  A nibble u stands for
 * (u - 8) * scale.  The order is that of the attention kernel's matrix
 * operands: a lane's K (V) operands of a tile are 2 runs of 4G bytes, and no
 * byte holds nibbles of two tokens.  A slot is page_id * page + token within the page.
 */
#ifndef TDA_AR_OPS_H
#define TDA_AR_OPS_H

#include "ar.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ar_kv_plan -- block tables and slot maps of a step, from the requests'
 * lengths.  Request b holds lens[b] tokens and gets new_tokens[b] more.  It keeps the
 * ceil(lens / page) pages it has and gets ceil((lens + new) / page) minus that
 * many from the free list, requests in order, pages in the list's order from
 * entry *free_used on.  The new tokens are numbered request by request:
 * request b's are cu[b] .. cu[b + 1] - 1.
 * Writes the new pages' ids to table[b][...], and
 *   lens_out [requests]       lens + new_tokens (may be lens itself)
 *   cu       [requests + 1]   running sum of new_tokens, from 0
 *   slots    [max_tokens]     of token i: its page id * page + its place in it; -1 from cu[requests] on
 *   request  [max_tokens]     of token i: b; -1 from cu[requests] on
 *   position [max_tokens]     of token i: its position in its request; -1 from cu[requests] on
 *   free_used_out [1]         *free_used + pages handed out (may be free_used itself)
 *   status   [1]              AR_OK, or why nothing was handed out:
 *     AR_EINVAL  a negative length, count or *free_used, a sum past 2^31 - 1, or a table entry
 *                in use (the last, partly filled page of a request that grows) that is negative
 *     AR_ETOOBIG a request needs more than table_width pages, or the new tokens exceed max_tokens
 *     AR_ENOMEM  the free list has too few entries left
 *   (the first of these that holds).  Then the table is unchanged, lens_out =
 *   lens, free_used_out = free_used, cu is all 0, and slots, request and position all -1.
 * Whole numbers only: the same inputs give the same outputs.
 * Errors: AR_EINVAL, AR_ETOOBIG (requests > 8192), AR_ECUDA.
 */
typedef struct ar_kv_plan_args {
    const int32_t *lens;
    const int32_t *new_tokens;
    int32_t *table;
    const int32_t *free_pages;
    const int32_t *free_used;
    int32_t *lens_out;
    int32_t *cu;
    int64_t *slots;
    int32_t *request;
    int32_t *position;
    int32_t *free_used_out;
    int32_t *status;
    int64_t table_stride;   /* elements from one request's row to the next, >= table_width */
    int64_t free_count;     /* entries of free_pages */
    int32_t requests;       /* 0 .. 8192 */
    int32_t table_width;
    int32_t page;           /* tokens of a page: a multiple of 16 */
    int32_t max_tokens;     /* entries of slots, request and position, >= 0 */
} ar_kv_plan_args;
AR_API int ar_kv_plan(const ar_kv_plan_args *args, ar_stream_t stream);

/*
 * ar_kv4_append -- round K and V rows to 4 bits and write them to their slots.
 * For every token, head and group of 32 channels, in binary32:
 *   scale = bfloat16(max|x| / 7), n = round-half-even(x / scale) kept within [-7, 7] (scale 0: n = 0).
 * A group that holds an infinity or a NaN gets a scale that is one, and reads
 * back as NaN.  A token whose slot is negative or past the pool is not written.
 * Two tokens of one call must not share a slot.
 * k, v: [tokens][kv_heads][head_dim] by their strides, channels contiguous.
 * Errors: AR_EINVAL, AR_ECUDA.
 */
typedef struct ar_kv4_rows_args {
    void *k;                /* append reads them, load writes them */
    void *v;
    void *pool;             /* append writes it, load reads it */
    const int64_t *slots;   /* [tokens] */
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    int64_t pages;          /* pages of the pool */
    int64_t tokens;
    int32_t dtype;          /* AR_F16 or AR_BF16 */
    int32_t kv_heads;
    int32_t head_dim;       /* 64, 128 or 256 */
    int32_t page;           /* a multiple of 16 */
} ar_kv4_rows_args;
AR_API int ar_kv4_append(const ar_kv4_rows_args *args, ar_stream_t stream);

/* ar_kv4_load -- the values of the given slots, n * scale rounded once to
 * dtype, into k and v (a slot that is negative or past the pool: zeros).
 * Errors: AR_EINVAL, AR_ECUDA. */
AR_API int ar_kv4_load(const ar_kv4_rows_args *args, ar_stream_t stream);

/*
 * ar_kv4_attend -- attention of the requests' newest tokens over the cache.
 * Request b's cache holds lens[b] tokens (its new ones among them, already
 * appended), token j in page table[b][j / page].  Its queries are rows
 * cu[b] .. cu[b + 1] - 1 of q, at its last positions; cu NULL: one query a
 * request.  Query head h reads kv head h / (q_heads / kv_heads).  The query at
 * position p sees token j if 0 <= j <= p and (window == 0 or j > p - window or
 * j < sinks).  With s_j = scale * q . k_j over those tokens:
 *   out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = ln sum_j exp(s_j);
 * a row that sees no token gets out = 0 and lse = -infinity.  Rows of no request (before cu[0], from cu[requests]
 * on: all of them after a plan that was refused) are not written, so that calls may share out and lse by requests.
 * Products take fp16 operands, sums and statistics are binary32, out is rounded once.  K and V enter as the whole
 * numbers they are.  bfloat16 q enters divided by the power of two that takes its row's largest value to [1, 2):
 * exact down to 2^-17 of that value, off by up to 2^-25 of it below.  Each exp(s_j) times its V scale is rounded
 * once: to 11 bits, or, where it is small, to 2^-33 of the largest V scale that the request's rows see (at least
 * 2^-80), so that groups of channels below 2^-22 of the largest have fewer.  Where V scales reach 2^k, k > 100, tokens
 * whose exp(s_j) is below 2^(k - 134) of the largest count as 0.
 * workspace: ar_kv4_workspace_bytes() bytes, 256-byte aligned, made ready once
 * by ar_kv4_workspace_init; calls that may overlap on the GPU need one each, and so do host threads that may
 * enqueue calls on one stream at the same time (a call is two launches, which must stay next to each other).
 * Its status (ar_kv4_status) says AR_EINVAL after a call that met a page id
 * outside the pool, a length past the table, or rows outside q in cu (the call
 * stays inside the buffers; outputs of such requests are undefined), and AR_ETIMEOUT
 * after a copy into shared memory that did not arrive (the call ends, its outputs are undefined).
 * Results do not depend on the order in which blocks run.
 * out must not overlap q (AR_EINVAL for the same address).
 * Errors: AR_EINVAL, AR_ETOOBIG (requests > 8192, tokens * query heads of a kv
 * head > 2^30, or a window > 2^30 shorter than the table), AR_ECUDA.
 */
typedef struct ar_kv4_attend_args {
    const void *q;          /* [tokens][q_heads][head_dim] by its strides, channels contiguous */
    void *out;              /* the same shape, by its own strides */
    float *lse;             /* [tokens][q_heads], contiguous; NULL: not written */
    const void *pool;
    const int32_t *table;   /* [requests][table_width] */
    const int32_t *lens;    /* [requests] */
    const int32_t *cu;      /* [requests + 1], or NULL */
    void *workspace;
    int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
    int64_t table_stride, pages;
    int32_t dtype;          /* AR_F16 or AR_BF16, of q and out */
    int32_t tokens;         /* rows of q (cu NULL: equal to requests) */
    int32_t requests;
    int32_t max_new;        /* most queries of a request: picks the kernel's shape, any number of them is right */
    int32_t q_heads, kv_heads;
    int32_t head_dim;       /* 64, 128 or 256 */
    int32_t page, table_width;
    int32_t window, sinks;  /* window 0: all tokens; sinks count only with a window */
    float scale;            /* finite */
} ar_kv4_attend_args;
AR_API int ar_kv4_attend(const ar_kv4_attend_args *args, ar_stream_t stream);

/* Bytes of an attention workspace on any GB300, whatever the call's sizes. */
AR_API size_t ar_kv4_workspace_bytes(void);
/* Zero a workspace's status and counters on `stream`.  Errors: AR_EINVAL, AR_ECUDA. */
AR_API int ar_kv4_workspace_init(void *workspace, ar_stream_t stream);
/* The first error recorded in a workspace since it was made ready (a
 * synchronous copy: covers the calls the caller has synchronised with). */
AR_API int ar_kv4_status(const void *workspace);

/*
 * ar_add_norm_fp8 -- residual, RMS norm and rounding to 8 bits in one pass.
 * Per row: h = x + residual (binary32; residual NULL: h = x), y = h / sqrt(mean(h^2) +
 * eps) * weight; per group of `group` channels (0: the row; the last group may
 * be short): scale = max|y| / 448 (1 where that is 0, as binary32 makes it for max|y| up to 224 * 2^-149),
 * out = e4m3(y / scale).
 * (A NaN is the largest: it is its group's scale, and out is NaN.)
 * A row whose sum of squares passes binary32 has y = 0 but where h is not finite; there y is NaN, and so are its
 * group's scale and out.
 * residual_out (may be residual or x themselves, by their strides; no other overlap): h rounded to dtype;
 * NULL: not written.
 * out [rows][dim] and scales [rows][ceil(dim / group)] are contiguous; the others go by their row strides.
 * Errors: AR_EINVAL, AR_ETOOBIG (dim > 32768), AR_ECUDA.
 */
typedef struct ar_add_norm_fp8_args {
    const void *x;
    const void *residual;
    const void *weight;     /* [dim] */
    void *out;              /* e4m3 bytes */
    float *scales;
    void *residual_out;
    int64_t x_stride, residual_stride, residual_out_stride;
    int64_t rows;
    int32_t dtype;          /* AR_F16 or AR_BF16, of x, residual, weight and residual_out */
    int32_t dim;
    int32_t group;          /* 0 .. dim */
    float eps;              /* >= 0 */
} ar_add_norm_fp8_args;
AR_API int ar_add_norm_fp8(const ar_add_norm_fp8_args *args, ar_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* TDA_AR_OPS_H */
