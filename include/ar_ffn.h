/*
 * ar_ffn.h -- C ABI of the operators of a decode step's feed-forward half
 * (same library as ar.h and ar_ops.h: libtda_ar.so).
 *
 * What ar_add_norm_fp8 writes (e4m3 rows with scales) goes through a product
 * with an e4m3 weight (ar_matmul_fp8), the gated activation (ar_silu_mul_fp8,
 * e4m3 again) and a second product, whose partial sums the all-reduce takes.
 * A layer with experts has the router before (ar_route_experts), the products
 * grouped by expert (ar_matmul_fp8 with offsets), and the weighted sum of each
 * token's rows after them (ar_experts_sum).
 *
 * Conventions as in ar_ops.h: device addresses on the current device, nothing
 * allocated, strides in elements, any stream, capturable; what the host can
 * see is refused (AR_EINVAL, AR_ETOOBIG) with nothing enqueued; what only the
 * device sees (offsets, row numbers, places) keeps the kernels inside the buffers.
 */
#ifndef TDA_AR_FFN_H
#define TDA_AR_FFN_H

#include "ar.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ar_matmul_fp8 -- product of e4m3 rows with e4m3 weights, a scale to each block of 128.
 * With x's row m and the weight's row n cut into groups g of 128 channels (the last may be short):
 *   out[m][n] = sum_g xs[m][g] * ws[n / 128][g] * sum_(k in g) x[m][k] * w[n][k]
 * Products are exact, sums binary32; the product of the two scales is rounded to binary32 and multiplies each group's sum, out is rounded once.
 * With x_row_scales, x has one scale a row (what ar_add_norm_fp8 gives with group 0); else one to 128
 * channels (its group 128).
 * offsets NULL: one weight for all rows; row m of out belongs to row m of x, and x_rows = rows.
 * offsets [experts + 1]: rows offsets[e] .. offsets[e + 1] - 1 of out take weight e.  They must not decrease.  Rows
 *   before offsets[0] and from offsets[experts] on are not written.
 * row_of [rows] (with or without offsets): row i of out belongs to row row_of[i] of x, any number of times each; a
 *   number outside x gives a row of zeros.  NULL: to row i.
 * Offsets outside 0 .. rows are taken as the nearest of these.  Where they decrease, the call stays inside the buffers, and what
 * it writes to out is undefined.
 * Results do not depend on the order in which blocks run; whether the groups are summed one after another or in
 * up to 16 parts, added in order, goes by the call's sizes.
 * Weights, x and out whose rows all begin on 16 bytes take the fast kernels (x_stride, weight_stride and expert_stride
 * multiples of 16 bytes; out is free), others a slower one.  Which of the fast ones goes by the sizes alone, the host cannot see the offsets: few
 * rows an expert on average take the one that reads an expert's weight for every 16 to 128 rows, which is slow where one expert has nearly all.
 * out must not overlap an input.
 * Logical ranks on one GPU: a product of many rows needs whole multiprocessors.  An exchange that is launched rank by rank
 * (ar_allreduce) and has a block on each of them, waiting for a rank whose product has not begun, keeps it from beginning
 * until the exchange's own limit; behind such products use the calls that launch all ranks at once (ar_allreduce_all).
 * Errors: AR_EINVAL, AR_ETOOBIG (rows or x_rows > 2^30, dim > 2^20, out_dim > 2^20, experts > 1024), AR_ECUDA.
 */
typedef struct ar_matmul_fp8_args {
    const void *x;              /* e4m3 [x_rows][dim] */
    const float *x_scales;      /* [x_rows][ceil(dim / 128)], or [x_rows][1] with x_row_scales */
    const void *weight;         /* e4m3 [experts][out_dim][dim] */
    const float *weight_scales; /* [experts][ceil(out_dim / 128)][ceil(dim / 128)], contiguous */
    void *out;                  /* [rows][out_dim] */
    const int32_t *offsets;     /* [experts + 1], or NULL */
    const int32_t *row_of;      /* [rows], or NULL */
    void *workspace;            /* ar_matmul_fp8_workspace() bytes, on 16 bytes, this call's alone until it has run; NULL: none */
    int64_t x_stride, x_scales_stride, weight_stride, expert_stride, out_stride;
    int64_t rows, x_rows;
    int32_t dtype;              /* AR_F16 or AR_BF16, of out */
    int32_t out_dim, dim;
    int32_t experts;            /* 1 without offsets */
    int32_t x_row_scales;       /* 0 or 1 */
} ar_matmul_fp8_args;
AR_API int ar_matmul_fp8(const ar_matmul_fp8_args *args, ar_stream_t stream);

/* Bytes of working memory with which a call that picks many rows (row_of) is faster: room for these rows and their scales, side by
 * side.  0: none is used. */
AR_API size_t ar_matmul_fp8_workspace(const ar_matmul_fp8_args *args);

/* The first error recorded by the products on the current device since the last call of this function: AR_ETIMEOUT
 * after a copy or a matrix instruction that did not end within its limit (the call ends, its outputs are
 * undefined), else AR_OK.  Synchronous: covers the calls that the caller has synchronised with. */
AR_API int ar_matmul_fp8_status(void);

/* A type of logits, beside ar_dtype's. */
#define AR_F32 4

/*
 * ar_route_experts -- the router's choice.  For every token the `chosen` experts with the largest logits, largest first, of
 * equal ones the one with the lower number; a logit that is NaN or -infinity is never chosen.  With m the
 * largest logit (+infinity counts as the largest binary32 number):
 *   weights[t][j] = exp(l_j - m) / sum exp(l - m), the sum over the chosen experts (normalize) or over all of them.
 * A token with fewer experts than that to choose from has expert -1, weight 0 and place -1 in what is left.
 * The (token, expert) pairs, ordered by expert and then token, are the rows of the experts' products:
 *   offsets [experts + 1]    where each expert's rows begin; offsets[experts] is their number
 *   rows    [tokens * chosen] the token of each row; -1 from offsets[experts] on
 *   place   [tokens][chosen]  the row of each pair
 * Errors: AR_EINVAL (chosen > experts too), AR_ETOOBIG (experts > 1024, chosen > 32, tokens * chosen > 2^30), AR_ECUDA.
 */
typedef struct ar_route_experts_args {
    const void *logits;     /* [tokens][experts] by logits_stride */
    float *weights;         /* [tokens][chosen] */
    int32_t *expert_ids;    /* [tokens][chosen] */
    int32_t *offsets;
    int32_t *rows;
    int32_t *place;
    int32_t *workspace;     /* ar_route_experts_workspace() bytes, this call's alone until it has run; NULL where that is 0 */
    int64_t logits_stride, tokens;
    int32_t dtype;          /* AR_F16, AR_BF16 or AR_F32 */
    int32_t experts, chosen;
    int32_t normalize;      /* 0 or 1 */
} ar_route_experts_args;
AR_API int ar_route_experts(const ar_route_experts_args *args, ar_stream_t stream);

/* Bytes of working memory that a call of these sizes (tokens, experts, chosen) needs; what is in it does not matter. */
AR_API size_t ar_route_experts_workspace(const ar_route_experts_args *args);

/*
 * ar_silu_mul_fp8 -- the gated activation, rounded to 8 bits.  Row r of x holds dim gates and dim factors after them:
 *   y_c = g_c / (1 + exp(-g_c)) * x[r][dim + c],   g_c = x[r][c]   (binary32)
 * per group of `group` channels (0: the row; the last group may be short): scale = max|y| / 448 (1 where that is 0, as binary32
 * makes it for max|y| up to 224 * 2^-149), out = e4m3(y / scale).  (A NaN is the largest: it is its group's scale, and out is NaN.)
 * y is off by less than 2^-19.9 of itself (exp and the quotient by the hardware's approximations), scale by 2^-19.7: where y / scale lies
 * that near to the middle of two e4m3 numbers, out may be either.  A row's output does not depend on where the row lies.
 * out [rows][dim] and scales [rows][ceil(dim / group)] are contiguous.
 * Errors: AR_EINVAL, AR_ETOOBIG (rows > 2^30, dim > 2^20), AR_ECUDA.
 */
typedef struct ar_silu_mul_fp8_args {
    const void *x;          /* [rows][2 * dim] by x_stride */
    void *out;              /* e4m3 bytes */
    float *scales;
    int64_t x_stride, rows;
    int32_t dtype;          /* AR_F16 or AR_BF16, of x */
    int32_t dim;
    int32_t group;          /* 0 .. dim */
} ar_silu_mul_fp8_args;
AR_API int ar_silu_mul_fp8(const ar_silu_mul_fp8_args *args, ar_stream_t stream);

/*
 * ar_experts_sum -- out[t] = sum_j weights[t][j] * x[place[t][j]], summed in binary32 in the order of j and rounded
 * once; a place outside x counts as nothing (whatever its weight).
 * out must not overlap x.
 * Errors: AR_EINVAL, AR_ETOOBIG (tokens or rows > 2^30, dim > 2^20, chosen > 1024), AR_ECUDA.
 */
typedef struct ar_experts_sum_args {
    const void *x;          /* [rows][dim] by x_stride */
    const float *weights;   /* [tokens][chosen] */
    const int32_t *place;   /* [tokens][chosen] */
    void *out;              /* [tokens][dim] by out_stride */
    int64_t x_stride, out_stride, rows, tokens;
    int32_t dtype;          /* AR_F16 or AR_BF16, of x and out */
    int32_t dim, chosen;
} ar_experts_sum_args;
AR_API int ar_experts_sum(const ar_experts_sum_args *args, ar_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* TDA_AR_FFN_H */
