/*
 * cb_serve.h -- operators around the MoE layer of a GB300 serving program:
 * the norm in front of it, routing from given logits, and products of a few
 * rows with 4-bit weights quantised in groups.
 *
 * Conventions are those of cb_fp4.h: device pointers, work enqueued on
 * `stream` of the current device, arguments checked before anything is
 * enqueued, no allocation and no synchronisation, no state: the calls can be
 * captured into a graph and are safe from several threads and on several
 * streams.  An empty call (no rows or tokens) returns CB_OK and takes NULL
 * pointers.
 */
#ifndef CB_SERVE_H
#define CB_SERVE_H

#include "cb_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Root-mean-square norm with the residual's addition:
 *   h = x + residual            (fp32; h = x without one)
 *   sum = h                     (rounded to x's type, if asked for)
 *   y = h / sqrt(mean_i h_i^2 + eps) * weight
 *   out = y                     (rounded once, if asked for)
 *   codes, scales               (if asked for): per row and 128 columns (the
 *     last ones of a row may be fewer) a scale s = max|y| / 448 and the e4m3
 *     code nearest the quotient y / s (y, s and the quotient in fp32), ties to
 *     the even one.  Y = s v(code).  A group of zeros has the scale 0 and zero
 *     codes; one that holds a NaN or an infinity a NaN scale and zero codes.
 * The norm is taken of the unrounded h; the sum of squares is fp32 (|h| up to
 * about 1e18; what is below 1e-18 may vanish beside eps = 0).  In place: sum may be x or residual itself and out may be x
 * itself (the same pointer, stride and type); otherwise nothing that is
 * written may overlap what is read or written beside it.
 */
#define CB_NORM_MAX_COLS 32768
#define CB_FP8_COLS 128 /* columns of a scale */
typedef struct {
  int64_t rows, cols;     /* cols: 1..CB_NORM_MAX_COLS                           */
  const void *x;          /* [rows][cols], row stride ld_x elements              */
  int64_t ld_x;
  const void *residual;   /* the same, or NULL                                   */
  int64_t ld_residual;
  const void *weight;     /* [cols]                                              */
  void *sum;              /* [rows][cols], or NULL                               */
  int64_t ld_sum;
  void *out;              /* [rows][cols], or NULL                               */
  int64_t ld_out;
  uint8_t *codes;         /* e4m3 [rows][cols], contiguous, or NULL              */
  float *scales;          /* [rows][ceil(cols / 128)], NULL where codes is       */
  float eps;              /* >= 0                                                */
  int32_t x_type;         /* cb_dtype_t of x, residual and sum                   */
  int32_t weight_type;    /* cb_dtype_t                                          */
  int32_t out_type;       /* cb_dtype_t                                          */
} cb_rms_norm_t;

/* Errors: CB_ERR_INVALID_ARG (NULL, negative rows, no columns, a row stride
 * below cols, an unknown type, eps negative or not finite, nothing to be
 * written, codes without scales, overlaps), CB_ERR_ALIGNMENT (a pointer not on
 * its element's size), CB_ERR_UNSUPPORTED (more columns, 2^31 rows, a wrong
 * GPU), CB_ERR_CUDA.  Rows that do not start on 16 bytes take smaller loads. */
CB_API cb_status_t cb_rms_norm(const cb_rms_norm_t *args, void *stream);

/*
 * Routing from logits l [n_tokens][E] (with the router's own bias in them):
 *   score   s_e = 1 / (1 + exp(-l_e))            CB_SCORE_SIGMOID
 *           s_e = exp(l_e) / sum_j exp(l_j)      CB_SCORE_SOFTMAX
 *   choice  c_e = s_e + bias_e (c_e = s_e without one), for balance
 *   groups  with n_groups > 1 (E / n_groups consecutive experts each): a
 *           group's value is the sum of its two largest c (CB_GROUP_TOP2) or
 *           its largest (CB_GROUP_MAX); the top_groups groups of the largest
 *           values are kept, ties to the lower group
 *   ids     the top_k experts of the largest c among those kept, c descending,
 *           ties to the lower index
 *   w       s_ids[0..k), divided by their sum with renormalise, times scale
 * The order is that of the real numbers: where 32 bits leave two choices too
 * near to tell they are made again in 64, so equal logits with equal biases
 * are ties, and hardly anything else is.  The weights are those of s, not c.
 *
 * An expert of logit -inf is out: it follows every other in the order, has
 * the score 0, and its group's value is taken of the others (groups without
 * any come last).  A NaN logit (or c) follows even those and has a NaN score;
 * it is not in the softmax's sum.  They are chosen only where nothing else is
 * left, by index; where the chosen weights' sum is 0 (all of them out) the
 * weights are 0.  +inf counts as the largest finite number.
 */
typedef enum { CB_SCORE_SIGMOID = 0, CB_SCORE_SOFTMAX = 1 } cb_score_t;
typedef enum { CB_GROUP_TOP2 = 0, CB_GROUP_MAX = 1 } cb_group_score_t;
#define CB_ROUTE_MAX_GROUPS 32
typedef struct {
  int64_t n_tokens;
  const void *logits;     /* [n_tokens][n_experts], row stride ld_logits         */
  int64_t ld_logits;
  const float *bias;      /* [n_experts], or NULL                                */
  int32_t *ids;           /* [n_tokens][top_k]                                   */
  float *w;               /* [n_tokens][top_k]                                   */
  float scale;
  int32_t logits_type;    /* cb_dtype_t                                          */
  int32_t n_experts;      /* 1..256                                              */
  int32_t top_k;          /* 1..min(16, experts of the kept groups)              */
  int32_t score;          /* cb_score_t                                          */
  int32_t n_groups;       /* a divisor of n_experts, 1..CB_ROUTE_MAX_GROUPS       */
  int32_t top_groups;     /* 1..n_groups                                         */
  int32_t group_score;    /* cb_group_score_t; with groups of one expert both are its c */
  int32_t renormalise;    /* 0 or 1                                              */
} cb_route_t;

/* Errors: CB_ERR_INVALID_ARG (NULL, negative or impossible sizes, an unknown
 * type or score, ld_logits < n_experts, a scale that is not finite, outputs
 * overlapping anything), CB_ERR_ALIGNMENT, CB_ERR_UNSUPPORTED (more than 256
 * experts, 16 of them or 32 groups, 2^31 tokens, a wrong GPU), CB_ERR_CUDA. */
CB_API cb_status_t cb_route(const cb_route_t *args, void *stream);

/*
 * A few rows by 4-bit integer weights with a scale and a zero point per group
 * of `group` elements of a row:
 *   W[j][i] = scales[i / group][j] (code[j][i] - zeros[i / group][j]),
 *   y[r][j] = sum_i x[r][i] W[j][i],
 * x in bf16, or e4m3 codes with a scale per row and 128 columns (cb_rms_norm's).
 * The integers code - zero are exact operands and every group's sum meets its
 * scale in fp32: nothing is rounded before the result.  An infinite element of x
 * makes its row of out NaN, whatever its weights: it meets the zero points too.
 * (Elements of bf16 x from 2^64 on may count as infinite, and what is below
 * 2^-57 may be lost.  Scales of W are below 2^58 in magnitude.)
 *
 * One matrix (n_experts = 1, ids NULL): out [n_tokens][n].  With ids
 * [n_tokens][top_k] (device, in [0, n_experts)) one matrix per expert, and
 * pair p = t top_k + s is x's row t (row p with x_per_slot) by the matrix of
 * ids[t][s]: out [n_tokens top_k][n], or with weights w [n_tokens][top_k] the sum
 * over s of w[t][s] times its rows: out [n_tokens][n].  An expert may come more
 * than once in a row.  A pair whose expert does not exist makes its row of out
 * NaN, and CB_ERR_DEVICE is put into *status.
 *
 * With swiglu the matrix's first n / 2 rows are a gate and the others the
 * values it opens: out has n / 2 columns, SiLU(y[j]) y[n / 2 + j], from the
 * unrounded sums.  Not with weights.
 */
#define CB_INT4_MAX_ROWS CB_MOE_MAX_FEW
#define CB_INT4_MAX_K 49152 /* with ids; eight times as much without */
typedef struct {
  const void *x;          /* bf16 [rows][k], or e4m3 with x_scales; row stride ld_x elements */
  const float *x_scales;  /* [rows][ceil(k / 128)], or NULL: x is bf16           */
  const uint8_t *codes;   /* [n_experts][n][k / 2], element 2i in the low nibble of byte i */
  const float *scales;    /* [n_experts][k / group][n]                           */
  const uint8_t *zeros;   /* [n_experts][k / group][n], 0..15, or NULL: all 8    */
  const int32_t *ids;     /* [n_tokens][top_k], or NULL                          */
  const float *w;         /* [n_tokens][top_k], or NULL                          */
  void *out;              /* row stride ld_out elements                          */
  int32_t *status;        /* device int32, or NULL: bad ids are not reported     */
  int64_t ld_x, ld_out;
  int64_t n, k;           /* n: a multiple of 16 (32 with swiglu), k: of group   */
  int32_t n_tokens;       /* 0..CB_INT4_MAX_ROWS                                 */
  int32_t top_k;          /* 1 without ids, else 1..16                           */
  int32_t n_experts;      /* 1 without ids, else 1..256                          */
  int32_t group;          /* 32, 64 or 128                                       */
  int32_t x_per_slot;     /* x has n_tokens top_k rows                           */
  int32_t swiglu;
  int32_t out_type;       /* cb_dtype_t                                          */
} cb_int4_matmul_t;

/* Errors: CB_ERR_INVALID_ARG (NULL, negative sizes, an unknown type or group,
 * n or k not such multiples, row strides below the columns, weights without
 * ids or with swiglu, x_per_slot without ids, out overlapping an input),
 * CB_ERR_ALIGNMENT (x, codes, scales, zeros: 16 bytes; several rows of x: 16 bytes each (8 in 8 bits);
 * out: its element; the others: 4), CB_ERR_UNSUPPORTED (more than
 * CB_INT4_MAX_ROWS tokens, 16 slots or 256 experts, n above 2^24, k above
 * CB_INT4_MAX_K, a wrong GPU), CB_ERR_CUDA. */
CB_API cb_status_t cb_int4_matmul_few(const cb_int4_matmul_t *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CB_SERVE_H */
