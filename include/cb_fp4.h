/*
 * cb_fp4.h -- 4-bit floating point with block scales on a GB300: quantisation
 * of a matrix's rows, its way back, and the product of two such matrices, one
 * pair or one right-hand matrix per expert.
 *
 * An element is an e2m1 code c (sign, 2 exponent bits, 1 mantissa bit):
 *   v(c) in {0, 0.5, 1, 1.5, 2, 3, 4, 6} and the same negated.
 * Two formats share it (the published OCP Microscaling Formats v1.0, and the
 * 16-element variant that the tensor core also takes):
 *   CB_FP4_MX: 32 consecutive elements of a row share a byte b in 0..254 that
 *     stands for 2^(b - 127); b = 255 is NaN.  X = 2^(b - 127) v(c).
 *   CB_FP4_NV: 16 consecutive elements share an e4m3 byte s (sign 0; 0x7F is
 *     NaN), and the matrix has one fp32 scale g.  X = g s v(c).
 *
 * Layouts (R rows, K columns, K a multiple of 32; nb = K / 32 or K / 16 blocks):
 *   codes   uint8 [R][K / 2], element 2i in the low nibble of byte i (as
 *           CB_W_INT4 packs its codes);
 *   scales  uint8 [ceil(R / 128)][ceil(nb / 4)][32][4][4]: the scale of row r
 *           and block j is byte [r / 128][j / 4][r % 32][r / 32 % 4][j % 4]:
 *           tiles of 128 rows x 4 blocks, in the order in which the tensor
 *           core takes them.  Padding rows and blocks of the last tiles are
 *           part of the array and must hold finite scales (the quantiser
 *           writes zeros).  cb_fp4_scale_bytes gives its size.
 *
 * Conventions are those of cb_moe.h: device pointers, 16-byte aligned where
 * not said otherwise, work enqueued on `stream` of the current device,
 * arguments checked before anything is enqueued, no allocation and no
 * synchronisation (but in cb_fp4_last_error).  The others can be captured into
 * a graph.  The calls keep no state but a device's error word: they are safe
 * from several threads and on several streams.
 */
#ifndef CB_FP4_H
#define CB_FP4_H

#include "cb_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { CB_FP4_MX = 0, CB_FP4_NV = 1 } cb_fp4_format_t;
typedef enum { CB_T_BF16 = 0, CB_T_F32 = 1 } cb_dtype_t;

/* Bytes of the scale array of a rows x cols matrix.  CB_ERR_INVALID_ARG: an
 * unknown format, negative rows, cols not a positive multiple of 32, NULL. */
CB_API cb_status_t cb_fp4_scale_bytes(int32_t format, int64_t rows, int64_t cols, uint64_t *bytes);

/*
 * Quantise x [rows][cols] (x_type, row stride ld elements) into codes and
 * scales.  Per block with a = its largest magnitude:
 *   MX: e = floor(log2 a) - 2, clamped to -127..125 (-127 for a = 0), scale 2^e;
 *   NV: s = the e4m3 value nearest a / (6 g), ties to the even code, at most
 *       448; g = *tensor_scale (device fp32), a value such as
 *       max|x| / (6 * 448) that puts the largest block scale at 448.  Where g
 *       is not above 0 (that formula's value for zeros) s = 0.
 * Each element is the nearest v of x / scale, ties to the even code,
 * magnitudes past 6 becoming 6.  The quotients are rounded as if computed
 * exactly, so a result depends on nothing but x and g.  (x / scale is 0 where
 * s = 0.)  A block that holds a NaN or an infinity gets the NaN scale and
 * zero codes.
 * tensor_scale must be NULL for MX.  codes and scales are as laid out above,
 * the scale array's padding is written as zeros.  ld >= cols; rows that do
 * not start on 16 bytes are read in smaller pieces.
 * Errors: CB_ERR_INVALID_ARG (an unknown format or type, NULL, negative rows,
 * cols not a positive multiple of 32, ld < cols, a tensor_scale where there
 * is none or none where there is one, x, codes and scales overlapping), CB_ERR_ALIGNMENT (codes or scales not
 * on 16 bytes, x not on its element's size, tensor_scale not on 4 bytes),
 * CB_ERR_UNSUPPORTED (2^31 row tiles or columns, or a wrong GPU),
 * CB_ERR_CUDA.
 */
CB_API cb_status_t cb_fp4_quantize(int32_t format, const void *x, int32_t x_type, int64_t rows, int64_t cols,
                                   int64_t ld, const float *tensor_scale, uint8_t *codes, uint8_t *scales,
                                   void *stream);

/* The way back: out [rows][cols] (out_type, row stride ld) = the values that
 * the codes and scales stand for, v s exactly in fp32 (infinite past its range,
 * which the quantiser's scales do not reach), times g rounded once to fp32,
 * rounded once more to bf16 where out_type says so.  Errors as above. */
CB_API cb_status_t cb_fp4_dequantize(int32_t format, const uint8_t *codes, const uint8_t *scales,
                                     const float *tensor_scale, int64_t rows, int64_t cols, void *out,
                                     int32_t out_type, int64_t ld, void *stream);

/*
 * out [m][n] = A B^T, A [m][k] and B [n][k] both of `format`:
 *   out[i][j] = g_a g_b sum_l A[i][l] B[j][l],
 * fp32 sums on the tensor core.  MX: rounded once, to out_type.  NV: g_a g_b
 * and its product with the sum are rounded to fp32 each (neither leaves its
 * range where the result does not), then to out_type.
 *
 * Experts' products: with n_groups = E >= 1 and tile_offsets (device int32
 * [E + 1], ascending from 0), B is E matrices and rows
 * [128 tile_offsets[e], 128 tile_offsets[e + 1]) of A meet the e-th:
 * b_codes [E][n][k / 2], b_scales E arrays of cb_fp4_scale_bytes(n, k), and
 * b_tensor_scale [E].  tile_offsets is what cb_moe_routing calls
 * tile_offsets: every expert's rows start a tile of 128.  Rows of A past
 * 128 tile_offsets[E] are not read, and those rows of out not written.
 * Without tile_offsets (NULL) n_groups must be 1.
 */
typedef struct {
  int32_t format;               /* cb_fp4_format_t, of both operands            */
  int32_t out_type;             /* cb_dtype_t                                   */
  int64_t m, n, k;              /* k: a positive multiple of 32                 */
  const uint8_t *a_codes;
  const uint8_t *a_scales;
  const float *a_tensor_scale;  /* device fp32, NV only, else NULL              */
  const uint8_t *b_codes;
  const uint8_t *b_scales;
  const float *b_tensor_scale;  /* device fp32 [n_groups], NV only, else NULL   */
  int32_t n_groups;
  const int32_t *tile_offsets;  /* device [n_groups + 1], or NULL               */
  void *out;                    /* row stride ld_out elements, on 16 bytes      */
  int64_t ld_out;               /* >= n                                         */
  int32_t *status;              /* device int32: CB_ERR_TIMEOUT is put there if
                                   a device-side wait ran past its bound (out
                                   is then garbage); else untouched.  NULL: the
                                   device's own word, see cb_fp4_last_error     */
} cb_fp4_matmul_t;

/* Errors: CB_ERR_INVALID_ARG (NULL, an unknown format or type, negative sizes,
 * a bad k, ld_out < n, tensor scales that do not fit the format, n_groups < 1,
 * or > 1 without tile_offsets, out overlapping an operand), CB_ERR_ALIGNMENT,
 * CB_ERR_UNSUPPORTED (a size of 2^31 or more, n_groups n of 2^31 or more, a
 * wrong GPU), CB_ERR_CUDA. */
CB_API cb_status_t cb_fp4_matmul(const cb_fp4_matmul_t *args, void *stream);

/* Synchronise the current device, return what its products without a status
 * word of their own ran into since the last such call (CB_OK or
 * CB_ERR_TIMEOUT), and clear it.  CB_ERR_UNSUPPORTED (a wrong GPU),
 * CB_ERR_CUDA. */
CB_API cb_status_t cb_fp4_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* CB_FP4_H */
