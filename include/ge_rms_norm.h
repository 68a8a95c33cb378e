/*
 * ge_rms_norm.h -- root-mean-square norm with the residual's addition, an
 * optional 8-bit output with scales, and its backward pass, for AMD MI355X
 * (gfx950).  It makes the A operand of the fused product in gemm_epilog.h and
 * uses that header's status codes, element types and conventions: row-major
 * device buffers owned by the caller, 16-byte aligned rows, asynchronous
 * calls on the caller's stream, all validation before any HIP call, nothing
 * allocated, copied or synchronised.
 *
 *   forward    h = x + r, rounded to the type (r optional)
 *              rstd = 1 / sqrt(mean_j h_j^2 + eps)
 *              y_j = h_j * rstd * gamma_j, stored as the output kind says
 *   backward   with g_j = dy_j * gamma_j and n_j = h_j * rstd:
 *              dx_j = rstd * (g_j - n_j * mean_k(g_k n_k)) + dh_j
 *              dgamma_j = sum over the rows of dy_j * n_j
 *              (dx is the gradient of both x and r; dh, optional, is the
 *              gradient that reaches h itself along the residual path)
 *
 * Sums and statistics are fp32; each output is rounded once, to nearest even.
 */
#ifndef GE_RMS_NORM_H
#define GE_RMS_NORM_H

#include "gemm_epilog.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Output kinds.
 *   PLAIN     y in x's type
 *   E4M3_ROW  y as E4M3 codes of y_j / s with one fp32 scale per row,
 *             s = max_j |y_j| / 448, at least 2^-126 (1 when that maximum is 0):
 *             the A operand and row_scale of an E4M3 product
 *             (gemm_epilog_execute_residual)
 *   MX        y as E4M3 codes with one E8M0 scale byte per 32 columns: with
 *             a = max |y_j| of the block, byte = floor(log2 a) - 8 + 127
 *             (clamped to 0..254; 127 when a is 0 or not finite): the
 *             A operand and a_scales of a block-scaled product.  Rows of
 *             scales are GE_MX_SCALE_LD(cols) bytes; only the first
 *             ceil(cols/32) of each are written.
 * Codes round to nearest even and saturate at +-448.  NaN values stay NaN and
 * do not count in the maxima. */
typedef enum { GE_NORM_PLAIN = 0, GE_NORM_E4M3_ROW = 1, GE_NORM_MX = 2 } ge_norm_out;

typedef struct {
    int64_t rows;   /* the most rows of a call                                  */
    int64_t cols;   /* values per row, at least 1                                */
    int32_t type;   /* GE_F32, GE_F16 or GE_BF16: x, r, h, gamma, dy, dh, dx,
                       dgamma, and y when out is PLAIN                           */
    int32_t out;    /* ge_norm_out                                               */
    int64_t ld;     /* row stride in elements of x, r, h, dy, dh and dx          */
    int64_t ldy;    /* row stride in elements of y                               */
    float eps;      /* >= 0                                                      */
} ge_norm_desc;

typedef struct ge_norm_s* ge_norm_handle;

/* Validate a description and plan the launches (host only).
 * Errors: GE_ERR_NULL; GE_ERR_SHAPE (rows < 0, cols < 1, either beyond
 * 2^31-1, ld or ldy < cols, an unknown output kind, eps negative or not
 * finite); GE_ERR_DTYPE; GE_ERR_ALIGN (a row stride that is not a multiple of
 * 16 bytes); GE_ERR_ALLOC. */
int ge_rms_norm_create(ge_norm_handle* h, const ge_norm_desc* desc);

/* Bytes of device workspace that ge_rms_norm_backward needs (the forward pass
 * needs none).  Errors: GE_ERR_NULL. */
int ge_rms_norm_workspace_size(ge_norm_handle h, size_t* bytes);

/* Forward pass over `rows` rows (0 <= rows <= the handle's).
 *   x, gamma   inputs; gamma has cols values
 *   residual   r, or NULL for h = x
 *   h          receives the rounded sum; NULL when it is not wanted (without a
 *              residual it must be NULL: h is x)
 *   y          output (see ge_norm_out)
 *   scales     E4M3_ROW: rows fp32 values; MX: the scale bytes, 16-byte
 *              aligned; PLAIN: NULL
 *   rstd       rows fp32 values for the backward pass, or NULL
 * h may be x or residual itself, and a PLAIN y with ldy == ld may be any of
 * them (each value is read before it is written, by the same thread); no
 * other overlap.
 * Errors: GE_ERR_NULL, GE_ERR_SHAPE (rows, or a y in place with rows of its
 * own), GE_ERR_ALIGN (a matrix or gamma that is
 * not 16-byte aligned, scales or rstd not 4-byte aligned), GE_ERR_EPILOG
 * (scales or h given or missing against the rules above), GE_ERR_HIP. */
int ge_rms_norm_forward(ge_norm_handle h, int64_t rows, const void* x, const void* residual, const void* gamma,
                        void* hsum, void* y, void* scales, float* rstd, void* stream);

/* Backward pass over `rows` rows.
 *   dy      gradient of y (of the values, before any 8-bit rounding)
 *   hsum    the forward's h (x without a residual)
 *   rstd    the forward's rstd
 *   dh      gradient reaching h itself, or NULL
 *   dx      output: gradient of x and of the residual; may be dy or dh itself
 *   dgamma  output, cols values; NULL when it is not wanted (no workspace then)
 * With rows == 0 dgamma is set to zero.  The sums are taken in an order that
 * the handle and rows alone decide: equal calls give equal bits.
 * Errors: GE_ERR_NULL, GE_ERR_SHAPE, GE_ERR_ALIGN, GE_ERR_WORKSPACE,
 * GE_ERR_HIP. */
int ge_rms_norm_backward(ge_norm_handle h, int64_t rows, const void* dy, const void* hsum, const void* gamma,
                         const float* rstd, const void* dh, void* dx, void* dgamma, void* workspace,
                         size_t workspace_bytes, void* stream);

/* One line of text: the launch shapes.  Errors: GE_ERR_NULL. */
int ge_rms_norm_describe(ge_norm_handle h, char* buf, size_t cap);

/* Release the handle (NULL is accepted).  Host only. */
int ge_rms_norm_free(ge_norm_handle h);

#ifdef __cplusplus
}
#endif

#endif /* GE_RMS_NORM_H */
