/*
 * The feed-forward block of language models: the C ABI of the gated product
 * with its gradients, of microscaled 4-bit matrices, and of their products.
 *
 * Each call takes its arguments as a struct that the caller fills (zeroed
 * first: a zero or NULL field means "not given") and may keep and reuse; the
 * library reads it during the call only. Matrices are rows x columns with
 * consecutive columns and a row stride in elements (of codes: in bytes).
 * Products are taken on the tensor cores with fp32 accumulators; activations
 * are computed in fp32 from these, off by at most 2^-19 of themselves for fp32
 * outputs and 2^-16 for others, as far as they are normal numbers of fp32 (GELU
 * by tanh: by 2^-21 times the argument of its exponential besides), and each
 * output is rounded once, to nearest even.
 * Every sum is taken in a fixed order, so results are identical from run to
 * run. Calls enqueue on `stream` without synchronising, may be captured into a
 * graph, and return 0 or a negative gemm_status_t with a message in
 * gemm_last_error(): GEMM_ERR_ARG for a bad size, stride, type or a missing
 * pointer, GEMM_ERR_ALIGN, GEMM_ERR_ARCH for a current device that is not of
 * compute capability 10.3 (all pointers belong to the current device),
 * GEMM_ERR_LAUNCH. Nothing is allocated: scratch is the caller's, of the size
 * that a ..._workspace function gives; concurrent calls need scratch of their
 * own. Waits inside the kernels are bounded: where a copy or a product has not
 * come after two seconds, which no launch takes, the outputs that hang on it
 * are NaN. Sizes (and twice `hidden`) are below 2^31, matrices of fewer than
 * 2^56 elements, and no output may overlap an input or another output.
 */
#ifndef SAT_FFN_H
#define SAT_FFN_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FFN_NONE = 0,      /* a(g) = g */
    FFN_SILU = 1,      /* g / (1 + exp(-g)) */
    FFN_GELU = 2,      /* g (1 + erf(g / sqrt 2)) / 2 */
    FFN_GELU_TANH = 3, /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */
    FFN_RELU = 4       /* max(g, 0), NaN of NaN; its derivative at 0 is 0 */
} ffn_activation_t;

/* ---- gated product -----------------------------------------------------------
 *
 *   g = x Wg,  u = x Wu,  h = a(g) * u
 *
 * x is rows x width, Wg and Wu take `width` inputs to `hidden` outputs each and
 * lie in one matrix, the gate's first: with w_by_output != 0 as 2 hidden x width
 * (a row per output), else as width x 2 hidden (a row per input). preact, where
 * not NULL, receives [g u] (rows x 2 hidden, rounded to the type) for the
 * backward pass; h is computed from g and u before that rounding. width == 0
 * gives g = u = 0.
 *
 * Any alignment to elements and any stride is correct. x and w are read as they
 * lie where they start on 16 bytes with row strides that are multiples of 16
 * bytes (with w_by_output == 0, hidden a multiple of 8 too); otherwise they are
 * copied into the workspace first.
 */
typedef struct {
    int64_t rows, width, hidden;
    int32_t type;        /* of all matrices: GEMM_C_BF16 or GEMM_C_F16 */
    int32_t activation;  /* ffn_activation_t */
    int32_t w_by_output;
    const void* x; /* rows x width */
    int64_t ldx;
    const void* w; /* 2 hidden x width, or width x 2 hidden */
    int64_t ldw;
    void* h; /* rows x hidden (forward only) */
    int64_t ldh;
    void* preact; /* rows x 2 hidden, or NULL: written by the forward pass, read by the backward pass */
    int64_t ldp;
    void* workspace; /* of the forward pass, 16-byte aligned; NULL where ffn_gated_workspace gives 0 */
    int64_t workspace_bytes;
} ffn_gated_args;

/* Scratch bytes of ffn_gated for args' sizes, pointers and strides (host only; negative for bad arguments). */
int64_t ffn_gated_workspace(const ffn_gated_args* args);

int ffn_gated(const ffn_gated_args* args, void* stream);

/* The gradients, from dh:
 *
 *   dg = dh * u * a'(g),  du = dh * a(g),  dx = [dg du] [Wg Wu]^T,  dw = x^T [dg du]
 *
 * g and u come from args->preact, or, where that is NULL, are computed again
 * from x and w (one product more, nothing kept). dg and du are rounded to the
 * type in the workspace: they are operands of the products, as x and w are. dw
 * lies as w does; accumulate != 0 adds to what dw holds (fp32 only, so that
 * what is added is not rounded to fewer bits; sums below 2^-126 may become 0). Either of dx and dw may be NULL
 * and is then not computed. With rows == 0 dw is set to 0 (or left, with
 * accumulate). args->h and args->workspace are not used. */
typedef struct {
    const void* dh; /* rows x hidden */
    int64_t lddh;
    void* dx; /* rows x width */
    int64_t lddx;
    void* dw;
    int64_t lddw;
    int32_t dw_type; /* GEMM_C_F32 or args->type */
    int32_t accumulate;
    void* workspace; /* 16-byte aligned */
    int64_t workspace_bytes;
} ffn_gated_grads;

/* Scratch bytes of ffn_gated_backward (host only; negative for bad arguments). */
int64_t ffn_gated_backward_workspace(const ffn_gated_args* args, const ffn_gated_grads* grads);

int ffn_gated_backward(const ffn_gated_args* args, const ffn_gated_grads* grads, void* stream);

/* ---- microscaled 4-bit matrices ------------------------------------------------
 *
 * MXFP4 of the OCP Microscaling Formats specification 1.0: elements E2M1 (sign
 * and 0, 0.5, 1, 1.5, 2, 3, 4, 6), one UE8M0 scale 2^(byte - 127) for each 32
 * consecutive columns of a row.
 *
 *   exponent = floor(log2(largest magnitude of the block)) - 2, at least -127
 *   code     = value / 2^exponent, rounded to the nearest of E2M1's, of two
 *              equally near ones to the one with an even code; past 6 it is 6
 *
 * A block of zeros has scale byte 0. A block with a NaN or an infinity has scale
 * byte 255 and codes 0, which stands for NaN in all its columns.
 *
 * codes: row r, columns 2 i and 2 i + 1 in the lower and upper four bits of byte
 *   r ldc + i; ldc a multiple of 16, at least 16 ceil(width / 32). Columns from
 *   width to the end of the last block are 0.
 * scales: tiles of 128 rows x 4 blocks, 512 bytes each, in the order in which the
 *   tensor core reads them. Row r, block b is byte
 *     (r / 128 * ceil(width / 128) + b / 4) * 512 + r % 32 * 16 + r % 128 / 32 * 4 + b % 4
 *   of mxfp4_scale_bytes(rows, width); bytes of rows and blocks past the end are 0.
 * Both start on 16 bytes. mxfp4_quantize writes all of both but what lies between
 * a row's last block and ldc.
 */
typedef struct {
    int64_t rows, width;
    int32_t type;     /* of values: gemm_ctype_t */
    int32_t reserved; /* 0 */
    void* values;     /* rows x width: read by mxfp4_quantize, written by mxfp4_dequantize */
    int64_t ldv;
    void* codes;
    int64_t ldc; /* bytes */
    void* scales;
} mxfp4_args;

/* Bytes of the scales of a matrix (host only; negative for bad sizes). */
int64_t mxfp4_scale_bytes(int64_t rows, int64_t width);

int mxfp4_quantize(const mxfp4_args* args, void* stream);

/* values = code x scale, rounded to the type where it does not hold that (fp16 past 65504 or below 2^-24). */
int mxfp4_dequantize(const mxfp4_args* args, void* stream);

/* ---- products of microscaled matrices ---------------------------------------------
 *
 *   out = alpha A B^T,   or, with `up` given,   out = a(alpha A B^T) * (alpha A Up^T)
 *
 * A is rows x width, B and Up are cols x width, all microscaled along width as
 * above. Without up, activation must be FFN_NONE. Scale bytes past the matrices'
 * rows and blocks must be 0, and so must the codes past width in a last block.
 */
typedef struct {
    int64_t rows, cols, width;
    int32_t out_type;   /* gemm_ctype_t */
    int32_t activation; /* ffn_activation_t */
    float alpha;
    int32_t reserved; /* 0 */
    const void* a_codes;
    int64_t lda; /* bytes, of codes */
    const void* a_scales;
    const void* b_codes;
    int64_t ldb;
    const void* b_scales;
    const void* up_codes; /* or NULL */
    int64_t ldu;
    const void* up_scales;
    void* out; /* rows x cols */
    int64_t ldo;
} mxfp4_gemm_args;

int mxfp4_gemm(const mxfp4_gemm_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SAT_FFN_H */
