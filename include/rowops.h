/*
 * Row operators over a rows x width fp32 matrix, one row at a time: softmax,
 * RMSNorm and LayerNorm. The C ABI of the library's second workload.
 *
 * "Scale coverage exposes a remaining GEMM gap" (section "Reductions: wide
 * rows and large working sets") times these three operators on rows x width
 * from 37 x 8191 to 16384 x 4096, in fp32. The page names them without
 * formulas; these are the textbook ones:
 *   softmax:   y_j = exp(x_j - max_k x_k) / sum_k exp(x_k - max_k x_k)
 *   RMSNorm:   y_j = x_j / sqrt(mean_k x_k^2 + eps) * gamma_j
 *   LayerNorm: y_j = (x_j - mu) / sqrt(var + eps) * gamma_j + beta_j,
 *              mu = mean_k x_k, var = mean_k (x_k - mu)^2 (biased)
 * gamma and beta may be NULL (taken as 1 and 0).
 *
 * X and Y are device pointers to rows x width floats with row strides ldx
 * and ldy (>= width); Y may be X (in place, same stride). Reductions are in
 * fp32 in a fixed order, so results are identical from run to run. The
 * calls enqueue one kernel on `stream` and return without synchronising;
 * they return 0 or a negative gemm_status_t (message in gemm_last_error):
 * GEMM_ERR_ARG for negative sizes, NULL X/Y, strides below the width or a
 * width above ROWOP_MAX_WIDTH; GEMM_ERR_ALIGN for pointers not 4-byte
 * aligned. rows == 0 or width == 0 does nothing.
 */
#ifndef SAT_ROWOPS_H
#define SAT_ROWOPS_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest row the kernels hold (512 threads x 64 values in registers). */
#define ROWOP_MAX_WIDTH 32768

int rowop_softmax(const float* X, int64_t ldx, float* Y, int64_t ldy, int64_t rows, int64_t width, void* stream);

int rowop_rmsnorm(const float* X, int64_t ldx, const float* gamma, float* Y, int64_t ldy, int64_t rows, int64_t width,
                  float eps, void* stream);

int rowop_layernorm(const float* X, int64_t ldx, const float* gamma, const float* beta, float* Y, int64_t ldy,
                    int64_t rows, int64_t width, float eps, void* stream);

/* ==== Row operators of language models ====================================
 *
 * What a language model needs beside its matrix products, one row (token) at
 * a time: the step between two blocks with its gradients, the loss that
 * trains a model from a larger one's stored top logits, and the check of
 * tokens that a small model drafted for a larger one.
 *
 * Each call takes its arguments as a struct that the caller fills (zeroed
 * first: a zero or NULL field means "not given") and may keep and reuse; the
 * library reads it during the call only. Matrices are rows x columns with
 * consecutive columns and a row stride in elements. Element types are those
 * of gemm_ctype_t. Whatever the types, sums, statistics and every
 * intermediate value are fp32, and each output is rounded once, to nearest
 * even. Results are identical from run to run: every sum is taken in a
 * fixed order. Calls enqueue on `stream` without synchronising and return 0
 * or a negative gemm_status_t, as above: GEMM_ERR_ARG for a bad size, stride,
 * type or a missing pointer, GEMM_ERR_ALIGN for a pointer that is not aligned
 * to its element, GEMM_ERR_LAUNCH. Nothing is allocated: scratch is the
 * caller's, of the size that a ..._workspace function gives; concurrent calls
 * need scratch of their own. Waits inside the kernels are bounded: where a
 * copy has not come after two seconds, which no launch takes, the outputs
 * that hang on it are NaN. Rows of any alignment and stride are correct.
 * The fast ones: in the block norm, where all of a call's rows start on
 * boundaries of eight elements (16 bytes in 16-bit types, 32 in fp32), the
 * weights' vectors on 32 bytes, and the width is a multiple of eight;
 * otherwise all of its elements move one by one. In the distillation logits
 * move by 16 bytes wherever their rows start, and the gradient where its rows
 * start on the same byte of 16 as the logits'. In the verification the draw is
 * fast where target, draft and noise rows start on 16 bytes.
 */

/* ---- block norm: norm after a block, gate, residual, norm before the next --
 *
 *   n = N_post(y);   h = residual_scale x + branch_scale (gate * n);   z = N_pre(h)
 *
 * x is the residual stream, y a block's output, z the next block's input.
 * N is none (n = y; with pre_norm none there is no z), RMS
 * (v / sqrt(mean v^2 + eps) gamma) or Layer ((v - mean v) / sqrt(var + eps)
 * gamma + beta, var biased), each with its own weights; a NULL gamma is 1, a
 * NULL beta 0, and beta belongs to Layer only. Row r is scaled by gate row
 * r / rows_per_gate: rows_per_gate >= rows for one vector for all rows, a
 * sequence's length for a row per sequence, 1 for a row per token. z is the
 * norm of h before its rounding to the stream's type.
 */
typedef enum { ROWOP_NORM_NONE = 0, ROWOP_NORM_RMS = 1, ROWOP_NORM_LAYER = 2 } rowop_norm_t;

/* Widest row of the block norm (of fewer than 2^31 rows). */
#define ROWOP_BLOCK_NORM_MAX_WIDTH 16384

typedef struct {
    int64_t rows, width;
    int32_t block_type;  /* of y and z (and dy, dz) */
    int32_t stream_type; /* of x and h (and dx, dh): GEMM_C_F32 or block_type */
    int32_t gate_type;   /* of gate (and dgate): GEMM_C_F32 or block_type */
    int32_t post_norm, pre_norm; /* rowop_norm_t */
    float post_eps, pre_eps;
    float residual_scale, branch_scale;
    const void* x; /* rows x width (forward only) */
    int64_t ldx;
    const void* y; /* rows x width */
    int64_t ldy;
    const float* post_gamma; /* width */
    const float* post_beta;
    const float* pre_gamma;
    const float* pre_beta;
    const void* gate; /* ceil(rows / rows_per_gate) x width, or NULL for 1 */
    int64_t ldg;
    int64_t rows_per_gate;
    void* h; /* rows x width: written by the forward pass, read by the backward pass. May be x, with its stride. */
    int64_t ldh;
    void* z; /* rows x width (forward only; NULL with pre_norm none). May be y, with its stride. */
    int64_t ldz;
    float* post_stats; /* rows x 2: each row's (mean, 1 / sqrt(var + eps)) of y; mean 0 for RMS. Written by the  */
    float* pre_stats;  /* forward pass where not NULL, read by the backward pass; of h likewise. */
} rowop_block_norm_args;

int rowop_block_norm(const rowop_block_norm_args* args, void* stream);

/* The gradients, from dh (the gradient of h from its other uses; NULL for 0)
 * and dz. Of *args the backward pass reads the sizes, types, scales, weights,
 * gate, y, h and the statistics (needed for each norm there is; h is needed
 * with a pre_norm). With a pre_norm dz is needed, without one dh is. Any
 * output may be NULL and is then not computed. dx may be dh and dy may be dz,
 * with their strides. Sums over rows go through fp32 partial sums in
 * `workspace`, in a fixed order. With rows == 0 the weights' gradients are
 * set to 0. */
typedef struct {
    const void* dh;
    int64_t lddh;
    const void* dz;
    int64_t lddz;
    void* dx; /* stream type */
    int64_t lddx;
    void* dy; /* block type */
    int64_t lddy;
    void* dgate; /* gate type, one row per gate row */
    int64_t lddg;
    float* dpost_gamma; /* width */
    float* dpost_beta;
    float* dpre_gamma;
    float* dpre_beta;
    void* workspace; /* 32-byte aligned */
    int64_t workspace_bytes;
} rowop_block_norm_grads;

/* Scratch bytes of the backward pass for args' sizes and gate (host only; negative for bad sizes). */
int64_t rowop_block_norm_workspace(const rowop_block_norm_args* args);

int rowop_block_norm_backward(const rowop_block_norm_args* args, const rowop_block_norm_grads* grads, void* stream);

/* ---- distillation from a teacher's top logits -------------------------------
 *
 * Row r has the student's logits s over the vocabulary and, of the teacher,
 * the k largest logits T_i with their ids. With temperature t,
 *
 *   p_i = exp(T_i / t - L),  L = log sum_i exp(T_i / t), or teacher_lse[r]
 *   q = softmax(s / t),      P = sum_i p_i
 *   loss[r] = weight[r] t^2 sum_i p_i (log p_i - log q_id(i))
 *   dlogits[r][j] = dloss[r] weight[r] t (P q_j - sum of the p_i whose id is j)
 *
 * teacher_lse, where given, is the log of the sum of exp(T / t) over the
 * teacher's whole vocabulary (then P < 1). An entry whose id is negative or
 * >= vocab, or whose logit is -inf, is absent. A row of weight 0, or with no
 * entry present, has loss, lse and gradient 0, whatever its logits are.
 * Student logits of -inf are tokens of probability 0. lse[r] is
 * log sum_j exp(s_j / t). rows is at most 2^26, vocab 2^30.
 */
#define ROWOP_DISTILL_MAX_K 1024

typedef struct {
    int64_t rows, vocab, k;
    int32_t logits_type, teacher_type;
    float temperature;  /* > 0 */
    const void* logits; /* rows x vocab */
    int64_t ldl;
    const int32_t* ids; /* rows x k */
    int64_t ldi;
    const void* teacher; /* rows x k */
    int64_t ldt;
    const float* teacher_lse; /* rows, or NULL */
    const float* weight;      /* rows, or NULL for 1 */
    float* loss;              /* rows */
    float* lse;               /* rows: written by rowop_distill where not NULL, read by the backward pass */
    const float* dloss;       /* rows: the gradient of each row's loss, or NULL for 1 */
    void* dlogits;            /* rows x vocab, of logits_type. May be logits, with its stride. */
    int64_t ldd;
} rowop_distill_args;

/* Writes loss, lse (where not NULL) and, where dlogits is not NULL, the
 * gradient: with the gradient of the loss known, one call reads the logits
 * once and writes their gradient once. */
int rowop_distill(const rowop_distill_args* args, void* stream);

/* Writes dlogits from a forward call's lse (loss is not used). In 32 bits lse
 * is good to |lse| 2^-24, a relative error of q; rows with |lse| above 64 (in
 * 16-bit logits 512) are read a second time for their sums instead, by one CTA. */
int rowop_distill_backward(const rowop_distill_args* args, void* stream);

/* ---- verification of drafted tokens -------------------------------------------
 *
 * Sequence b has up to `drafts` drafted tokens x_0, x_1, ... With
 * p_i = softmax(target row i / temperature) and q_i = softmax(draft row i /
 * draft_temperature), token i is accepted while
 *
 *   uniforms[b][i] q_i(x_i) < p_i(x_i).
 *
 * At the first token n that is not, the next token is drawn from
 * max(p_n - q_n, 0); after all have been accepted (n = lengths[b]), from p_n.
 * So the tokens are distributed as the target's own. The draw is an
 * exponential race: the token that maximises r_j / noise[b][j], the lowest of
 * them where several do, for r the unnormalised probabilities and noise
 * independent Exp(1) values (> 0). Where p - q is nowhere positive (which
 * only rounding brings about after a refusal) the draw is from p_n.
 * With draft NULL the drafts have no distribution (q_i is 1 at x_i, 0
 * elsewhere). With temperature 0 the target's distribution is 1 at its
 * largest logit (the lowest token of several): tokens are accepted while they
 * are that token, and uniforms, noise and draft are not read.
 *
 * accepted[b] = n; out[b] = the n accepted tokens, the drawn one, then -1.
 * logprobs[b], where not NULL, holds log p of each of out[b]'s tokens
 * (temperature 0: at temperature 1), then 0. A drafted token outside the vocabulary is
 * refused. Logits of -inf have probability 0. A row without a distribution (all -inf, or a NaN or
 * +inf in it) refuses the token and draws -1, with logprob 0; a draft row
 * without one refuses the token, and the draw is from p_n. With drafts == 0
 * this is plain sampling. batch is at most 2^20, vocab 2^30.
 */
#define ROWOP_VERIFY_MAX_DRAFTS 64

typedef struct {
    int64_t batch, drafts, vocab;
    int32_t logits_type;     /* of target and draft */
    float temperature;       /* >= 0 */
    float draft_temperature; /* > 0 where draft is read */
    const void* target;      /* batch (drafts + 1) x vocab: row b (drafts + 1) + i */
    int64_t ldt;
    const void* draft; /* batch drafts x vocab: row b drafts + i; or NULL */
    int64_t ldq;
    const int32_t* tokens;  /* batch x drafts */
    const int32_t* lengths; /* batch: drafted tokens of each sequence, clamped to 0 .. drafts; NULL: all drafts */
    const float* uniforms;  /* batch x drafts, in [0, 1) */
    const float* noise;     /* batch x vocab, > 0 */
    int64_t ldn;
    int32_t* accepted; /* batch */
    int32_t* out;      /* batch x (drafts + 1) */
    float* logprobs;   /* batch x (drafts + 1), or NULL */
    void* workspace;   /* 16-byte aligned */
    int64_t workspace_bytes;
} rowop_verify_args;

/* Scratch bytes of rowop_verify (host only; negative for bad sizes). */
int64_t rowop_verify_workspace(int64_t batch, int64_t drafts, int64_t vocab);

int rowop_verify(const rowop_verify_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#ifdef __cplusplus
constexpr int kRowopMaxWidth = ROWOP_MAX_WIDTH;
#endif

#endif
