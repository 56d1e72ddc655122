/*
 * dyt_lm.h - C ABI of the operators around a decoder's blocks on AMD Instinct
 * MI355X (gfx950): root-mean-square norm (plain, with the residual add in
 * front, with an 8-bit output), embedding lookup with its gradient, log
 * probabilities of given tokens with entropy, top alternatives and gradient,
 * and an AdamW step over many tensors. Library libdyt_lm.so.
 *
 * Conventions: those of dyt.h (device pointers, dtype codes, dyt_status,
 * stream as void*, validation before anything is enqueued, caller-owned
 * buffers, no device allocation, float32 arithmetic and accumulation, no
 * floating-point atomics: results are bitwise reproducible and depend on the
 * arguments only). No output may overlap an input or another output, except
 * where it says so.
 */
#ifndef DYT_LM_H_
#define DYT_LM_H_

#include <stddef.h>
#include <stdint.h>

#include "dyt.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DYT_LM_ABI_VERSION 1

int dyt_lm_abi_version(void);
const char* dyt_lm_build_id(void);

/* --------------------------------------------------- root-mean-square norm
 * Over an M x N row-major activation, per row i:
 *
 *   rstd_i = 1 / sqrt(sum_j x[i,j]^2 / N + eps)    n[i,j] = x[i,j] rstd_i
 *   y[i,j] = gamma[j] n[i,j]                       d[i,j] = dy[i,j] gamma[j]
 *   dx[i,j] = rstd_i (d[i,j] - n[i,j] sum_j (d n)[i,j] / N)
 *   dgamma[j] = sum_i dy[i,j] n[i,j]
 *
 * x, y, dy, dx, h, r, dres: [M, N] of x_dtype; ld*: row pitch in elements
 * (>= N; 0 means N). gamma, dgamma: [N] of param_dtype. rstd: [M] float32.
 * The squares are float32: a row whose sum of squares passes 3.4e38 has
 * rstd = 0, and elements below 1e-19 lose digits in their squares (which matters with
 * an eps of 0 only). M == 0 or N == 0: nothing is read; the backward still writes
 * zeros to dgamma.
 */
int dyt_rms_forward(const void* x, int64_t ldx, const void* gamma, void* y, int64_t ldy,
                    float* rstd, int64_t M, int64_t N, float eps, int x_dtype, int param_dtype,
                    void* stream);

/* h = x + r (rounded to x_dtype), then the norm of h; contiguous rows. */
int dyt_rms_forward_residual(const void* x, const void* r, const void* gamma, void* h, void* y,
                             float* rstd, int64_t M, int64_t N, float eps, int x_dtype,
                             int param_dtype, void* stream);

/* The norm in 8 bits: q[i,j] = y[i,j] / scale rounded to the nearest e4m3
 * value (float8 with 4 exponent and 3 mantissa bits, largest value 448), from
 * the float32 y. A scale is the largest |y| of its columns / 448, at least
 * 2^-126; one for each row (group 0, scales [M]) or for each `group` = 32, 64
 * or 128 neighbouring columns (scales [M, ceil(N / group)]). q: [M, N]
 * contiguous bytes. A NaN element becomes a NaN code and is left out of the
 * scale. With r (or NULL): h = x + r is written too, and x is contiguous. */
int dyt_rms_forward_q8(const void* x, int64_t ldx, const void* r, const void* gamma, void* h,
                       void* q, float* scales, int64_t M, int64_t N, int group, float eps,
                       int x_dtype, int param_dtype, void* stream);

/* Bytes of workspace the backward needs (0 for an empty problem or bad arguments). */
size_t dyt_rms_backward_workspace_size(int64_t M, int64_t N, int x_dtype, int param_dtype);

int dyt_rms_backward(const void* x, int64_t ldx, const void* dy, int64_t lddy, const float* rstd,
                     const void* gamma, void* dx, int64_t lddx, void* dgamma, void* workspace,
                     size_t workspace_bytes, int64_t M, int64_t N, int x_dtype, int param_dtype,
                     void* stream);

/* dx = dres + (the norm's backward of dy at h); contiguous rows. */
int dyt_rms_backward_residual(const void* h, const void* dy, const void* dres, const float* rstd,
                              const void* gamma, void* dx, void* dgamma, void* workspace,
                              size_t workspace_bytes, int64_t M, int64_t N, int x_dtype,
                              int param_dtype, void* stream);

/* --------------------------------------------------------------- embedding
 *
 *   y[t] = scale weight[token_t]      dweight[v] = scale sum_{t: token_t = v} dy[t]
 *
 * tokens: [T] integers of `token_bits` (32 or 64). A token outside [0, V)
 * (padding, an ignored place) gives a row of zeros and takes part in no
 * gradient. weight: [V, D] of w_dtype, y and dy: [T, D], dweight: [V, D];
 * ld*: row pitch in elements (>= D; 0 means D). T and V are at most 2^31 - 2,
 * D 2^30. Products and sums are float32, rounded once.
 */
int dyt_embed_forward(const void* weight, int64_t ldw, const void* tokens, void* y, int64_t ldy,
                      int64_t T, int64_t V, int64_t D, float scale, int w_dtype, int y_dtype,
                      int token_bits, void* stream);

/* Bytes of workspace the backward needs (0 for an empty problem or bad arguments). */
size_t dyt_embed_backward_workspace_size(int64_t T, int64_t V, int64_t D);

/* Writes every row of dweight, zeros for tokens that do not occur; with
 * `accumulate` it adds to the rows of those that do and leaves the others
 * alone. Sums are taken in the order of the places, in pieces that depend on
 * T, V, D and how often a token occurs. */
int dyt_embed_backward(const void* dy, int64_t lddy, const void* tokens, void* dweight, int64_t lddw,
                       void* workspace, size_t workspace_bytes, int64_t T, int64_t V, int64_t D,
                       float scale, int dy_dtype, int dw_dtype, int token_bits, int accumulate,
                       void* stream);

/* ------------------------------------------------- token log probabilities
 * Over a row x of V logits, z[j] = scale x[j], with a token c:
 *
 *   lse = log sum_j exp(z[j])        logp = z[c] - lse
 *   entropy = lse - sum_j p[j] z[j]  p[j] = exp(z[j] - lse)
 *   dx[j] = scale (dlogp ([j = c] - p[j]) - dentropy p[j] (z[j] - lse + entropy))
 *
 * logits, dlogits: [T, V] of dtype; ld*: row pitch in elements (>= V; 0 means
 * V). tokens: [T] of `token_bits` (32 or 64); one outside [0, V) (an ignored
 * place) has logp = 0 and no gradient of it. logp, entropy, lse, dlogp,
 * dentropy: [T] float32. scale (an inverse temperature): positive and finite.
 * V is at most 2^26 (with alternatives 2^23), T 2^31 - 1.
 *
 * A logit of -inf, or with scale x below -2.35e38 (float32's range as a power of
 * two: the lowest float32 and bfloat16 values), is a masked place: p = 0 and
 * gradient 0, but for the row's own token, whose dx is scale dlogp there too (as
 * everywhere, [j = c] - p[j] is 1) and whose logp is -inf. A row of nothing else has
 * lse = -inf, logp = -inf, entropy 0 and gradient 0, the token's included. A NaN, +inf
 * or scale x above 2.35e38 makes its row's results NaN. Exponentials below 2^-126 count as 0.
 *
 * norm: [T, 3] float32, m and log2 s with p[j] = 2^(k x[j] - m - log2 s), k the float32
 * product of scale and log2(e), and the entropy: a row's lse in powers of two, in two
 * numbers (log2 s -inf where every place is masked). The gradient from norm keeps its digits
 * wherever the logits lie; from the one float32 lse its relative error grows with
 * |lse| 2^-23.
 *
 * top_logp, top_tokens: [T, top] (top 0: NULL), the log probabilities
 * (float32) and places (int64) of the `top` largest logits in falling order,
 * equal ones from the lowest place on; top at most V and
 * DYT_LOGPROB_MAX_TOP. In a row with a NaN the places are some places.
 */
#define DYT_LOGPROB_MAX_TOP 64

size_t dyt_logprob_forward_workspace_size(int64_t T, int64_t V, int top, int dtype);

int dyt_logprob_forward(const void* logits, int64_t ld, const void* tokens, float* logp,
                        float* entropy, float* lse, float* top_logp, int64_t* top_tokens,
                        void* workspace, size_t workspace_bytes, int64_t T, int64_t V, float scale,
                        int top, int dtype, int token_bits, void* stream);

/* As dyt_logprob_forward, and writes norm. */
int dyt_logprob_forward_norm(const void* logits, int64_t ld, const void* tokens, float* logp,
                             float* entropy, float* lse, float* norm, float* top_logp,
                             int64_t* top_tokens, void* workspace, size_t workspace_bytes,
                             int64_t T, int64_t V, float scale, int top, int dtype, int token_bits,
                             void* stream);

/* entropy and lse are the forward's; dlogp and dentropy may each be NULL (no
 * gradient of it). dlogits may be the logits themselves (same address and
 * pitch). A row whose upstream gradients are zero gets zeros, whatever it
 * holds. */
int dyt_logprob_backward(const void* logits, int64_t ld, const void* tokens, const float* entropy,
                         const float* lse, const float* dlogp, const float* dentropy, void* dlogits,
                         int64_t ldd, int64_t T, int64_t V, float scale, int dtype, int token_bits,
                         void* stream);

/* The same with the forward's norm in place of entropy and lse. */
int dyt_logprob_backward_norm(const void* logits, int64_t ld, const void* tokens, const float* norm,
                              const float* dlogp, const float* dentropy, void* dlogits, int64_t ldd,
                              int64_t T, int64_t V, float scale, int dtype, int token_bits,
                              void* stream);

/* -------------------------------------------------------------------- AdamW
 *
 *   g' = grad_scale g      m = beta1 m + (1 - beta1) g'      v = beta2 v + (1 - beta2) g'^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 *
 * for every element of `count` tensors. param: param_dtype; grad: grad_dtype,
 * the parameter's or DYT_F32. master: float32 or NULL; where given the step is
 * the master's, and param is written from it. state_bits 32: exp_avg and
 * exp_avg_sq are float32 [n], the scales NULL. state_bits 8: they are codes [n]
 * in blocks of 128 elements with a scale each (float32 [ceil(n / 128)]):
 *   first moment   int8  c stands for scale sign(c) (c / 127)^2
 *   second moment  uint8 c stands for scale (c / 255)^4
 * The scale is the block's largest absolute value, at least 2^-126. A new value
 * between two codes takes the upper one if a random number in (0, 1) is below
 * its place between them: with `seeded` one that depends on seed, step, the
 * tensor's place in the list and the element's index, else 1/2. The second
 * moment's code is at least 1 where the moment is not zero; one below 2^-126 counts as
 * zero, in the step too. The step itself
 * uses the values before they are coded. A NaN or infinite moment spoils its
 * block's codes. All zero bytes and scales are states of zero.
 *
 * lr_dev (float32), step_dev (int64) and grad_scale (float32): device pointers
 * to one element or NULL; the first two are read in place of lr and step, so
 * that a captured step follows them. No two tensors may share memory that is
 * written.
 */
typedef struct dyt_adamw_tensor {
    void* param;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    float* avg_scale;
    float* sq_scale;
    float* master;
    int64_t n; /* 0 to 2^34 */
    int32_t param_dtype, grad_dtype;
} dyt_adamw_tensor;

typedef struct dyt_adamw_options {
    double lr, beta1, beta2, eps, weight_decay; /* finite, >= 0; the betas below 1 */
    int64_t step;                               /* from 1 on */
    const float* lr_dev;
    const int64_t* step_dev;
    const float* grad_scale;
    uint32_t seed;
    int32_t seeded;     /* 0 or 1 */
    int32_t state_bits; /* 8 or 32 */
    int32_t reserved;   /* 0 */
} dyt_adamw_options;

int dyt_adamw_step(const dyt_adamw_tensor* tensors, int64_t count, const dyt_adamw_options* options,
                   void* stream);

/* The status that dyt_adamw_step would refuse this call with, or DYT_OK; enqueues
 * nothing. (For a step of several calls, all or none of which are to be taken.) */
int dyt_adamw_check(const dyt_adamw_tensor* tensors, int64_t count, const dyt_adamw_options* options);

/* The values [n] of values_dtype that 8-bit codes stand for; second: 0 the
 * first moment's codes, 1 the second's. */
typedef struct dyt_adamw_codes {
    const void* codes;
    const float* scale;
    void* values;
    int64_t n;
    int32_t second;
    int32_t reserved; /* 0 */
} dyt_adamw_codes;

int dyt_adamw_values(const dyt_adamw_codes* list, int64_t count, int values_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DYT_LM_H_ */
