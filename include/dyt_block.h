/*
 * dyt_block.h - C ABI of the operators a transformer block needs around its
 * normalisation on AMD Instinct MI355X (gfx950): layer norm (plain and with
 * the residual add in front) and attention (grouped key heads, causal and
 * length masks, a learned relative position bias), forward and backward.
 * Library libdyt_block.so.
 *
 * Layer norm over an M x N row-major activation, per row i:
 *
 *   mean_i = sum_j x[i,j] / N          var_i = sum_j (x[i,j] - mean_i)^2 / N
 *   rstd_i = 1 / sqrt(var_i + eps)     n[i,j] = (x[i,j] - mean_i) rstd_i
 *   y[i,j] = gamma[j] n[i,j] + beta[j]
 *   d[i,j] = dy[i,j] gamma[j]
 *   dx[i,j] = rstd_i (d[i,j] - sum_j d[i,j] / N - n[i,j] sum_j (d n)[i,j] / N)
 *   dgamma[j] = sum_i dy[i,j] n[i,j]   dbeta[j] = sum_i dy[i,j]
 *
 * Attention over q [B, Sq, Hq, D], k and v [B, Sk, Hkv, D], Hq a multiple of
 * Hkv (query head h reads key head h / (Hq / Hkv)), with pos = start_b + i:
 *
 *   key j is visible to query i of batch b if j < len_b and, with the causal
 *   mask, j <= pos
 *   s[i,j] = scale q_i . k_j + table[bucket(j - pos), h]   (visible pairs)
 *   p[i,j] = exp(s[i,j]) / sum_j exp(s[i,j])               (0 elsewhere)
 *   o_i = sum_j p[i,j] v_j
 *   stats[b,h,i] = log sum_j exp(s[i,j])
 *   dv_j = sum_i p[i,j] do_i       ds[i,j] = p[i,j] (do_i . v_j - do_i . o_i)
 *   dq_i = scale sum_j ds[i,j] k_j    dk_j = scale sum_i ds[i,j] q_i
 *   dtable[t,h] = sum of ds over the pairs of bucket t
 *
 * A query that sees no key gives o = 0 and stats = -inf, and takes part in no
 * gradient; at a negative position, or in a batch entry of no keys, whatever
 * its q and do hold. Keys that no query of the batch entry sees (at or past
 * len_b, or past the last causal position) are never read: their memory may
 * hold anything, NaN included. Keys and values that some query sees, and the q
 * and do of queries that see a key, have to be finite: a product with an exact
 * zero of p still spreads a NaN.
 *
 * Buckets: with `bidirectional`, num_buckets / 2 per direction (keys after
 * the query, j > pos, take the upper half) and the distance is |j - pos|;
 * otherwise all of them and the distance is max(pos - j, 0). Of a
 * direction's n buckets the first e = n / 2 hold one distance each; bucket
 * e + t starts at the smallest whole distance d with
 * (d / e)^(n - e) >= (max_distance / e)^t, and the last takes the rest.
 *
 * Conventions: those of dyt.h (device pointers, dtype codes, dyt_status,
 * stream as void*, validation before anything is enqueued, caller-owned
 * buffers, no device allocation, float32 arithmetic and accumulation, no
 * floating-point atomics: results are bitwise reproducible and depend on the
 * arguments only). In the 16-bit types the probabilities and their gradients
 * are rounded to that type for the second matrix products, as the operands of
 * the matrix cores are (in float16 |p (do . v - do . o)| stays below 65,504 and
 * loses digits under 2^-14); the sums are float32. The backward takes p from the
 * float32 stats: its relative error grows with |stats| 2^-23, and a row whose
 * visible scores all lie beyond +-10^7 (a table's entries of -10^9 and no other
 * key in sight) has p of that row's largest score's keys only, not normalised.
 */
#ifndef DYT_BLOCK_H_
#define DYT_BLOCK_H_

#include <stddef.h>
#include <stdint.h>

#include "dyt.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DYT_BLOCK_ABI_VERSION 1

int dyt_block_abi_version(void);
const char* dyt_block_build_id(void);

/* ------------------------------------------------------------- layer norm
 * x, y, dy, dx, h, r, dres: [M, N] of x_dtype; ld*: row pitch in elements
 * (>= N; 0 means N). gamma, beta, dgamma, dbeta: [N] of param_dtype. mean,
 * rstd: [M] float32. M == 0 or N == 0: nothing is read; the backward still
 * writes zeros to dgamma and dbeta.
 */
int dyt_ln_forward(const void* x, int64_t ldx, const void* gamma, const void* beta, void* y,
                   int64_t ldy, float* mean, float* rstd, int64_t M, int64_t N, float eps,
                   int x_dtype, int param_dtype, void* stream);

/* h = x + r (rounded to x_dtype), then the layer norm of h; contiguous rows. */
int dyt_ln_forward_residual(const void* x, const void* r, const void* gamma, const void* beta,
                            void* h, void* y, float* mean, float* rstd, int64_t M, int64_t N,
                            float eps, int x_dtype, int param_dtype, void* stream);

/* Bytes of workspace the backward needs (0 for an empty problem or bad arguments). */
size_t dyt_ln_backward_workspace_size(int64_t M, int64_t N, int x_dtype, int param_dtype);

int dyt_ln_backward(const void* x, int64_t ldx, const void* dy, int64_t lddy, const float* mean,
                    const float* rstd, const void* gamma, void* dx, int64_t lddx, void* dgamma,
                    void* dbeta, void* workspace, size_t workspace_bytes, int64_t M, int64_t N,
                    int x_dtype, int param_dtype, void* stream);

/* dx = dres + (layer norm's backward of dy at h); contiguous rows. */
int dyt_ln_backward_residual(const void* h, const void* dy, const void* dres, const float* mean,
                             const float* rstd, const void* gamma, void* dx, void* dgamma,
                             void* dbeta, void* workspace, size_t workspace_bytes, int64_t M,
                             int64_t N, int x_dtype, int param_dtype, void* stream);

/* -------------------------------------------------------------- attention */

/* Largest head dimension, number of buckets and max_distance. */
#define DYT_ATTN_MAX_D 128
#define DYT_ATTN_MAX_BUCKETS 128
#define DYT_ATTN_MAX_DISTANCE 1024

/* Strides of a [B, S, H, D] tensor in elements; the stride of D is 1. */
typedef struct dyt_attn_strides {
    int64_t b, s, h;
} dyt_attn_strides;

/*
 * One attention problem. All of q, k, v, o, do, dq, dk, dv have `dtype`.
 *   seqlens_k  [B] int32 or NULL: valid keys of each batch entry, clamped to
 *              [0, Sk] (NULL: Sk)
 *   q_start    [B] int32 or NULL: position of query row 0 (NULL: Sk - Sq);
 *              may be negative
 *   table      [num_buckets, Hq] of table_dtype, contiguous, or NULL: no bias
 *   causal, bidirectional: 0 or 1
 *   scale      positive and finite
 * Sk and Sq Hq / Hkv are at most 2^28, Hq and Hkv 2^20, B Hq and B Hkv 2^24, and
 * no launch may need 2^32 threads (two a row and head, backward two a key and head).
 * num_buckets is even when bidirectional, and >= 2 (>= 4 when
 * bidirectional); max_distance is larger than a direction's exact buckets.
 */
typedef struct dyt_attn_desc {
    int64_t B, Sq, Sk, Hq, Hkv, D;
    dyt_attn_strides q, k, v, o, dout, dq, dk, dv;
    const int32_t* seqlens_k;
    const int32_t* q_start;
    const void* table;
    int32_t dtype, table_dtype;
    int32_t causal, bidirectional;
    int32_t num_buckets, max_distance;
    float scale;
    int32_t reserved; /* 0 */
} dyt_attn_desc;

/* Workspace bytes of the two calls (0 also for invalid arguments). */
size_t dyt_attn_forward_workspace_size(const dyt_attn_desc* desc);
size_t dyt_attn_backward_workspace_size(const dyt_attn_desc* desc);

/* o and stats [B, Hq, Sq] float32 (contiguous) are written. */
int dyt_attn_forward(const dyt_attn_desc* desc, const void* q, const void* k, const void* v,
                     void* o, float* stats, void* workspace, size_t workspace_bytes,
                     void* stream);

/* dq, dk, dv and, with a table, dtable [num_buckets, Hq] of table_dtype are
 * written whole (zeros where nothing contributes). o and stats are the
 * forward's. dq, dk and dv may be interleaved (slices of one tensor); sharing
 * an element with each other, or memory with anything else, is refused. */
int dyt_attn_backward(const dyt_attn_desc* desc, const void* q, const void* k, const void* v,
                      const void* o, const void* dout, const float* stats, void* dq, void* dk,
                      void* dv, void* dtable, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Host only: the smallest distance of every bucket of one direction, written
 * to borders[] (room for num_buckets values); returns their number or 0. */
int dyt_attn_bucket_borders(int num_buckets, int max_distance, int bidirectional,
                            int32_t* borders);

#ifdef __cplusplus
}
#endif

#endif /* DYT_BLOCK_H_ */
