/*
 * mla_layer_ops.h -- C ABI of the attention layer around the latent pool on
 * GB300 (sm_103a): norms of queries and latents with the rotary positions and
 * the pool write, the per-head products of latent attention's absorbed and
 * expanded forms, and causal attention over expanded keys and values.
 *
 *   absorbed (few new tokens): mla_norm_rope_write -> mla_head_product (queries
 *     to the latent space) -> mla_tree_verify_run -> mla_head_product (latent
 *     outputs to values)
 *   expanded (prompts): mla_norm_rope_write -> mla_kv_defrag (a request's rows
 *     in one run) -> mla_head_product (latents to keys and values)
 *     -> mla_prefill_run
 *
 * Conventions (as in mla_tree_verify.h): every pointer named "device" is a
 * CUDA device pointer; buffers are caller-owned; nothing allocates or
 * synchronises, so every call may be captured in a CUDA graph; no call keeps
 * state of its own; the return value is MTV_OK (0) or a negative MTV_E* code.
 * Nothing is launched then, with one exception: MTV_E_CUDA of a split
 * mla_prefill_run whose second kernel was refused, which leaves out and lse
 * unwritten.  `err` (device, may be NULL) is a sticky 32-bit word the kernels
 * OR MTV_DEVERR_* bits into; data-dependent problems never trap.
 */
#ifndef MLA_LAYER_OPS_H_
#define MLA_LAYER_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_step_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest k_dim and n_dim of mla_head_product. */
#define MTV_MAX_HEAD_DIM 1024
/* Most heads of mla_head_product and mla_prefill_run, and most requests of the
 * latter. */
#define MTV_MAX_HEADS 65535
/* Longest head that mla_norm_rope_write normalises. */
#define MTV_MAX_NORM_DIM 1024
/* Most query or key rows of mla_prefill_run. */
#define MTV_MAX_PREFILL_ROWS (1 << 30)
/* Most splits of mla_prefill_run's keys. */
#define MTV_MAX_PREFILL_SPLITS 64
/* What mla_prefill_run's nsplit holds above the split count: see there. */
#define MTV_PREFILL_SPLIT_LAST 256
/* Test only, added n times (1 .. 255) to the dtype of mla_head_product or
 * mla_prefill_run: waits inside the tensor-core kernels that have to spin give
 * up once 512 (n - 1) cycles of their block have passed, in place of a second. */
#define MTV_TEST_GIVE_UP 0x100

/*
 * mla_head_product -- one matrix product a head.
 *
 *   out[t, h, n] = sum_k x[t, h, k] w[h, k, n]
 *
 * summed in fp32, rounded once to nearest-even.  With one up-projection
 * U [heads, part, 512] it is the absorption of a query's plain part (x the
 * queries, w[h] = U[h]: k_dim = part, n_dim = 512), the values of latent
 * outputs (w[h] = U[h] transposed, by its strides), and, with
 * x_head_stride = 0, the expansion of one latent a token to every head.
 *
 * x              device: element (t, h, k) at t * x_tok_stride +
 *                h * x_head_stride + k (strides in elements; x_head_stride 0
 *                gives every head the same rows).
 * w              device: element (h, k, n) at h * w_head_stride +
 *                k * w_k_stride + n * w_n_stride.
 * out            device: element (t, h, n) at t * out_tok_stride +
 *                h * out_head_stride + n.  Distinct elements may not share an
 *                address, nor overlap x or w.
 * num_tokens     0 .. 2^31 - 1.
 * num_heads      0 .. MTV_MAX_HEADS.
 * k_dim, n_dim   1 .. MTV_MAX_HEAD_DIM.
 * dtype          MTV_DTYPE_BF16 or MTV_DTYPE_FP16, of x, w and out.
 * err            device uint32 or NULL: MTV_DEVERR_TIMEOUT when a bounded wait
 *                gave up (outputs of that block may be missing).
 *
 * Any strides are taken.  The tensor-core kernel runs where every address and
 * every stride but the innermost is a multiple of 16 bytes, n_dim is a multiple
 * of 8 and w is dense in k or in n; other layouts take a plain kernel.
 */
int mla_head_product(const void* x, int64_t x_tok_stride, int64_t x_head_stride, const void* w,
                     int64_t w_head_stride, int64_t w_k_stride, int64_t w_n_stride, void* out,
                     int64_t out_tok_stride, int64_t out_head_stride, int64_t num_tokens, int num_heads, int k_dim,
                     int n_dim, int dtype, uint32_t* err, void* stream);

/*
 * mla_prefill_workspace -- workspace of mla_prefill_run and its split count,
 * from upper bounds.  Host only; reads no device.
 *
 * num_sms        SM count of the device (>= 1).
 * bs, max_q, max_kv, num_q, num_heads   as for mla_prefill_run.
 * nsplit_out     host: the nsplit of mla_prefill_run.  The keys are split where
 *                the queries alone leave SMs without work: all blocks' where
 *                there are fewer than SMs, else those of the last, part-filled
 *                wave.
 * bytes_out      host: 0 with one split.
 */
int mla_prefill_workspace(int num_sms, int bs, int64_t max_q, int64_t max_kv, int64_t num_q, int num_heads,
                          int* nsplit_out, uint64_t* bytes_out);

/*
 * mla_prefill_run -- attention of new tokens over expanded keys and values.
 *
 * For request r with n queries (rows qo_indptr[r] ..) and L keys (rows
 * kv_indptr[r] ..), query i and head h:
 *   s_j = scale (q[i, h, 0:128] . k_nope[j, h, :] + q[i, h, 128:192] . k_rope[j, :])
 *   out = softmax(s) v[:, h, :],  lse = ln sum exp(s)
 * over the keys j < L, and with `causal` j <= L - n + i (the last query sees
 * every key).  A query that sees no key has out = 0, lse = -inf.  Scores, sums
 * and lse are held in fp32.  The product with v takes the weights rounded to dtype
 * (by half a step at most, or in fp16 2^-32 of the row's largest where that is
 * more), and out is divided by the sum of the rounded ones.
 *
 * q              device, [num_q, heads, 192]: element (t, h, d) at t * q_tok_stride
 *                + h * q_head_stride + d (strides in elements, here and below).
 * k_nope, v      device, [num_kv, heads, 128] each, with strides as q.
 * k_rope         device, [num_kv, 64], row t at t * k_rope_stride: shared by
 *                the heads.
 * qo_indptr      device, int64 [bs + 1]: offsets of the requests' queries.
 * kv_indptr      device, int32 [bs + 1]: offsets of their keys.
 * bs             0 .. MTV_MAX_HEADS.
 * max_q, max_kv  host: bounds of n and L (they size the grid).
 * num_q, num_kv  host: rows of the buffers, at most MTV_MAX_PREFILL_ROWS.
 * num_heads      0 .. MTV_MAX_HEADS.
 * dtype          MTV_DTYPE_BF16 or MTV_DTYPE_FP16: q, k_nope, k_rope, v, out.
 *                All their addresses and strides are multiples of 16 bytes.
 * scale          > 0, finite also as a multiple of log2(e).
 * causal         0 or 1.
 * out            device, [num_q, heads, 128] with strides as q.
 * lse            device, fp32 [num_q, heads], or NULL to leave it out.
 * nsplit         mla_prefill_workspace's, or any n + MTV_PREFILL_SPLIT_LAST * b
 *                with 1 <= n <= MTV_MAX_PREFILL_SPLITS: the keys of the last b
 *                blocks (256 rows of a head; all blocks where b is 0 or more
 *                than there are) are split n ways.
 * workspace      device, 256-byte aligned, with n > 1: n * rows * 129 * 4 bytes at
 *                least, rows being num_q * num_heads with b = 0, else 256 a split
 *                block.  Calls that may overlap need one each.  With n = 1 it may
 *                be NULL.
 * err            device uint32 or NULL.  MTV_DEVERR_INDPTR: a decreasing
 *                offset, one past num_q or num_kv, or a request past max_q or
 *                max_kv (its rows are left as they were).  MTV_DEVERR_TIMEOUT:
 *                a bounded wait gave up (rows of that block may be left as they
 *                were, or NaN where its keys are split).
 * Rows of no request are left as they were.  Keys and values that no query of
 * their request sees may hold anything, NaN included; one that some query of a
 * request sees has to be finite for the request's other queries to be right.
 */
int mla_prefill_run(const void* q, int64_t q_tok_stride, int64_t q_head_stride, const void* k_nope,
                    int64_t k_tok_stride, int64_t k_head_stride, const void* k_rope, int64_t k_rope_stride,
                    const void* v, int64_t v_tok_stride, int64_t v_head_stride, const int64_t* qo_indptr,
                    const int32_t* kv_indptr, int bs, int64_t max_q, int64_t max_kv, int64_t num_q, int64_t num_kv,
                    int num_heads, int dtype, float scale, int causal, void* out, int64_t out_tok_stride,
                    int64_t out_head_stride, float* lse, int nsplit, void* workspace, uint64_t workspace_bytes,
                    uint32_t* err, void* stream);

/*
 * mla_norm_rope_write -- mla_rope_write with root-mean-square norms in the
 * same pass: of every token's latent part, and of every query head.
 *
 *   latent:  row[0:512]   = c / sqrt(mean(c^2) + eps) * c_weight
 *            row[512:576] = the key part, turned
 *   query head x of nope_dim + rope_dim values: y = x / sqrt(mean(x^2) + eps) *
 *     q_weight over the whole head; q_nope = its first nope_dim values, q_rope
 *     = its last rope_dim, turned
 * Computed in fp32, rounded once to nearest-even.  Rotation, positions,
 * num_valid, out_cache_loc, kv_pool and err are those of mla_rope_write.
 *
 * eps            finite, >= 0.
 * dtype          MTV_DTYPE_* of the inputs, weights and query outputs.
 * q_in           device, or NULL to leave the queries out: element d <
 *                nope_dim + rope_dim of head h of token t at t * q_tok_stride +
 *                h * q_head_stride + d.
 * nope_dim       0 .. MTV_MAX_NORM_DIM - rope_dim.
 * q_weight       device [nope_dim + rope_dim], or NULL: the heads are not
 *                normalised then, only their last rope_dim values are read
 *                and turned, and q_nope has to be NULL.
 * q_nope         device (NULL with nope_dim = 0), strides as q_in.
 * q_rope         device, strides as q_in.  q_nope may be q_in and q_rope
 *                q_in + nope_dim, with q_in's strides; any other overlap gives
 *                unspecified values.
 * c_weight       device [512], or NULL: the latent part is not normalised.
 */
int mla_norm_rope_write(const uint64_t* turns, int rope_dim, float amplitude, int layout, const int64_t* positions,
                        int64_t num_tokens, const int64_t* num_valid, int dtype, float eps, const void* q_in,
                        int64_t q_tok_stride, int64_t q_head_stride, int num_heads, int nope_dim,
                        const void* q_weight, void* q_nope, int64_t q_nope_tok_stride, int64_t q_nope_head_stride,
                        void* q_rope, int64_t q_rope_tok_stride, int64_t q_rope_head_stride, const void* c_in,
                        int64_t c_tok_stride, const void* c_weight, const void* k_in, int64_t k_tok_stride,
                        const int64_t* out_cache_loc, void* kv_pool, int64_t num_slots, uint32_t* err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_LAYER_OPS_H_ */
