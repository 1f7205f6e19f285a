/*
 * mla_step_ops.h -- C ABI of what a serving step needs before and after MLA
 * tree-verify attention on GB300 (sm_103a): the page tables and slot maps of
 * its paged latent pool built from request lengths, the rotary positions of
 * the queries together with the write of new latent rows into the pool, and
 * the log probabilities, entropy and top tokens of the target's logits.
 *
 *   lengths -> mla_page_table_update -> mla_slot_map_build -> mla_rope_write
 *     -> mla_tree_mask_build -> mla_tree_verify_run -> (rest of the model)
 *     -> mla_token_logprobs -> mla_tree_accept -> mla_page_table_update
 *
 * Conventions (as in mla_tree_verify.h): every pointer named "device" is a
 * CUDA device pointer; buffers are caller-owned; nothing allocates or
 * synchronises, so every call may be captured in a CUDA graph; no call keeps
 * state of its own, so calls on different buffers may overlap on different
 * streams and come from different host threads; the return value is MTV_OK (0)
 * or a negative MTV_E* code.  Nothing is launched then, with one exception:
 * MTV_E_CUDA of a call that takes two kernels, when the first was launched and
 * the second refused.  mla_page_table_update of more than 16,384 entries has
 * then moved pages without writing held and num_free, so that its buffers no
 * longer describe each other; mla_token_logprobs with token_rows has written
 * everything but logprobs.  `err` (device, may be NULL) is a sticky 32-bit word
 * the kernels OR MTV_DEVERR_* bits into; data-dependent problems never trap.
 */
#ifndef MLA_STEP_OPS_H_
#define MLA_STEP_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_tree_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A page table entry outside [0, num_pages), a row that needs more pages than
 * it may hold or than are free, or a free list that is not one. */
#define MTV_DEVERR_PAGES 0x20
/* A token or row index outside its range. */
#define MTV_DEVERR_TOKEN 0x40
/* A row of logits with a NaN or +inf, or with an unusable temperature. */
#define MTV_DEVERR_LOGITS 0x80

/* Most requests of one mla_slot_map_build and rows of one
 * mla_page_table_update (their offsets are kept in shared memory). */
#define MTV_MAX_REQUESTS 8192
/* Longest head part that mla_rope_write turns. */
#define MTV_MAX_ROPE_DIM 256
/* Most alternatives of one mla_token_logprobs, and its largest vocabulary. */
#define MTV_MAX_TOP 32
#define MTV_MAX_VOCAB (1 << 20)

/* ------------------------------------------------------------ data types */
#define MTV_DTYPE_BF16 0
#define MTV_DTYPE_FP16 1
#define MTV_DTYPE_FP32 2

/*
 * mla_page_table_update -- grow or shrink every row of a page table to the
 * tokens it has to hold, from and to a stack of free pages.
 *
 * need_r = ceil(lens[r] / page_size).  Rows with need_r < held[r] release the
 * entries [need_r, held[r]), rows with need_r > held[r] get new entries.
 * Releases come first: released pages are pushed in descending order of (row,
 * entry), so that the first row's first released page ends on top; new pages
 * are popped in ascending order of (row, entry).  Growing rows and releasing
 * the same entries again therefore restores the stack.
 *
 * lens           device, int32 [num_rows]: tokens row r has to hold from now
 *                on (0 releases the row), -1 to leave the row as it is.
 * num_rows       host, 0 .. MTV_MAX_REQUESTS.
 * page_size      host, tokens a page, >= 1.
 * page_table     device, int32, row r at page_table + r * table_stride; its
 *                first held[r] entries are its pages.  Entries past them are
 *                neither read nor cleared.
 * table_stride   host, elements from row to row, >= max_pages.
 * max_pages      host, entries a row may hold; num_rows * max_pages < 2^31.
 * held           device, int32 [num_rows], in and out.
 * free_pages     device, int32 [free_capacity], in and out: the stack,
 *                free_pages[num_free - 1] is its top.
 * num_free       device, int32 [1], in and out.
 * err            device uint32 or NULL.  MTV_DEVERR_PAGES: lens[r] needs more
 *                than max_pages, held[r] is outside [0, max_pages], the free
 *                pages do not suffice (the first row that does not fit and
 *                every later row that would grow), or num_free is outside
 *                [0, free_capacity] (nothing is done then) or would pass
 *                free_capacity (pages past it are lost).  MTV_DEVERR_INDPTR:
 *                lens[r] < -1.  A flagged row is left as it is.
 *
 * A page belongs to one row.  The updates in place need no memory besides these
 * buffers; two calls on the same buffers have to be ordered by the caller.
 */
int mla_page_table_update(const int32_t* lens, int num_rows, int page_size, int32_t* page_table,
                          int64_t table_stride, int64_t max_pages, int32_t* held, int32_t* free_pages,
                          int64_t free_capacity, int32_t* num_free, uint32_t* err, void* stream);

/*
 * mla_slot_map_build -- the index buffers of one verify step from request
 * lengths and a page table: what mla_tree_mask_build, mla_tree_verify_run,
 * mla_tree_accept and mla_rope_write read.
 *
 * With p_r = prefix_lens[r], n_r = tree_sizes[r], and the slot of token j of
 * request r, slot(r, j) = page_table[rows[r]][j / page_size] * page_size +
 * j % page_size:
 *   kv_indptr[r + 1] = sum of p up to r,  qo_indptr[r + 1] = sum of n up to r
 *   kv_indices[kv_indptr[r] + j]    = slot(r, j)              j < p_r
 *   out_cache_loc[qo_indptr[r] + t] = slot(r, p_r + t)        t < n_r
 *   positions[qo_indptr[r] + t]     = p_r + number of t's ancestors
 *
 * page_table     device, int32, row i at page_table + i * table_stride,
 *                max_pages entries readable in each of its num_rows rows.
 * num_pages      pages of the pool: entries are checked against it.
 * page_size      host, >= 1.
 * rows           device, int32 [bs]: the table row of request r, or NULL when
 *                request r is row r.  Requests may share a row.
 * prefix_lens    device, int32 [bs].
 * tree_sizes     device, int32 [bs], or NULL when there are no tree tokens.
 * parents        device, int32 [q_capacity] (as in mla_tree_mask_build), or
 *                NULL when every tree is a chain.
 * bs             host, 0 .. MTV_MAX_REQUESTS.
 * kv_indptr      device, int32 [bs + 1] output.
 * kv_indices     device, int64 [kv_capacity] output, or NULL to leave it out.
 * qo_indptr      device, int64 [bs + 1] output.
 * out_cache_loc  device, int64 [q_capacity] output, or NULL to leave it out.
 * positions      device, int64 [q_capacity] output, or NULL to leave it out.
 * err            device uint32 or NULL.  MTV_DEVERR_INDPTR: a negative length
 *                (taken as 0), sums past 2^31 - 1 (the offsets are held there;
 *                slots and positions go by the request's own length) or past a
 *                capacity (the offsets are published, nothing is written past
 *                the capacity: mla_tree_verify_run skips such a request).
 *                MTV_DEVERR_PAGES: a token past its row's max_pages, a row
 *                outside [0, num_rows) or an entry outside [0, num_pages): the
 *                slot is then -1, which mla_tree_verify_run masks.
 *                MTV_DEVERR_PARENT: a parent outside [-1, t - 1] (taken as -1).
 * Elements behind the last request's are left as they were.
 */
int mla_slot_map_build(const int32_t* page_table, int64_t table_stride, int64_t num_rows, int64_t max_pages,
                       int64_t num_pages, int page_size, const int32_t* rows, const int32_t* prefix_lens,
                       const int32_t* tree_sizes, const int32_t* parents, int bs, int32_t* kv_indptr,
                       int64_t* kv_indices, int64_t kv_capacity, int64_t* qo_indptr, int64_t* out_cache_loc,
                       int64_t* positions, int64_t q_capacity, uint32_t* err, void* stream);

/* ------------------------------------------------------- rotary positions */
/* Pairs (x[2i], x[2i+1]).                                                   */
#define MTV_ROPE_INTERLEAVED 0
/* Pairs (x[i], x[i + rope_dim/2]).                                          */
#define MTV_ROPE_HALF 1

/* Scaling of the frequencies base^(-2i/rope_dim) for contexts longer than
 * original_len.                                                             */
#define MTV_ROPE_SCALE_NONE 0
/* f / factor (position interpolation).                                      */
#define MTV_ROPE_SCALE_LINEAR 1
/* YaRN (Peng et al. 2023, "NTK-by-parts" and attention scaling): pairs that
 * turn more than beta_fast times in original_len keep f, those that turn less
 * than beta_slow times get f / factor, a linear ramp over the pair index in
 * between; amplitude 0.1 ln(factor) + 1 unless given.                       */
#define MTV_ROPE_SCALE_YARN 2
/* By wavelength: pairs that turn more than high_turns times in original_len
 * keep f, less than low_turns get f / factor, and in between f and f / factor
 * are blended linearly in the number of turns.                              */
#define MTV_ROPE_SCALE_WAVELENGTH 3

typedef struct mtv_rope_scaling {
  int32_t kind;        /* MTV_ROPE_SCALE_*                                    */
  int32_t reserved;    /* 0                                                   */
  double factor;       /* >= 1                                                */
  double original_len; /* > 0 (YARN, WAVELENGTH)                              */
  double beta_fast, beta_slow;   /* YARN: beta_fast > beta_slow > 0           */
  double low_turns, high_turns;  /* WAVELENGTH: high_turns > low_turns > 0    */
  double amplitude;    /* factor on the rotated values; 0 = the kind's own    */
} mtv_rope_scaling_t;

/*
 * mla_rope_freqs -- the frequency table of mla_rope_write, on the host.
 *
 * turns[i] is pair i's angle per position as a 64-bit fraction of a full turn,
 * f_i / (2 pi) * 2^64: position * turns[i] modulo 2^64 is the angle with its
 * whole turns gone, so far positions lose nothing.
 *
 * rope_dim       even, 2 .. MTV_MAX_ROPE_DIM.
 * base           > 1.
 * scaling        NULL for MTV_ROPE_SCALE_NONE.
 * turns          host, uint64 [rope_dim / 2] output: copy it to the device.
 * amplitude      host output, for mla_rope_write.
 */
int mla_rope_freqs(int rope_dim, double base, const mtv_rope_scaling_t* scaling, uint64_t* turns,
                   float* amplitude);

/*
 * mla_rope_write -- turn the rotary part of every query head, and write every
 * token's latent row (latent part as it is, key part turned) into the pool.
 *
 * For token t at position P_t, pair i and angle a = 2 pi frac(P_t turns[i]):
 *   y1 = amplitude (x1 cos a - x2 sin a)
 *   y2 = amplitude (x1 sin a + x2 cos a)
 * (with `inverse`, -a in place of a: the transposed map.)  Computed in fp32,
 * rounded once to nearest-even.
 *
 * turns          device, uint64 [rope_dim / 2].
 * rope_dim       even, 2 .. MTV_MAX_ROPE_DIM; 64 when kv_pool is given.
 * amplitude      finite.
 * layout         MTV_ROPE_INTERLEAVED or MTV_ROPE_HALF.
 * inverse        0 or 1.
 * positions      device, int64 [num_tokens].
 * num_tokens     host: rows of the buffers.
 * num_valid      device, int64 [1], or NULL: only tokens below it are done
 *                (a padded batch: pass qo_indptr + bs).  The others' inputs may
 *                be read, but nothing of theirs is written.
 * dtype          MTV_DTYPE_* of q_in, q_out, k_in and c_in.
 * q_in, q_out    device, or both NULL to leave the queries out; element d < rope_dim of head h
 *                of token t at t * tok_stride + h * head_stride + d (strides in
 *                elements): the rotary part of a head, e.g. q + 512 with
 *                strides 64 * 576 and 576.  q_out may be q_in with the same
 *                strides; any other overlap gives unspecified values.
 * k_in           device: key part, element d of token t at t * k_tok_stride + d.
 * c_in           device: latent part [512], at t * c_tok_stride.
 * out_cache_loc  device, int64 [num_tokens]: the pool row of each token.  Rows
 *                of one call have to be distinct (else which token's values
 *                they hold is unspecified).
 * kv_pool        device, bf16 [num_slots, 576], 16-byte aligned, or NULL to
 *                leave the pool out (k_in, c_in, out_cache_loc too).
 * err            device uint32 or NULL: MTV_DEVERR_SLOT_RANGE for a slot
 *                outside [0, num_slots) (that row is not written).
 */
int mla_rope_write(const uint64_t* turns, int rope_dim, float amplitude, int layout, int inverse,
                   const int64_t* positions, int64_t num_tokens, const int64_t* num_valid, int dtype,
                   const void* q_in, int64_t q_in_tok_stride, int64_t q_in_head_stride, void* q_out,
                   int64_t q_out_tok_stride, int64_t q_out_head_stride, int num_heads, const void* k_in,
                   int64_t k_tok_stride, const void* c_in, int64_t c_tok_stride, const int64_t* out_cache_loc,
                   void* kv_pool, int64_t num_slots, uint32_t* err, void* stream);

/*
 * mla_token_logprobs -- log probabilities of given tokens, entropy and top
 * alternatives of rows of logits, each logit read once.
 *
 * With z = logits[r] * inv_temperature[r], m = max z rounded to fp32 and S =
 * sum exp(z - m), each z - m one fused multiply-add:
 *   stats[0][r] = m,  stats[1][r] = ln S        (the row's ln sum exp z is their sum)
 *   stats[2][r] = ln S - sum exp(z - m) (z - m) / S           (entropy, nats)
 *   logprobs[i] = (z[tokens[i]] - m) - ln S     of row token_rows[i]
 *   top_tokens[k][r], top_logprobs[k][r]        the k-th largest logit of row
 *     r, equal logits in the order of their ids.
 * top_tokens[0] is contiguous [num_rows]: the target_tokens of mla_tree_accept.
 *
 * logits         device, [num_rows, vocab] of dtype, row r at r * row_stride
 *                elements (>= 0; no alignment beyond the element's).  -inf is
 *                a probability of 0.
 * dtype          MTV_DTYPE_*.
 * vocab          1 .. MTV_MAX_VOCAB.
 * inv_temperature  device, fp32 [num_rows] (positive, finite), or NULL for 1.
 * tokens         device, int32 [num_tokens], or NULL with num_tokens == 0; -1
 *                gives a log probability of 0 (padding of a sum).
 * token_rows     device, int32 [num_tokens]: the row that scores token i (a
 *                tree node's parent row), or NULL when token i is scored by
 *                row i (num_tokens <= num_rows then).
 * logprobs       device, fp32 [num_tokens] output.
 * stats          device, fp32 [3, num_rows] output.
 * top_k          0 .. MTV_MAX_TOP (may exceed vocab).
 * top_tokens, top_logprobs  device, int32 / fp32 [top_k, num_rows] outputs
 *                (may be NULL with top_k == 0); -1 and -inf where a row has
 *                no further logit above -inf.
 * err            device uint32 or NULL.  MTV_DEVERR_LOGITS: a row with a NaN
 *                or +inf logit, an unusable temperature or a largest z past
 *                fp32's range: its stats, its
 *                tokens' logprobs and its top_logprobs are NaN, its top_tokens
 *                -1.  MTV_DEVERR_TOKEN: a token outside [-1, vocab) or a row
 *                outside [0, num_rows): its logprob is NaN.
 * A row whose logits are all -inf has stats (-inf, -inf, 0), log probabilities
 * -inf, and no top tokens.
 */
int mla_token_logprobs(const void* logits, int dtype, int64_t num_rows, int vocab, int64_t row_stride,
                       const float* inv_temperature, const int32_t* tokens, const int32_t* token_rows,
                       int64_t num_tokens, float* logprobs, float* stats, int top_k, int32_t* top_tokens,
                       float* top_logprobs, uint32_t* err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_STEP_OPS_H_ */
