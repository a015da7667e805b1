/*
 * mla_heads.h -- C ABI of the GB300 (sm_103a) operators on ordinary heads,
 * beside the latent ones: norms and rotation of queries and keys, the write of
 * keys and values into a paged cache, causal attention over whole prompts
 * (latent attention before absorption: 128 heads of 192 and 128 values) and
 * attention of new tokens over the pages.  Query heads come in groups: n_q =
 * G * n_kv, and query head h reads key head h / G.
 *
 * Norm of a head x of D values (mean over the D values; all in fp32):
 *   MLA_NORM_RMS    y = x / sqrt(mean(x^2) + eps) * weight
 *   MLA_NORM_LAYER  y = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * weight + bias
 * and the rotation of mla_rope.h follows on [rot_off, rot_off + rot_dim).  The
 * result is rounded to the tensor's type once, behind both.
 *
 * Attention: query token i of the n that a sequence of len keys has sees key p
 * < len, and where `causal` is set p <= len - n + i (the queries are the
 * sequence's newest tokens):
 *   z_p = softmax_scale * (q . k_p),  out = sum_p softmax(z)_p v_p,  lse = ln sum_p exp(z_p)
 * A token that sees nothing, or scores -inf on all that it sees, gets out = 0
 * and lse = -inf.  Keys and values outside a sequence do not matter, nor do
 * table entries of pages behind it, and a NaN or infinity in a key or value
 * reaches only the tokens that see it: a score that is NaN or +inf makes out
 * and lse NaN, a value that is not finite makes its column of out NaN or
 * infinite.
 *
 * A paged cache holds pages of 128 rows: place r of page g of head h is at
 * g * block_stride + r * row_stride + h * head_stride, so pages ordered by
 * token, by head, and keys and values that share a page all work.  Key p of
 * sequence b lies in page block_table[b, p / 128], place p % 128.  A page id
 * outside [0, num_blocks), or a position beyond the table, is masked out and
 * raises MLA_DEVICE_BAD_BLOCK.
 *
 * Numerics: products of 16-bit values are exact and summed in fp32; the softmax
 * runs in fp32 with a running maximum and sum; the weights enter the second
 * product rounded once to the heads' type (at most 2^-8 (bf16) or 2^-11 (fp16)
 * relative each; in fp16 a weight below 2^-21 of the row's largest may be off by
 * 2^-32 of that instead; they are summed unrounded), so an output is off by up
 * to that times sum_p softmax_p |v_p|, and in fp16 by 2^-32 max_p |v_p| for each
 * key at most, on top of its own rounding.  The result of a call
 * does not depend on timing: a repeated call gives the same bits.
 *
 * Conventions are those of mla_sparse.h: device pointers owned by the caller,
 * asynchronous on `stream`, argument errors returned before any launch with
 * mla_heads_last_error() describing them, every device-side wait bounded
 * (mla_sparse_set_wait_limit_ns; a wait that runs out raises
 * MLA_DEVICE_TIMEOUT, and the next launch runs in full).
 */
#ifndef MLA_HEADS_H_
#define MLA_HEADS_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_rope.h"
#include "mla_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status bit beside those of mla_sparse.h: cu_q or cu_k decreases or leaves [0, T]. */
#define MLA_DEVICE_BAD_LENGTH 0x8u

typedef enum mla_norm_kind { MLA_NORM_NONE = 0, MLA_NORM_RMS = 1, MLA_NORM_LAYER = 2 } mla_norm_kind;

/* The norm of a tensor's heads (a host struct; NULL in a call: none). */
typedef struct mla_head_norm {
  const void* weight;  /* [head_dim], or NULL: ones */
  const void* bias;    /* [head_dim], or NULL: zeros (MLA_NORM_LAYER only) */
  int32_t kind;        /* mla_norm_kind */
  int32_t fp32;        /* weight and bias are fp32; 0: of the heads' type */
  float eps;           /* >= 0, finite */
  int32_t reserved;    /* 0 */
} mla_head_norm;

/*
 * mla_norm_rope -- norm and rotate the heads of one or two tensors of the same
 * tokens, in one pass.  dims, params, positions and the tensors are those of
 * mla_rope_apply, with these differences: inverse must be 0; rot_dim 0 rotates
 * nothing (params and positions may then be NULL); in place (out is x, same
 * strides) whole heads are read and written; rows of out must be distinct.
 * Heads of any size, stride and alignment of whole elements work; those of
 * which head, strides and, in the half layout, the rotation's halves are
 * multiples of 16 bytes run in 16-byte accesses.  One launch, two
 * where the tensors need accesses of different kinds.
 */
mla_status mla_norm_rope(const mla_rope_dims* dims, const mla_rope_params* params, const int32_t* positions,
                         const mla_rope_tensor* q, const mla_head_norm* q_norm, const mla_rope_tensor* k,
                         const mla_head_norm* k_norm, void* stream);

/* A pool of pages of one of keys and values; strides in elements, >= 0. */
typedef struct mla_kv_cache {
  void* data;
  int64_t block_stride, row_stride, head_stride;
} mla_kv_cache;

typedef struct mla_append_dims {
  int32_t T;          /* tokens, >= 0 (0: no-op) */
  int32_t n_kv;       /* key and value heads, >= 1 */
  int32_t d_qk, d_v;  /* values of a key head and of a value head, >= 1 */
  int32_t rot_dim;    /* 0 (none), or even, in [2, 256] */
  int32_t rot_off;    /* of the keys */
  int32_t half;       /* 0: interleaved pairs, 1: half layout */
  int32_t dtype;      /* mla_rope_dtype of all tensors */
  int32_t num_blocks; /* pages of both caches, in [1, 2^24) */
} mla_append_dims;

/* The new keys or values: element (t, h, d) at t * token_stride + h * head_stride + d. */
typedef struct mla_append_input {
  const void* x;
  int64_t token_stride, head_stride;
} mla_append_input;

/*
 * mla_kv_append -- write the keys of T tokens, normed and rotated, and their
 * values, as they are, to rows[t] of a paged cache (page rows[t] / 128, place
 * rows[t] % 128; mla_page_plan's cache_index): a negative row is skipped, one
 * at or beyond num_blocks * 128 is skipped and raises MLA_DEVICE_BAD_BLOCK.
 * Rows are expected to be distinct.  q (or NULL) are the tokens' queries,
 * normed and rotated in the same launch to q->out (in place where it is q->x);
 * q->rows must be NULL.  rows int64 [T], positions int32 [T] (may be NULL where
 * rot_dim is 0).  Caches and outputs may have no byte in common with one
 * another or with an input; views that interleave are told apart by their
 * strides.  Of tokens with the same row, the row holds values of one or of
 * several.  One launch, up to three where the tensors need accesses of
 * different kinds (16 bytes, single values of smaller and of larger heads).
 */
mla_status mla_kv_append(const mla_append_dims* dims, const mla_rope_params* params, const int32_t* positions,
                         const int64_t* rows, const mla_append_input* k, const mla_head_norm* k_norm,
                         const mla_kv_cache* k_cache, const mla_append_input* v, const mla_kv_cache* v_cache,
                         const mla_rope_tensor* q, const mla_head_norm* q_norm, void* stream);

/* A tensor of packed heads: element (t, h, d) at t * token_stride + h * head_stride + d. */
typedef struct mla_heads_tensor {
  const void* data;
  int64_t token_stride, head_stride;
} mla_heads_tensor;

typedef struct mla_prompt_dims {
  int32_t B;                  /* sequences, >= 0 (0: no-op) */
  int32_t T;                  /* rows of q, out and lse, >= 0 */
  int32_t Tk;                 /* packed: rows of k and v, >= 0; paged: 0 */
  int32_t n_q, n_kv;          /* heads, n_q a multiple of n_kv, at most 128 to one */
  int32_t d_qk, d_v;          /* multiples of 8, at most 192 and 128 */
  int32_t dtype;              /* MLA_ROPE_BF16 or MLA_ROPE_FP16 */
  int32_t causal;             /* 0 or 1 */
  int32_t num_blocks;         /* paged: pages of the caches, in [1, 2^24); packed: 0 */
  int32_t max_blocks_per_seq; /* paged: block_table row width, in [1, 2^23]; packed: 0 */
} mla_prompt_dims;

/* Bytes of workspace mla_prompt_attn_fwd needs for these dims; 0 for invalid
 * dims.  It needs no initialisation and carries nothing from call to call;
 * calls that may overlap in time need one each.  Some 12 bytes a sequence and,
 * where sequences may have more than 512 keys, room for the parts of items that
 * are cut along their keys, whether or not any is: as many as the dims allow, at
 * most 640 of 1024 * d_v + 2048 bytes (85 MB at d_v = 128), twice that size with
 * d_v above 64 and 4096 rows (T * n_q / n_kv) or more of a key head a sequence. */
size_t mla_prompt_workspace_bytes(const mla_prompt_dims* dims);

/*
 * mla_prompt_attn_fwd -- attention of whole prompts or chunks of them.
 *
 * Sequence b has the query rows [cu_q[b], cu_q[b + 1]).  Its keys are
 *   packed  rows [cu_k[b], cu_k[b + 1]) of k and v (cu_k NULL: those of cu_q), or
 *   paged   the first act_seqs[b] of its pages, with num_blocks > 0.
 * Rows of out and lse outside [cu_q[0], cu_q[B]) stay as they were.  Offsets
 * outside [0, T] ([0, Tk]) are clamped, a sequence that ends before it begins
 * is empty, and either raises MLA_DEVICE_BAD_LENGTH.
 *
 * cu_q, cu_k  int32 [B + 1]; block_table int32 [B, max_blocks_per_seq],
 * act_seqs int32 [B] (negative counts as 0)
 * q, k, v     16-byte aligned, strides multiples of 8 elements; k and v packed
 *             or pools of pages
 * out         dense [T, n_q, d_v], 16-byte aligned; lse fp32 [T, n_q] or NULL
 * workspace   >= mla_prompt_workspace_bytes(dims) bytes, 256-byte aligned
 * out, lse and the workspace may not overlap one another or the inputs
 * (MLA_ERR_UNSUPPORTED).  Two launches on `stream` (the plan of the work, the
 * attention), three where sequences may have more than 512 keys (the join of
 * rows whose keys several SMs shared), capturable into a CUDA graph; the first
 * call on each device sets kernel attributes: make it before any stream capture
 * begins.  T * n_q below 2^31 - 1024, Tk below 2^31 - 257.
 */
mla_status mla_prompt_attn_fwd(const mla_prompt_dims* dims, const mla_heads_tensor* q, const mla_kv_cache* k,
                               const mla_kv_cache* v, const int32_t* cu_q, const int32_t* cu_k,
                               const int32_t* block_table, const int32_t* act_seqs, void* out, float* lse,
                               float softmax_scale, void* workspace, size_t workspace_bytes, void* stream);

typedef struct mla_paged_dims {
  int32_t B;                  /* sequences, >= 0 (0: no-op) */
  int32_t S1;                 /* query rows of a sequence, >= 1 */
  int32_t n_q, n_kv;          /* heads, n_q a multiple of n_kv, at most 128 to one */
  int32_t d_qk, d_v;          /* multiples of 8, at most 192 and 128 */
  int32_t dtype;              /* MLA_ROPE_BF16 or MLA_ROPE_FP16 */
  int32_t num_blocks;         /* pages of the caches, in [1, 2^24) */
  int32_t max_blocks_per_seq; /* block_table row width, in [1, 2^23] */
} mla_paged_dims;

/* As mla_prompt_workspace_bytes; up to 64 rows (S1 * n_q / n_kv) of a key head
 * at most 20 MB (5 MB for 4 rows at d_v = 128), with more what prompts need. */
size_t mla_paged_workspace_bytes(const mla_paged_dims* dims);

/*
 * mla_paged_attn_fwd -- attention of each sequence's newest tokens (one, or a
 * chain of S1) over its pages.  Row b * S1 + s of q, out and lse is token s of
 * sequence b; q_lens int32 [B] (NULL: S1 each; negative counts as 0, more than
 * S1 as S1) are the tokens that there are, the rows behind them get out = 0 and
 * lse = -inf.  act_seqs counts the new tokens too.  Tensors, workspace,
 * overlaps and the first call as mla_prompt_attn_fwd; B * S1 * n_q below 2^31 -
 * 1024.  Up to 64 rows (S1 * n_q / n_kv) of a key head: two launches (the
 * attention, the join of heads that several SMs shared); more go through the
 * kernels of prompts.
 */
mla_status mla_paged_attn_fwd(const mla_paged_dims* dims, const mla_heads_tensor* q, const mla_kv_cache* k,
                              const mla_kv_cache* v, const int32_t* block_table, const int32_t* act_seqs,
                              const int32_t* q_lens, void* out, float* lse, float softmax_scale, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Description of the last error of a call of this header on this thread. */
const char* mla_heads_last_error(void);

/* Synchronises `stream`, returns these calls' sticky device status bits
 * (MLA_DEVICE_BAD_BLOCK, MLA_DEVICE_BAD_LENGTH, MLA_DEVICE_TIMEOUT) and clears
 * them when `clear` is nonzero; MLA_ERR_DEVICE_STATUS when any bit is set. */
mla_status mla_heads_device_status(void* stream, uint32_t* flags, int32_t clear);

#ifdef __cplusplus
}
#endif
#endif /* MLA_HEADS_H_ */
