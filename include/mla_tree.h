/*
 * mla_tree.h -- C ABI of the GB300 (sm_103a) dense MLA attention over a whole
 * paged cache, for single tokens, chains and trees of drafted tokens.
 *
 * The cache is the one of mla_sparse.h (512-wide latent rows, bf16 or INT8
 * with one fp32 scale per 128 values, and 64-wide bf16 rope rows, shared by
 * all query heads, in pages of 128 rows).  Sequence b has act_b cached
 * positions; its newest n_b (tree_lens[b], at most S1; S1 without tree_lens)
 * are the drafted tokens, already written to the cache: drafted token j sits
 * at position c_b + j, c_b = act_b - n_b.  Token (b, s), s < n_b, sees
 *
 *   every position p with 0 <= p < c_b and p < act_b, and
 *   the drafted tokens j < n_b with bit j of its tree_mask row set (position
 *   c_b + j >= 0); without a tree_mask the tokens j <= s (a chain: causal
 *   attention of the sequence's newest tokens).
 *
 *   z_p  = softmax_scale * (q_nope[t, h, :] . kv_nope[r_p, :] + q_rope[t, h, :] . kv_rope[r_p, :])
 *   out  = sum_p softmax(z)_p kv_nope[r_p, :],   lse = ln sum_p exp(z_p)
 *   r_p  = block_table[b, p / 128] * 128 + p % 128
 *
 * A token that sees nothing, or scores -inf on all that it sees, and padding
 * tokens s >= n_b get out = 0 and lse = -inf.  What lies in rows at and beyond
 * act_b does not matter, nor do table entries of pages beyond it, and a NaN or
 * infinity in a row reaches only the tokens that see it.  Those get what the
 * formulas give: a score that is NaN or +inf makes out and lse NaN, and an
 * infinite value whose score is -inf (weight 0) makes its column of out NaN.
 * A block id outside [0, num_blocks), or a position beyond the table, is
 * masked out and raises MLA_DEVICE_BAD_BLOCK.  Negative act_b and tree_lens
 * count as 0.
 *
 * Numerics: products of bf16 values are exact and summed in fp32; INT8 rows
 * are bf16(fp32(code) * scale), as in mla_sparse.h; the softmax runs in fp32
 * with a running maximum and sum.  The weights enter the second product
 * rounded to bf16 once (at most 2^-8 relative each, as one rounding of a bf16
 * result costs; they are summed for l and lse unrounded), so an output is off by
 * up to 2^-8 sum_p softmax_p |kv_nope_p| on top of its own rounding:
 * mla_sparse_attn_fwd, which keeps 16 bits of a weight, holds a tighter bound.
 * out is rounded to bf16 once.  The result of a call does not depend on timing: a repeated call
 * gives the same bits.
 *
 * Conventions are those of mla_sparse.h: device pointers owned by the caller,
 * asynchronous on `stream`, argument errors returned before any launch with
 * mla_tree_last_error() describing them, every device-side wait bounded
 * (mla_sparse_set_wait_limit_ns; a wait that runs out raises
 * MLA_DEVICE_TIMEOUT, and the next launch runs in full).
 */
#ifndef MLA_TREE_H_
#define MLA_TREE_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace mla_tree_attn_fwd needs for these dims on any device;
 * 0 for invalid dims.  The workspace needs no initialisation and carries
 * nothing from call to call; calls that may overlap in time (other streams,
 * graphs replayed side by side) need one each. */
size_t mla_tree_workspace_bytes(const mla_dims* dims);

/*
 * dims        as mla_sparse_attn_fwd (n_kv 1, d_nope 512, d_rope 64, block_size
 *             128, n_q <= 128); S1 <= 2^20, max_blocks_per_seq <= 2^23, B * S1 *
 *             n_q < 2^31 - 256; topk is ignored
 * q_nope      bf16 [B*S1, n_q, 512], q_rope bf16 [B*S1, n_q, 64]
 * kv_nope     bf16 | int8 [num_blocks*128, 512], kv_rope bf16 [num_blocks*128, 64]
 * kv_scales   fp32 [num_blocks*128, 4] for MLA_KV_INT8, else NULL
 * block_table int32 [B, max_blocks_per_seq], act_seqs int32 [B]
 * tree_lens   int32 [B] or NULL
 * tree_mask   uint64 [B*S1, ceil(S1 / 64)] or NULL; bits at and beyond n_b are ignored
 * out         bf16 [B*S1, n_q, 512], lse fp32 [B*S1, n_q] or NULL
 * workspace   >= mla_tree_workspace_bytes(dims) bytes, 256-byte aligned
 * q, kv, out and scales 16-byte aligned, tree_mask 8-byte, the rest 4-byte;
 * out, lse and the workspace may not overlap one another or the inputs
 * (MLA_ERR_UNSUPPORTED).
 * Up to three launches on `stream` (INT8 rows of calls with three or more
 * blocks of 128 (token, head) rows a sequence are turned into bf16 in the
 * workspace first, if that takes no more than 4 GB; the attention; the merge of
 * rows whose keys several clusters shared), capturable into a CUDA graph.  The
 * expanded rows take 128 KB of workspace for every block of the pool, whether
 * the call uses it or not; above 32,768 blocks the attention converts the rows
 * itself, which takes 1.15 to 1.9 times as long.  Every row block goes through all
 * key tiles of its sequence: right for drafts, up to twice the work of a causal
 * kernel for a prompt.  The first call on each
 * device sets the kernels' shared-memory attribute and looks up the driver's
 * tensor-map encoder: make it before any stream capture begins.
 */
mla_status mla_tree_attn_fwd(const mla_dims* dims, const void* q_nope, const void* q_rope, const void* kv_nope,
                             const void* kv_rope, const float* kv_scales, const int32_t* block_table,
                             const int32_t* act_seqs, const int32_t* tree_lens, const uint64_t* tree_mask, void* out,
                             float* lse, float softmax_scale, void* workspace, size_t workspace_bytes, void* stream);

/* Description of the last error of an mla_tree_* call on this thread. */
const char* mla_tree_last_error(void);

/* Synchronises `stream`, returns the call's sticky device status bits
 * (MLA_DEVICE_BAD_BLOCK, MLA_DEVICE_TIMEOUT) and clears them when `clear` is
 * nonzero; MLA_ERR_DEVICE_STATUS when any bit is set. */
mla_status mla_tree_device_status(void* stream, uint32_t* flags, int32_t clear);

#ifdef __cplusplus
}
#endif
#endif /* MLA_TREE_H_ */
