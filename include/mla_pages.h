/*
 * mla_pages.h -- C ABI of the GB300 (sm_103a) page plan: block tables, slot
 * maps and positions of one step, built on the GPU from request lengths.
 *
 * The attention calls (mla_sparse.h, mla_tree.h), the indexer, the cache
 * writer and the prolog read their pages through block_table, act_seqs and
 * cache_index; this call makes them for a step in which sequence b holds
 * ctx_b cached positions and adds new_b tokens:
 *
 *   act_b        = ctx_b + new_b
 *   have_b       = ceil(ctx_b / 128), need_b = ceil(act_b / 128) - have_b
 *   block_table[b, have_b + k] = free_blocks[sum_{a < b} need_a + k], k < need_b
 *   new token i of sequence b sits in slot ctx_b + i:
 *   cache_index  = block_table[b, slot / 128] * 128 + slot % 128
 *   position     = ctx_b + i, or with a tree of drafted tokens ctx_b + its
 *                  depth (the number of its drafted ancestors)
 *   tree_mask    bit j: token j is i itself or an ancestor of i
 *
 * The first sum need_b entries of free_blocks are taken, in order of
 * sequence and of block; the other entries of block_table stay as they were.
 * A call on the same inputs gives the same outputs.
 *
 * Two layouts of the new tokens:
 *   padded  S1 >= 1: token i of sequence b is row b * S1 + i, T = B * S1, and
 *           rows i >= new_b are padding (new_b above S1 counts as S1);
 *   packed  S1 = 0: the tokens of all sequences follow one another, T is the
 *           capacity, and rows behind the last token are padding.
 * Padding rows get cache_index -1 (which the cache writer and the prolog
 * skip), seq_ids -1, position 0 and an empty mask.
 *
 * Problems found on the device never fault.  A token without a page (the
 * free list is used up, the table is too narrow, the capacity T is too small)
 * gets cache_index -1, a missing table entry -1, and MLA_DEVICE_NO_PAGE is
 * raised; a block id outside [0, num_blocks) gives cache_index -1 and
 * MLA_DEVICE_BAD_BLOCK.  Negative lengths count as 0.
 *
 * Conventions are those of mla_sparse.h: device pointers owned by the caller,
 * asynchronous on `stream` (one launch, nothing allocated), argument errors
 * returned before any launch with mla_page_last_error() describing them.
 * Outputs may not overlap inputs (act_seqs is not ctx_lens) or one another:
 * MLA_ERR_UNSUPPORTED.
 */
#ifndef MLA_PAGES_H_
#define MLA_PAGES_H_

#include <stdint.h>

#include "mla_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status bit beside those of mla_sparse.h: no page for a token. */
#define MLA_DEVICE_NO_PAGE 0x4u

typedef struct mla_page_dims {
  int32_t B;                  /* sequences, >= 0 (0: no-op) */
  int32_t S1;                 /* padded: rows per sequence, >= 1; packed: 0 */
  int32_t T;                  /* rows of the per-token outputs (padded: B * S1) */
  int32_t block_size;         /* 128 */
  int32_t num_blocks;         /* physical blocks of the cache, in [1, 2^24) */
  int32_t max_blocks_per_seq; /* block_table row width W >= 1 */
  int32_t num_free;           /* entries of free_blocks, >= 0 */
} mla_page_dims;

typedef struct mla_page_io {
  const int32_t* ctx_lens;    /* [B] cached positions before the step */
  const int32_t* new_lens;    /* [B], or NULL: S1 each (padded only) */
  const int32_t* free_blocks; /* [num_free] ids of free blocks (NULL when num_free is 0) */
  const int32_t* parents;     /* [B, S1] or NULL (padded only): the drafted parent of each token; a value
                                 outside [0, i) for token i: it follows the cached context directly */
  int32_t* block_table;       /* [B, W], updated in place */
  int32_t* act_seqs;          /* [B] output */
  int64_t* cache_index;       /* [T] output */
  int32_t* positions;         /* [T] output or NULL */
  int32_t* seq_ids;           /* [T] output or NULL: the token's sequence */
  int32_t* cu_seqs;           /* [B + 1] output or NULL: running sums of new_b */
  uint64_t* tree_mask;        /* [T, ceil(S1 / 64)] output or NULL (padded only; without parents: a chain) */
  int32_t* num_taken;         /* [1] output or NULL: sum need_b, at most num_free */
} mla_page_io;

mla_status mla_page_plan(const mla_page_dims* dims, const mla_page_io* io, void* stream);

/* Description of the last error of an mla_page_* call on this thread. */
const char* mla_page_last_error(void);

/* Synchronises `stream`, returns the plan's sticky device status bits
 * (MLA_DEVICE_NO_PAGE, MLA_DEVICE_BAD_BLOCK) and clears them when `clear` is
 * nonzero; MLA_ERR_DEVICE_STATUS when any bit is set. */
mla_status mla_page_device_status(void* stream, uint32_t* flags, int32_t clear);

#ifdef __cplusplus
}
#endif
#endif /* MLA_PAGES_H_ */
