/*
 * mla_rope.h -- C ABI of the GB300 (sm_103a) rotary positions: the cosines
 * and sines that the prolog reads (mla_prolog.h), and the rotation itself
 * applied to heads in place or on their way to a paged cache (the Lightning
 * Indexer's queries and index keys, mla_indexer.h).
 *
 * Pair i of the rot_dim rotated values (i < rot_dim / 2) of a token at
 * position p turns by the angle a = p * f_i:
 *
 *   f_i = theta^(-2 i / rot_dim)                                 MLA_ROPE_NONE
 *   f_i / factor                                                 MLA_ROPE_LINEAR
 *   (theta * factor^(rot_dim / (rot_dim - 2)))^(-2 i / rot_dim)  MLA_ROPE_NTK
 *     (rot_dim 2: the exponent's divisor counts as 1)
 *   f_i (1 - r_i) + f_i / factor r_i                             MLA_ROPE_YARN
 *     r_i = clamp((i - low) / max(high - low, 0.001), 0, 1),
 *     low = max(floor(d(beta_fast)), 0), high = min(ceil(d(beta_slow)), rot_dim - 1),
 *     d(beta) = rot_dim ln(orig_positions / (2 pi beta)) / (2 ln theta)
 *     ("YaRN: Efficient Context Window Extension of Large Language Models":
 *     pairs that turn often within the trained length keep their angle,
 *     those that turn rarely are stretched)
 *
 *   y_a = mscale (x_a cos a - x_b sin a),  y_b = mscale (x_a sin a + x_b cos a)
 *
 * with the pair (x_a, x_b) at offsets (2 i, 2 i + 1) of the rotated part
 * (interleaved) or (i, i + rot_dim / 2) (half).  `inverse` turns by -a, which
 * is also the gradient of the forward call.  Values outside
 * [rot_off, rot_off + rot_dim) are copied.
 *
 * Numerics: frequencies are computed in fp64 on the host; position times
 * frequency is taken modulo whole turns in 64-bit fixed point, so an angle is
 * off by at most |p| 2^-48 turns; cos, sin and the rotation are fp32; one
 * rounding to the tensor's type at the end.
 *
 * Conventions are those of mla_sparse.h: device pointers owned by the caller,
 * asynchronous on `stream` (one launch per call, two where only one of two
 * tensors has 16-byte aligned rows; nothing allocated), argument
 * errors returned before any launch with mla_rope_last_error() describing
 * them.
 */
#ifndef MLA_ROPE_H_
#define MLA_ROPE_H_

#include <stdint.h>

#include "mla_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mla_rope_scaling {
  MLA_ROPE_NONE = 0,
  MLA_ROPE_LINEAR = 1,
  MLA_ROPE_NTK = 2,
  MLA_ROPE_YARN = 3
} mla_rope_scaling;

typedef enum mla_rope_dtype { MLA_ROPE_BF16 = 0, MLA_ROPE_FP16 = 1, MLA_ROPE_FP32 = 2 } mla_rope_dtype;

/* The frequency scheme (a host struct). */
typedef struct mla_rope_params {
  double theta;           /* base, > 1 */
  double factor;          /* context extension, >= 1 (ignored by MLA_ROPE_NONE) */
  double orig_positions;  /* trained length (YARN), >= 1 */
  double beta_fast;       /* turns within it above which a pair keeps its angle (YARN), > 0 */
  double beta_slow;       /* turns below which it is stretched in full (YARN), in (0, beta_fast] */
  double mscale;          /* magnitude on cosine and sine, > 0 and finite in fp32 */
  int32_t scaling;        /* mla_rope_scaling */
} mla_rope_params;

/*
 * mla_rope_table -- cos and sin, fp32 [T, rot_dim / 2] (the prolog's inputs
 * for rot_dim 64), times mscale, for positions int32 [T].  rot_dim even, in
 * [2, 256]; T = 0 is a no-op.  The three may not overlap (MLA_ERR_UNSUPPORTED).
 */
mla_status mla_rope_table(const mla_rope_params* params, int32_t T, int32_t rot_dim, const int32_t* positions,
                          float* cos, float* sin, void* stream);

/* One tensor of mla_rope_apply: element (t, h, d) at t * token_stride + h *
 * head_stride + d.  out may be x with the same strides (in place; the rotated
 * part alone is read and written); otherwise no output may have a byte in common
 * with what the call reads or with the other output (MLA_ERR_UNSUPPORTED).
 * Views that interleave, such as the queries and keys of one fused tensor, are
 * told apart by their strides.  With `rows`, token t is written to row rows[t]
 * of out instead of row t: a negative row is skipped, one at or beyond num_rows
 * is skipped and raises MLA_DEVICE_BAD_BLOCK (as the cache writer does); rows
 * are expected to be distinct. */
typedef struct mla_rope_tensor {
  const void* x;
  void* out;
  int64_t x_token_stride, x_head_stride;     /* elements, >= 0 */
  int64_t out_token_stride, out_head_stride; /* elements; with `rows` the token stride is a row's */
  const int64_t* rows;                       /* [T] or NULL */
  int64_t num_rows;                          /* rows of out (with `rows`) */
  int32_t n_heads;                           /* >= 1 */
  int32_t head_dim;                          /* >= rot_off + rot_dim */
  int32_t rot_off;                           /* >= 0 */
  int32_t reserved;                          /* 0 */
} mla_rope_tensor;

typedef struct mla_rope_dims {
  int32_t T;        /* tokens, >= 0 (0: no-op) */
  int32_t rot_dim;  /* even, in [2, 256] */
  int32_t half;     /* 0: interleaved pairs, 1: half layout */
  int32_t inverse;  /* 0 or 1 */
  int32_t dtype;    /* mla_rope_dtype of both tensors */
} mla_rope_dims;

/*
 * mla_rope_apply -- rotate the heads of one or two tensors (queries, and keys
 * or NULL) of the same tokens.  positions int32 [T].  Any strides and
 * alignments of whole elements work; a tensor whose pointers, strides, head
 * size and rotated part are multiples of 16 bytes (the halves of the part in the
 * half layout) runs in 16-byte accesses, whatever the other one is.
 */
mla_status mla_rope_apply(const mla_rope_dims* dims, const mla_rope_params* params, const int32_t* positions,
                          const mla_rope_tensor* q, const mla_rope_tensor* k, void* stream);

/* Description of the last error of an mla_rope_* call on this thread. */
const char* mla_rope_last_error(void);

/* Synchronises `stream`, returns the rotation's sticky device status bits
 * (MLA_DEVICE_BAD_BLOCK) and clears them when `clear` is nonzero;
 * MLA_ERR_DEVICE_STATUS when any bit is set. */
mla_status mla_rope_device_status(void* stream, uint32_t* flags, int32_t clear);

#ifdef __cplusplus
}
#endif
#endif /* MLA_ROPE_H_ */
