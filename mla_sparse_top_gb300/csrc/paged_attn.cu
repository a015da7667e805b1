// Attention of new tokens over a paged cache of keys and values for GB300
// (sm_103a); formulas in mla_heads.h.
#include <cuda_runtime.h>

#include "heads.h"

namespace mlaheads {

__device__ unsigned int g_paged_status = 0;

cudaError_t paged_status(unsigned int* v, bool clear) { return read_status(g_paged_status, v, clear); }

namespace {

mla_status check_dims(const mla_paged_dims& d) {
  const mla_status st = check_head_dims(d.n_q, d.n_kv, d.d_qk, d.d_v, d.dtype);
  if (st != MLA_OK) return st;
  if (d.B < 0 || d.S1 < 1 || d.S1 > (1 << 20)) return fail(MLA_ERR_SHAPE, "B must be >= 0, S1 in [1, 2^20]");
  if (static_cast<int64_t>(d.B) * d.S1 * d.n_q >= (1ll << 31) - 256 || d.B > (1 << 24))
    return fail(MLA_ERR_SHAPE, "B * S1 * n_q must be below 2^31 - 256, B at most 2^24");
  if (d.num_blocks < 1 || d.num_blocks >= (1 << 24)) return fail(MLA_ERR_SHAPE, "num_blocks=%d outside [1, 2^24)", d.num_blocks);
  if (d.max_blocks_per_seq < 1 || d.max_blocks_per_seq > (1 << 23))
    return fail(MLA_ERR_SHAPE, "max_blocks_per_seq=%d outside [1, 2^23]", d.max_blocks_per_seq);
  return MLA_OK;
}

Problem problem_of(const mla_paged_dims& d) {
  Problem p = {};
  p.B = d.B;
  p.S1 = d.S1;
  p.T = d.B * d.S1;
  p.n_q = d.n_q;
  p.n_kv = d.n_kv;
  p.d_qk = d.d_qk;
  p.d_v = d.d_v;
  p.dtype = d.dtype;
  p.causal = 1;
  p.num_blocks = d.num_blocks;
  p.W = d.max_blocks_per_seq;
  return p;
}

}  // namespace
}  // namespace mlaheads

extern "C" {

size_t mla_paged_workspace_bytes(const mla_paged_dims* dims) {
  using namespace mlaheads;
  no_error();
  if (dims == nullptr || check_dims(*dims) != MLA_OK) return 0;
  return tiles_workspace(problem_of(*dims));
}

mla_status mla_paged_attn_fwd(const mla_paged_dims* dims, const mla_heads_tensor* q, const mla_kv_cache* k,
                              const mla_kv_cache* v, const int32_t* block_table, const int32_t* act_seqs,
                              const int32_t* q_lens, void* out, float* lse, float softmax_scale, void* workspace,
                              size_t workspace_bytes, void* stream) {
  using namespace mlaheads;
  no_error();
  if (!dims || !q || !k || !v) return fail(MLA_ERR_NULL, "dims, q, k or v is NULL");
  const mla_status st = check_dims(*dims);
  if (st != MLA_OK) return st;
  Problem p = problem_of(*dims);
  if (p.B == 0) return MLA_OK;
  p.q = *q;
  p.k = *k;
  p.v = *v;
  p.block_table = block_table;
  p.act_seqs = act_seqs;
  p.q_lens = q_lens;
  p.out = out;
  p.lse = lse;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  p.workspace = workspace;
  const mla_status cst = check_problem(p, workspace_bytes, tiles_workspace(p));
  if (cst != MLA_OK) return cst;
  return launch_tiles(p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
