// What the sources behind mla_heads.h share on the host.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mla_heads.h"
#include "areas.h"

namespace mlaheads {

using mlasp::aligned;
using mlasp::Area;
using mlasp::overlap;

// Records the text for mla_heads_last_error() and returns s.
mla_status fail(mla_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void no_error();

// The device status word of a source: read, and cleared where asked.
cudaError_t prep_status(unsigned int* v, bool clear);
cudaError_t prompt_status(unsigned int* v, bool clear);
cudaError_t paged_status(unsigned int* v, bool clear);

template <typename Symbol>
cudaError_t read_status(const Symbol& word, unsigned int* v, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(v, word, sizeof *v);
  const unsigned int zero = 0;
  if (e == cudaSuccess && clear && *v != 0) e = cudaMemcpyToSymbol(word, &zero, sizeof zero);
  return e;
}

#define HEADS_CUDA(call, what)                                                                              \
  do {                                                                                                      \
    const cudaError_t err_ = (call);                                                                        \
    if (err_ != cudaSuccess) return mlaheads::fail(MLA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(err_)); \
  } while (0)

}  // namespace mlaheads

namespace mlaheads {

constexpr int kPage = 128;
constexpr int kMaxDqk = 192, kMaxDv = 128, kMaxGroup = 128;

// An attention call, checked.  Query rows of sequence b: [cu_q[b], cu_q[b + 1]),
// or with S1 > 0 the first q_lens[b] (S1) of b * S1 ...  Keys: pages with
// num_blocks > 0, else rows [cu_k[b], cu_k[b + 1]) (cu_q's where it is null).
struct Problem {
  int B, S1, T, Tk, n_q, n_kv, d_qk, d_v, dtype, causal, num_blocks, W;
  mla_heads_tensor q;
  mla_kv_cache k, v;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* block_table;
  const int32_t* act_seqs;
  const int32_t* q_lens;
  void* out;
  float* lse;
  float scale_log2;
  void* workspace;
};

mla_status check_head_dims(int n_q, int n_kv, int d_qk, int d_v, int dtype);
// Pointers, alignment, strides and overlaps of a call whose dims are checked.
mla_status check_problem(const Problem& p, size_t workspace_bytes, size_t needed);

// The kernels on 128-row tiles (prompt_attn.cu).
size_t tiles_workspace(const Problem& p);
mla_status launch_tiles(const Problem& p, cudaStream_t s);

}  // namespace mlaheads
