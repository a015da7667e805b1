// Attention of prompts for GB300 (sm_103a); formulas in mla_heads.h.
//
// A warp takes one query row through its keys, with the running maximum and sum
// of the softmax in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "heads.h"

namespace mlaheads {

__device__ unsigned int g_prompt_status = 0;

cudaError_t prompt_status(unsigned int* v, bool clear) { return read_status(g_prompt_status, v, clear); }

template <typename E>
__global__ void __launch_bounds__(128) rows_kernel(const __grid_constant__ Problem p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int h = static_cast<int>(row % p.n_q), t = static_cast<int>(row / p.n_q);
  if (t >= p.T) return;
  int b = 0, first = 0, n = 0;
  if (p.S1 > 0) {
    b = t / p.S1;
    first = b * p.S1;
    n = p.q_lens != nullptr ? min(p.S1, max(0, p.q_lens[b])) : p.S1;
  } else {
    bool bad = false, found = false;
    for (int i = 0; i < p.B && !found; ++i) {
      const int lo = min(max(p.cu_q[i], 0), p.T), hi = min(max(p.cu_q[i + 1], 0), p.T);
      bad = bad || lo != p.cu_q[i] || hi != p.cu_q[i + 1] || hi < lo;
      found = t >= lo && t < hi;
      b = i;
      first = lo;
      n = hi - lo;
    }
    if (bad) atomicOr(&g_prompt_status, MLA_DEVICE_BAD_LENGTH);
    if (!found) return;
  }
  int len, key0 = 0;
  if (p.num_blocks > 0) {
    len = max(0, p.act_seqs[b]);
  } else {
    const int32_t* cu = p.cu_k != nullptr ? p.cu_k : p.cu_q;
    key0 = min(max(cu[b], 0), p.Tk);
    const int end = min(max(cu[b + 1], 0), p.Tk);
    if (key0 != cu[b] || end != cu[b + 1] || end < key0) atomicOr(&g_prompt_status, MLA_DEVICE_BAD_LENGTH);
    len = max(0, end - key0);
  }
  const int i = t - first;
  if (i >= n) len = 0;
  const int sees = p.causal ? static_cast<int>(min(static_cast<int64_t>(len), static_cast<int64_t>(len) - n + i + 1)) : len;
  const int hk = h / (p.n_q / p.n_kv);
  float q[kMaxDqk / 32], o[kMaxDv / 32];
  for (int k = 0; k < kMaxDqk / 32; ++k) {
    const int d = lane + 32 * k;
    q[k] = d < p.d_qk ? static_cast<float>(static_cast<const E*>(p.q.data)[t * p.q.token_stride + h * p.q.head_stride + d]) : 0.f;
  }
  for (int k = 0; k < kMaxDv / 32; ++k) o[k] = 0.f;
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  for (int key = 0; key < sees; ++key) {
    int64_t ko, vo;
    if (p.num_blocks > 0) {
      const int page = key / kPage, id = page < p.W ? p.block_table[static_cast<int64_t>(b) * p.W + page] : -1;
      if (id < 0 || id >= p.num_blocks) {
        bad = true;
        continue;
      }
      ko = id * p.k.block_stride + (key % kPage) * p.k.row_stride + hk * p.k.head_stride;
      vo = id * p.v.block_stride + (key % kPage) * p.v.row_stride + hk * p.v.head_stride;
    } else {
      ko = static_cast<int64_t>(key0 + key) * p.k.row_stride + hk * p.k.head_stride;
      vo = static_cast<int64_t>(key0 + key) * p.v.row_stride + hk * p.v.head_stride;
    }
    float z = 0.f;
    for (int k = 0; k < kMaxDqk / 32; ++k) {
      const int d = lane + 32 * k;
      if (d < p.d_qk) z = fmaf(q[k], static_cast<float>(static_cast<const E*>(p.k.data)[ko + d]), z);
    }
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    z *= p.scale_log2;
    const float top = fmaxf(m, z), mm = top == -INFINITY ? 0.f : top;
    const float f = exp2f(m - mm), e = exp2f(z - mm);
    m = top;
    l = l * f + e;
    for (int k = 0; k < kMaxDv / 32; ++k) {
      const int d = lane + 32 * k;
      if (d < p.d_v) o[k] = o[k] * f + e * static_cast<float>(static_cast<const E*>(p.v.data)[vo + d]);
    }
  }
  if (bad && lane == 0) atomicOr(&g_prompt_status, MLA_DEVICE_BAD_BLOCK);
  for (int k = 0; k < kMaxDv / 32; ++k) {
    const int d = lane + 32 * k;
    if (d < p.d_v) static_cast<E*>(p.out)[(static_cast<int64_t>(t) * p.n_q + h) * p.d_v + d] = static_cast<E>(l == 0.f ? 0.f : o[k] / l);
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[static_cast<int64_t>(t) * p.n_q + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

mla_status check_head_dims(int n_q, int n_kv, int d_qk, int d_v, int dtype) {
  if (dtype != MLA_ROPE_BF16 && dtype != MLA_ROPE_FP16) return fail(MLA_ERR_DTYPE, "dtype %d is neither bf16 nor fp16", dtype);
  if (n_q < 1 || n_kv < 1 || n_q % n_kv != 0)
    return fail(MLA_ERR_SHAPE, "n_q=%d must be a multiple of n_kv=%d, both >= 1", n_q, n_kv);
  if (n_q / n_kv > kMaxGroup) return fail(MLA_ERR_UNSUPPORTED, "%d query heads to a key head: at most %d", n_q / n_kv, kMaxGroup);
  if (n_q > (1 << 16)) return fail(MLA_ERR_SHAPE, "n_q=%d above 2^16", n_q);
  if (d_qk < 8 || d_qk % 8 || d_v < 8 || d_v % 8)
    return fail(MLA_ERR_SHAPE, "d_qk=%d and d_v=%d must be multiples of 8, at least 8", d_qk, d_v);
  if (d_qk > kMaxDqk || d_v > kMaxDv)
    return fail(MLA_ERR_UNSUPPORTED, "d_qk=%d and d_v=%d: at most %d and %d", d_qk, d_v, kMaxDqk, kMaxDv);
  return MLA_OK;
}

mla_status check_problem(const Problem& p, size_t workspace_bytes, size_t needed) {
  const bool paged = p.num_blocks > 0, empty_k = !paged && p.Tk == 0;
  if (!p.q.data || !p.out || (!empty_k && (!p.k.data || !p.v.data)) || (needed > 0 && !p.workspace) ||
      (p.S1 == 0 && !p.cu_q) || (paged && (!p.block_table || !p.act_seqs)))
    return fail(MLA_ERR_NULL, "a required pointer is NULL");
  if (!isfinite(p.scale_log2)) return fail(MLA_ERR_SHAPE, "softmax_scale is not finite");
  const int64_t strides[] = {p.q.token_stride, p.q.head_stride, p.k.row_stride, p.k.head_stride, p.v.row_stride,
                             p.v.head_stride, paged ? p.k.block_stride : 0, paged ? p.v.block_stride : 0};
  for (int64_t s : strides) {
    if (s < 0 || s >= (int64_t(1) << 39)) return fail(MLA_ERR_SHAPE, "strides must be in [0, 2^39)");
    if (s % 8) return fail(MLA_ERR_ALIGN, "strides must be multiples of 8 elements");
  }
  if (!aligned(p.q.data, 16) || !aligned(p.k.data, 16) || !aligned(p.v.data, 16) || !aligned(p.out, 16))
    return fail(MLA_ERR_ALIGN, "q, k, v and out must be 16-byte aligned");
  if (!aligned(p.cu_q, 4) || !aligned(p.cu_k, 4) || !aligned(p.block_table, 4) || !aligned(p.act_seqs, 4) ||
      !aligned(p.q_lens, 4) || !aligned(p.lse, 4) || !aligned(p.workspace, 256))
    return fail(MLA_ERR_ALIGN, "workspace 256-byte, the int32 tensors and lse 4-byte aligned");
  if (workspace_bytes < needed) return fail(MLA_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, needed);
  // blocks read and write in no order: nothing that a call reads may be an output
  const int64_t rows = static_cast<int64_t>(p.T) * p.n_q;
  auto kv = [&](const mla_kv_cache& c, int d) {
    const Area pages = {reinterpret_cast<uintptr_t>(c.data), {p.num_blocks, kPage, p.n_kv},
                        {2 * c.block_stride, 2 * c.row_stride, 2 * c.head_stride}, 2ll * d};
    const Area packed = {reinterpret_cast<uintptr_t>(c.data), {1, p.Tk, p.n_kv}, {0, 2 * c.row_stride, 2 * c.head_stride}, 2ll * d};
    return paged ? pages : empty_k ? mlasp::run(nullptr, 0) : packed;
  };
  const Area in[] = {{reinterpret_cast<uintptr_t>(p.q.data), {1, p.T, p.n_q}, {0, 2 * p.q.token_stride, 2 * p.q.head_stride}, 2ll * p.d_qk},
                     kv(p.k, p.d_qk), kv(p.v, p.d_v), mlasp::run(p.cu_q, 4ll * (p.B + 1)), mlasp::run(p.cu_k, 4ll * (p.B + 1)),
                     mlasp::run(p.block_table, 4ll * p.B * p.W), mlasp::run(p.act_seqs, 4ll * p.B), mlasp::run(p.q_lens, 4ll * p.B)};
  const Area outs[] = {mlasp::run(p.out, rows * p.d_v * 2), mlasp::run(p.lse, rows * 4),
                       mlasp::run(needed > 0 ? p.workspace : nullptr, static_cast<int64_t>(needed))};
  for (const Area& o : outs)
    for (const Area& i : in)
      if (overlap(o, i)) return fail(MLA_ERR_UNSUPPORTED, "an output or the workspace overlaps an input");
  if (overlap(outs[0], outs[1]) || overlap(outs[0], outs[2]) || overlap(outs[1], outs[2]))
    return fail(MLA_ERR_UNSUPPORTED, "out, lse and the workspace overlap");
  return MLA_OK;
}

size_t tiles_workspace(const Problem&) { return 256; }

mla_status launch_tiles(const Problem& p, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(p.T) * p.n_q + 3) / 4;
  if (p.dtype == MLA_ROPE_BF16) rows_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), 128, 0, s>>>(p);
  else rows_kernel<__half><<<static_cast<unsigned>(blocks), 128, 0, s>>>(p);
  HEADS_CUDA(cudaGetLastError(), "launch");
  return MLA_OK;
}

namespace {

Problem problem_of(const mla_prompt_dims& d) {
  Problem p = {};
  p.B = d.B;
  p.T = d.T;
  p.Tk = d.Tk;
  p.n_q = d.n_q;
  p.n_kv = d.n_kv;
  p.d_qk = d.d_qk;
  p.d_v = d.d_v;
  p.dtype = d.dtype;
  p.causal = d.causal;
  p.num_blocks = d.num_blocks;
  p.W = d.max_blocks_per_seq;
  return p;
}

mla_status check_dims(const mla_prompt_dims& d) {
  const mla_status st = check_head_dims(d.n_q, d.n_kv, d.d_qk, d.d_v, d.dtype);
  if (st != MLA_OK) return st;
  if (d.B < 0 || d.T < 0 || d.Tk < 0 || d.causal < 0 || d.causal > 1)
    return fail(MLA_ERR_SHAPE, "B, T and Tk must be >= 0, causal 0 or 1");
  if (static_cast<int64_t>(d.T) * d.n_q >= (1ll << 31) - 256 || d.B > (1 << 24))
    return fail(MLA_ERR_SHAPE, "T * n_q must be below 2^31 - 256, B at most 2^24");
  if (d.num_blocks < 0 || d.num_blocks >= (1 << 24)) return fail(MLA_ERR_SHAPE, "num_blocks=%d outside [0, 2^24)", d.num_blocks);
  if (d.num_blocks > 0 ? d.max_blocks_per_seq < 1 || d.max_blocks_per_seq > (1 << 23) || d.Tk != 0 : d.max_blocks_per_seq != 0)
    return fail(MLA_ERR_SHAPE, "paged keys need max_blocks_per_seq in [1, 2^23] and Tk 0, packed ones max_blocks_per_seq 0");
  return MLA_OK;
}

}  // namespace
}  // namespace mlaheads

extern "C" {

size_t mla_prompt_workspace_bytes(const mla_prompt_dims* dims) {
  using namespace mlaheads;
  no_error();
  if (dims == nullptr || check_dims(*dims) != MLA_OK) return 0;
  return tiles_workspace(problem_of(*dims));
}

mla_status mla_prompt_attn_fwd(const mla_prompt_dims* dims, const mla_heads_tensor* q, const mla_kv_cache* k,
                               const mla_kv_cache* v, const int32_t* cu_q, const int32_t* cu_k,
                               const int32_t* block_table, const int32_t* act_seqs, void* out, float* lse,
                               float softmax_scale, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace mlaheads;
  no_error();
  if (!dims || !q || !k || !v) return fail(MLA_ERR_NULL, "dims, q, k or v is NULL");
  const mla_status st = check_dims(*dims);
  if (st != MLA_OK) return st;
  Problem p = problem_of(*dims);
  if (p.num_blocks > 0 && cu_k) return fail(MLA_ERR_UNSUPPORTED, "cu_k is for packed keys");
  if (p.num_blocks == 0 && (block_table || act_seqs)) return fail(MLA_ERR_UNSUPPORTED, "block_table and act_seqs are for paged keys");
  if (p.B == 0 || p.T == 0) return MLA_OK;
  p.q = *q;
  p.k = *k;
  p.v = *v;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.block_table = block_table;
  p.act_seqs = act_seqs;
  p.out = out;
  p.lse = lse;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  p.workspace = workspace;
  const mla_status cst = check_problem(p, workspace_bytes, tiles_workspace(p));
  if (cst != MLA_OK) return cst;
  return launch_tiles(p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
