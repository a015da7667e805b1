// Dense MLA attention over the whole paged cache for GB300 (sm_103a): single
// tokens, chains and trees of drafted tokens (formulas in mla_tree.h).
//
// First form: one warp per (token, head).  Lane l holds latent dims
// [16 l, 16 l + 16) and rope dims 2 l, 2 l + 1 of the query and of the running
// output; keys go one by one through an online softmax.  Bound by issue.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/mla_tree.h"
#include "ptx.cuh"

namespace mlatree {

using namespace mlasp;

__device__ unsigned int g_tree_status = 0;

struct Params {
  const uint8_t* q_nope;
  const uint8_t* q_rope;
  const uint8_t* kv_nope;
  const uint8_t* kv_rope;
  const float* kv_scales;
  const int32_t* block_table;
  const int32_t* act_seqs;
  const int32_t* tree_lens;
  const uint64_t* tree_mask;
  uint16_t* out;
  float* lse;
  int B, S1, n_q, W, num_blocks, int8;
  float scale_log2;
};

__device__ __forceinline__ void unpack(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

__global__ void __launch_bounds__(256) tree_simple_kernel(const Params p) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<int64_t>(p.B) * p.S1 * p.n_q) return;
  const int t = static_cast<int>(row / p.n_q), b = t / p.S1, s = t - b * p.S1;
  float q[16], o[16], qr[2];
  const uint4* qp = reinterpret_cast<const uint4*>(p.q_nope + row * 1024) + 2 * lane;
  unpack(__ldg(qp), q);
  unpack(__ldg(qp + 1), q + 8);
  const uint32_t qw = __ldg(reinterpret_cast<const uint32_t*>(p.q_rope + row * 128) + lane);
  qr[0] = __uint_as_float(qw << 16);
  qr[1] = __uint_as_float(qw & 0xFFFF0000u);
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = 0.f;
  const int64_t act = max(0, __ldg(p.act_seqs + b));
  const int n = p.tree_lens != nullptr ? min(p.S1, max(0, __ldg(p.tree_lens + b))) : p.S1;
  const int64_t ctx = act - n;
  const int words = (p.S1 + 63) / 64;
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  for (int64_t pos = 0; pos < act && s < n; ++pos) {
    const int64_t j = pos - ctx;
    if (j >= 0) {
      const bool see = p.tree_mask != nullptr
                           ? (__ldg(p.tree_mask + static_cast<int64_t>(t) * words + (j >> 6)) >> (j & 63)) & 1
                           : j <= s;
      if (!see) continue;
    }
    const int64_t lb = pos >> 7;
    const int id = lb < p.W ? __ldg(p.block_table + static_cast<int64_t>(b) * p.W + lb) : -1;
    if (id < 0 || id >= p.num_blocks) {
      bad = true;
      continue;
    }
    const int64_t r = static_cast<int64_t>(id) * 128 + (pos & 127);
    float k[16];
    if (p.int8) {
      const uint4 c = __ldg(reinterpret_cast<const uint4*>(p.kv_nope + r * 512) + lane);
      const float sc = __ldg(p.kv_scales + r * 4 + (lane >> 3));
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const int lo = static_cast<int8_t>(w[e >> 2] >> (8 * (e & 3)));
        const int hi = static_cast<int8_t>(w[e >> 2] >> (8 * ((e & 3) + 1)));
        const uint32_t pr = pack_bf16x2(static_cast<float>(lo) * sc, static_cast<float>(hi) * sc);
        k[e] = __uint_as_float(pr << 16);
        k[e + 1] = __uint_as_float(pr & 0xFFFF0000u);
      }
    } else {
      const uint4* kp = reinterpret_cast<const uint4*>(p.kv_nope + r * 1024) + 2 * lane;
      unpack(__ldg(kp), k);
      unpack(__ldg(kp + 1), k + 8);
    }
    const uint32_t kw = __ldg(reinterpret_cast<const uint32_t*>(p.kv_rope + r * 128) + lane);
    float z = qr[0] * __uint_as_float(kw << 16) + qr[1] * __uint_as_float(kw & 0xFFFF0000u);
#pragma unroll
    for (int e = 0; e < 16; ++e) z = fmaf(q[e], k[e], z);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    z *= p.scale_log2;
    if (!(z <= m)) {  // also for NaN
      const float f = m == -INFINITY ? 0.f : exp2f(m - z);
      l *= f;
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] *= f;
      m = z;
    }
    const float w = m == -INFINITY ? 0.f : exp2f(z - m);
    l += w;
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = fmaf(w, k[e], o[e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  uint4* op = reinterpret_cast<uint4*>(p.out + row * 512) + 2 * lane;
  op[0] = make_uint4(y[0], y[1], y[2], y[3]);
  op[1] = make_uint4(y[4], y[5], y[6], y[7]);
  if (lane == 0) {
    if (p.lse != nullptr) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
    if (bad) atomicOr(&g_tree_status, MLA_DEVICE_BAD_BLOCK);
  }
}

}  // namespace mlatree

namespace {

thread_local char g_tree_error[256] = "";

mla_status tree_fail(mla_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mla_status tree_fail(mla_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_tree_error, sizeof g_tree_error, fmt, ap);
  va_end(ap);
  return s;
}

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

mla_status check_dims(const mla_dims& d) {
  if (d.kv_dtype != MLA_KV_BF16 && d.kv_dtype != MLA_KV_INT8)
    return tree_fail(MLA_ERR_DTYPE, "kv_dtype %d is neither MLA_KV_BF16 nor MLA_KV_INT8", d.kv_dtype);
  if (d.B < 1 || d.S1 < 1 || d.num_blocks < 1 || d.max_blocks_per_seq < 1)
    return tree_fail(MLA_ERR_SHAPE, "B, S1, num_blocks and max_blocks_per_seq must be >= 1");
  if (d.n_q < 1 || d.n_q > 128) return tree_fail(MLA_ERR_SHAPE, "n_q=%d outside [1, 128]", d.n_q);
  if (d.n_kv != 1) return tree_fail(MLA_ERR_UNSUPPORTED, "n_kv=%d: only one latent KV head is implemented", d.n_kv);
  if (d.d_nope != 512 || d.d_rope != 64 || d.block_size != 128)
    return tree_fail(MLA_ERR_UNSUPPORTED, "d_nope=%d d_rope=%d block_size=%d: only 512/64/128 are implemented",
                     d.d_nope, d.d_rope, d.block_size);
  if (d.num_blocks >= (1 << 24)) return tree_fail(MLA_ERR_SHAPE, "num_blocks=%d must be < 2^24", d.num_blocks);
  if (static_cast<int64_t>(d.B) * d.S1 >= (1ll << 31) || static_cast<int64_t>(d.B) * d.S1 * d.n_q >= (1ll << 31))
    return tree_fail(MLA_ERR_SHAPE, "B * S1 * n_q must be < 2^31");
  return MLA_OK;
}

}  // namespace

extern "C" {

size_t mla_tree_workspace_bytes(const mla_dims* dims) {
  g_tree_error[0] = '\0';
  if (dims == nullptr || check_dims(*dims) != MLA_OK) return 0;
  return 256;
}

mla_status mla_tree_attn_fwd(const mla_dims* dims, const void* q_nope, const void* q_rope, const void* kv_nope,
                             const void* kv_rope, const float* kv_scales, const int32_t* block_table,
                             const int32_t* act_seqs, const int32_t* tree_lens, const uint64_t* tree_mask, void* out,
                             float* lse, float softmax_scale, void* workspace, size_t workspace_bytes, void* stream) {
  g_tree_error[0] = '\0';
  if (dims == nullptr) return tree_fail(MLA_ERR_NULL, "dims is NULL");
  const mla_dims d = *dims;
  const mla_status st = check_dims(d);
  if (st != MLA_OK) return st;
  const bool int8 = d.kv_dtype == MLA_KV_INT8;
  if (!q_nope || !q_rope || !kv_nope || !kv_rope || !block_table || !act_seqs || !out || !workspace)
    return tree_fail(MLA_ERR_NULL, "a required pointer is NULL");
  if (int8 && !kv_scales) return tree_fail(MLA_ERR_DTYPE, "kv_scales is required for an INT8 cache");
  if (!isfinite(softmax_scale)) return tree_fail(MLA_ERR_SHAPE, "softmax_scale is not finite");
  if (!aligned(q_nope, 16) || !aligned(q_rope, 16) || !aligned(kv_nope, 16) || !aligned(kv_rope, 16) ||
      !aligned(out, 16) || (int8 && !aligned(kv_scales, 16)))
    return tree_fail(MLA_ERR_ALIGN, "q/kv/out/scales pointers must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(act_seqs, 4) || !aligned(tree_lens, 4) || !aligned(tree_mask, 8) ||
      !aligned(lse, 4) || !aligned(workspace, 256))
    return tree_fail(MLA_ERR_ALIGN, "workspace 256-byte, tree_mask 8-byte, the int32 tensors and lse 4-byte aligned");
  const size_t need = mla_tree_workspace_bytes(dims);
  if (workspace_bytes < need) return tree_fail(MLA_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  mlatree::Params p;
  p.q_nope = static_cast<const uint8_t*>(q_nope);
  p.q_rope = static_cast<const uint8_t*>(q_rope);
  p.kv_nope = static_cast<const uint8_t*>(kv_nope);
  p.kv_rope = static_cast<const uint8_t*>(kv_rope);
  p.kv_scales = int8 ? kv_scales : nullptr;
  p.block_table = block_table;
  p.act_seqs = act_seqs;
  p.tree_lens = tree_lens;
  p.tree_mask = tree_mask;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.B = d.B;
  p.S1 = d.S1;
  p.n_q = d.n_q;
  p.W = d.max_blocks_per_seq;
  p.num_blocks = d.num_blocks;
  p.int8 = int8;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  const int64_t rows = static_cast<int64_t>(d.B) * d.S1 * d.n_q;
  mlatree::tree_simple_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return tree_fail(MLA_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

const char* mla_tree_last_error(void) { return g_tree_error; }

mla_status mla_tree_device_status(void* stream, uint32_t* flags, int32_t clear) {
  g_tree_error[0] = '\0';
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return tree_fail(MLA_ERR_CUDA, "cudaStreamSynchronize: %s", cudaGetErrorString(e));
  unsigned int v = 0;
  e = cudaMemcpyFromSymbol(&v, mlatree::g_tree_status, sizeof v);
  if (e != cudaSuccess) return tree_fail(MLA_ERR_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  if (clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(mlatree::g_tree_status, &zero, sizeof zero);
    if (e != cudaSuccess) return tree_fail(MLA_ERR_CUDA, "clearing the status word: %s", cudaGetErrorString(e));
  }
  if (flags) *flags = v;
  if (v != 0) return tree_fail(MLA_ERR_DEVICE_STATUS, "tree attention device status 0x%x", v);
  return MLA_OK;
}

}  // extern "C"
