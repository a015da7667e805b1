// What the attention kernels behind mla_heads.h share.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "heads.h"
#include "ptx.cuh"

namespace mlasp {
unsigned long long host_wait_limit_ns();
}

namespace mlaheads {

using namespace mlasp;

// Waits of a whole warp on barrier i of its CTA's context: bounded, all lanes agree.
template <typename Ctx>
__device__ __forceinline__ bool warp_wait(const Ctx& c, int i, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait<false>(c.bar(i), parity, c.abort, c.wait_ns));
}
// The value of lane 0, which lets the compiler keep it in uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
// a / b and the rest; 64-bit division is slow, and hardly ever needed.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b, int64_t& rest) {
  const int64_t q = ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
  rest = a - q * b;
  return q;
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const void* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar) : "memory");
}

// NaN and infinities of a pair of 16-bit values become zero.
template <typename E>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  constexpr uint32_t kExp = __is_same(E, __half) ? 0x7C00u : 0x7F80u;
  if ((w & kExp) == kExp) w &= 0xFFFF0000u;
  if ((w & kExp << 16) == kExp << 16) w &= 0x0000FFFFu;
  return w;
}
template <typename E>
__device__ __forceinline__ bool finite4(uint4 v) {
  constexpr uint32_t kExp = __is_same(E, __half) ? 0x7C007C00u : 0x7F807F80u;
  constexpr uint32_t kOne = __is_same(E, __half) ? 0x04000400u : 0x00800080u;  // carries out of a full exponent alone
  const uint32_t c = ((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) | ((v.z & kExp) + kOne) | ((v.w & kExp) + kOne);
  return (c & 0x80008000u) == 0;
}

// fp32 pairs (one instruction for two lanes of arithmetic).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <typename E>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (__is_same(E, __half)) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What a running maximum is kept below the scores' own by, in powers of two.  fp16 goes down to
// 2^-14 in full and to 2^-24 in steps of that: weights 2^7 larger than 2^(z - maximum) use the room
// above (they stay below 2^15, the sums are fp32 and the lift cancels): a weight 18 nats under the
// largest is off by 1.5% at most, where it had been lost.
template <typename E>
constexpr float kLift = __is_same(E, __half) ? 7.f : 0.f;

// ------------------------------------------------------------------ host side
inline mla_status tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* encode) {
  cudaDriverEntryPointQueryResult q;
  void* fn = nullptr;
  HEADS_CUDA(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q), "looking up cuTensorMapEncodeTiled");
  if (fn == nullptr || q != cudaDriverEntryPointSuccess) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  *encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return MLA_OK;
}

// A launch that may begin while the launch before it on the stream ends: the
// kernel waits (griddepcontrol.wait) before it touches what that one writes.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A tensor of 16-bit values, the innermost dimension adjacent; strides in elements, of dimensions 1 ...
inline mla_status tmap(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, int dtype, const void* base, int rank, const int64_t* size, const int64_t* stride, const int* box, const char* what) {
  cuuint64_t dim[4], st[3];
  cuuint32_t bx[4], es[4];
  for (int i = 0; i < rank; ++i) {
    dim[i] = static_cast<cuuint64_t>(size[i]);
    bx[i] = static_cast<cuuint32_t>(box[i]);
    es[i] = 1;
    // a dimension of one place is never stepped over: any legal stride will do
    if (i > 0) st[i - 1] = size[i] > 1 ? static_cast<cuuint64_t>(stride[i - 1]) * 2 : ((static_cast<cuuint64_t>(size[0]) * 2 + 15) & ~cuuint64_t(15));
  }
  // L2 fetches whole lines of a run that lies together: a head's values of one token, or rows behind one another
  const bool wide = size[0] * 2 % 256 == 0 || stride[0] == size[0];
  const CUresult r = encode(m, dtype == MLA_ROPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, static_cast<cuuint32_t>(rank),
                              const_cast<void*>(base), dim, st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              wide ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MLA_ERR_CUDA, "tensor map of %s: error %d", what, static_cast<int>(r));
  return MLA_OK;
}

}  // namespace mlaheads
