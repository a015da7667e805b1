// What the rotary kernels share (formulas in mla_rope.h): angles from 64-bit
// fixed-point turns, 16-byte packs of values, and the host's frequencies.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/mla_rope.h"

namespace mlarp {

constexpr int kMaxPairs = 128;  // rot_dim <= 256

struct Freqs {
  uint64_t turn[kMaxPairs];  // turns per position, 64-bit fraction
  float mscale;
};

// cos and sin of position * frequency, times mscale.  With x the rest in turns,
// sin(2 pi x) = x (2 pi - (2 pi)^3 / 3! x^2 + ...) up to x^9 and cos(2 pi x) = 1
// - (2 pi)^2 / 2! x^2 + ... up to x^10: the next terms are below 4e-9 and 8e-10
// at an eighth of a turn.  2 pi goes in as two fp32 values; the errors are 2.6 u
// of the sine and 1.3 u (u = 2^-24), found over two million angles.
__device__ __forceinline__ float2 cos_sin(int32_t pos, uint64_t turn, float mscale) {
  const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turn;
  const uint32_t top = static_cast<uint32_t>(frac >> 32), quadrant = top + 0x20000000u;
  const float hi = static_cast<float>(static_cast<int32_t>(top - (quadrant & 0xC0000000u)));
  // 23 bits of the low word as the fraction of a value in [1, 2): no second conversion
  const float lo = __uint_as_float(0x3F800000u | static_cast<uint32_t>(frac) >> 9) - 1.f;
  const float x = __fmul_rn(hi + lo, 0x1p-32f), z = x * x;
  float p = fmaf(z, 42.058693f, -76.705856f);
  p = fmaf(p, z, 81.605247f);
  p = fmaf(p, z, -41.341702f);
  p = fmaf(p, z, -1.7484555e-7f);
  const float s = fmaf(x, 6.2831855f, __fmul_rn(x, p));
  float c = fmaf(z, -26.426256f, 60.244640f);
  c = fmaf(c, z, -85.456818f);
  c = fmaf(c, z, 64.939392f);
  c = fmaf(c, z, -19.739208f);
  c = fmaf(c, z, 1.f);
  // a quarter turn on: (cos, sin) becomes (-sin, cos)
  const bool swap = (quadrant & 0x40000000u) != 0;
  const uint32_t m = __float_as_uint(mscale), sign_s = quadrant & 0x80000000u;
  const uint32_t sign_c = (quadrant ^ quadrant << 1) & 0x80000000u;
  return make_float2((swap ? s : c) * __uint_as_float(m ^ sign_c), (swap ? c : s) * __uint_as_float(m ^ sign_s));
}

// Two 16-bit values of a word as fp32, and back with one rounding each.
template <typename E>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (sizeof(E) == 2 && __is_same(E, __half)) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename E>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (__is_same(E, __half)) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// One fused operation each, spelt out: a pair's result is the same in every kernel and place.
__device__ __forceinline__ float2 turn2(float a, float b, float2 cs) {
  return make_float2(fmaf(a, cs.x, -__fmul_rn(b, cs.y)), fmaf(a, cs.y, __fmul_rn(b, cs.x)));
}

// V values of type E in memory; W words in registers (single 16-bit values take a word).
template <typename E, int V>
struct Pack {
  static constexpr int W = sizeof(E) * V < 4 ? 1 : sizeof(E) * V / 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const E* p) {
    if constexpr (W == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if constexpr (sizeof(E) == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ void store(E* p) const {
    if constexpr (W == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (sizeof(E) == 2) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
};

// Checks the scheme and fills the fixed-point turns per position; `fail` records an error and gives its status.
template <typename Fail>
mla_status make_freqs(const mla_rope_params* q, int rot, Freqs* f, Fail&& fail) {
  if (q == nullptr) return fail(MLA_ERR_NULL, "params is NULL");
  if (rot < 2 || rot > 2 * kMaxPairs || (rot & 1))
    return fail(MLA_ERR_SHAPE, "rot_dim=%d must be even, in [2, 256]", rot);
  if (q->scaling < MLA_ROPE_NONE || q->scaling > MLA_ROPE_YARN)
    return fail(MLA_ERR_SHAPE, "scaling %d unknown", q->scaling);
  if (!(q->theta > 1.0) || !isfinite(q->theta)) return fail(MLA_ERR_SHAPE, "theta must be finite and above 1");
  if (!(q->mscale > 0.0) || !isfinite(static_cast<float>(q->mscale)))
    return fail(MLA_ERR_SHAPE, "mscale must be above 0 and finite in fp32");
  if (q->scaling != MLA_ROPE_NONE && (!(q->factor >= 1.0) || !isfinite(q->factor)))
    return fail(MLA_ERR_SHAPE, "factor must be finite and at least 1");
  const bool yarn = q->scaling == MLA_ROPE_YARN;
  if (yarn && (!(q->orig_positions >= 1.0) || !isfinite(q->orig_positions) || !(q->beta_slow > 0.0) ||
               !(q->beta_fast >= q->beta_slow) || !isfinite(q->beta_fast)))
    return fail(MLA_ERR_SHAPE, "orig_positions must be at least 1 and 0 < beta_slow <= beta_fast");
  const double two_pi = 6.283185307179586476925;
  double ln = log(q->theta);
  if (q->scaling == MLA_ROPE_NTK) ln += log(q->factor) * rot / std::max(rot - 2, 1);
  double low = 0, high = 0;
  if (yarn) {
    low = std::max(floor(rot * log(q->orig_positions / (two_pi * q->beta_fast)) / (2 * ln)), 0.0);
    high = std::min(ceil(rot * log(q->orig_positions / (two_pi * q->beta_slow)) / (2 * ln)), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double v = exp(-ln * 2 * i / rot);
    if (q->scaling == MLA_ROPE_LINEAR) v /= q->factor;
    if (yarn) {
      const double r = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      v = v * (1 - r) + v / q->factor * r;
    }
    f->turn[i] = static_cast<uint64_t>(v / two_pi * 0x1p64);  // v <= 1: below 2^62
  }
  f->mscale = static_cast<float>(q->mscale);
  return MLA_OK;
}

}  // namespace mlarp
