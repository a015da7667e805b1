// Rotary positions for GB300 (sm_103a): cosine / sine tables and the rotation
// of heads (formulas in mla_rope.h).
//
// Angles.  A pair's frequency is kept as a 64-bit fixed-point fraction of a
// turn per position, so position * frequency modulo 2^64 is the angle modulo
// whole turns, exactly, at the cost of one 64-bit multiply: no fp64 (slow
// here) and no loss at far positions.  Its top bits are the quadrant; the rest,
// at most an eighth of a turn either way, converts to fp32 with full relative
// precision and goes into the Taylor series of sine and cosine.
//
// The rotation is bound by memory.  A thread keeps one token and one unit of a
// head (16 bytes, or one pair of values where alignment forbids that) and walks
// over heads, 64 bytes in flight: its angles are made once, offsets advance by
// one addition, and nothing is shared between threads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "../../include/mla_rope.h"

namespace mlarp {

constexpr int kThreads = 512;
constexpr int kTableThreads = 256;
constexpr int kMaxPairs = 128;  // rot_dim <= 256
constexpr int kSingles = 192;  // threads of a block where values go one by one
constexpr int kMaxPasses = 16, kMaxSinglePasses = 32;  // heads of a thread

__device__ unsigned int g_rope_status = 0;

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

struct TableParams {
  Freqs f;
  const int32_t* positions;
  float* cos;
  float* sin;
  int T, pairs;
};

// A thread makes V adjacent pairs of kTableTokens positions, blockDim.y apart.  V = 4
// (16-byte stores, an index for four values) wherever rows are that aligned:
// 65536 positions of 32 pairs in 6.2 to 6.9 us, box by box (one position a thread,
// 1.7 rounds of blocks, 8.2; single values 10.2).
template <int V>
constexpr int kTableTokens = V == 4 ? 2 : 4;
template <int V>
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ TableParams p) {
  constexpr int kTokens = kTableTokens<V>;
  const int i = threadIdx.x * V;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * (blockDim.y * kTokens) + threadIdx.y;
  int32_t pos[kTokens];
#pragma unroll
  for (int u = 0; u < kTokens; ++u)
    pos[u] = t0 + u * blockDim.y < p.T ? __ldg(p.positions + t0 + u * blockDim.y) : 0;
  uint64_t turn[V];
#pragma unroll
  for (int j = 0; j < V; ++j) turn[j] = p.f.turn[i + j];
  float* cos = p.cos + t0 * p.pairs + i;
  float* sin = p.sin + t0 * p.pairs + i;
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    if (t0 + u * blockDim.y >= p.T) return;
    float2 v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = cos_sin(pos[u], turn[j], p.f.mscale);
    const uint32_t at = u * blockDim.y * p.pairs;
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(cos + at) = make_float4(v[0].x, v[1].x, v[2].x, v[3].x);
      *reinterpret_cast<float4*>(sin + at) = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
    } else {
      cos[at] = v[0].x;
      sin[at] = v[0].y;
    }
  }
}

struct Tensor {
  const void* x;
  void* out;
  int64_t xt, xh, ot, oh;  // strides in elements
  const int64_t* rows;
  int64_t num_rows;
  int n_heads, rot_off;
  int rot_units;    // units of a head that hold rotated values
  int units;        // all units of a head (in place: the rotated ones)
  int tok_rows;     // tokens of a block
  int head_rows;    // heads that a block takes at a time
  int passes;       // times that it does
  int head_blocks;  // blocks over the heads
  int unit_blocks;  // blocks over the units of a head (more than a block's threads)
  uint32_t per_unit, per_head_row;  // 2^22 / units and / head_rows, rounded up
  int blocks;
};

struct Params {
  Freqs f;
  const int32_t* positions;
  Tensor t[2];
  int T, pairs, half, inverse;
};

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

// Turns the pairs of a unit: of two packs (value i of a with value i of b) or within one.
template <typename E, int V, bool kTwo, int N>
__device__ __forceinline__ void turn_unit(Pack<E, V>& a, Pack<E, V>& b, const float2 (&cs)[N]) {
  constexpr int W = Pack<E, V>::W;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    if constexpr (sizeof(E) == 4) {
      if constexpr (kTwo) {
        const float2 y = turn2(__uint_as_float(a.w[k]), __uint_as_float(b.w[k]), cs[k]);
        a.w[k] = __float_as_uint(y.x);
        b.w[k] = __float_as_uint(y.y);
      } else if (k % 2 == 0) {
        const float2 y = turn2(__uint_as_float(a.w[k]), __uint_as_float(a.w[k + 1]), cs[k / 2]);
        a.w[k] = __float_as_uint(y.x);
        a.w[k + 1] = __float_as_uint(y.y);
      }
    } else if constexpr (kTwo) {
      const float2 u = unpack2<E>(a.w[k]), v = unpack2<E>(b.w[k]);
      const float2 y = turn2(u.x, v.x, cs[V == 1 ? 0 : 2 * k]);
      if constexpr (V == 1) {
        a.w[k] = pack2<E>(y.x, 0.f);
        b.w[k] = pack2<E>(y.y, 0.f);
      } else {
        const float2 z = turn2(u.y, v.y, cs[2 * k + 1]);
        a.w[k] = pack2<E>(y.x, z.x);
        b.w[k] = pack2<E>(y.y, z.y);
      }
    } else {
      const float2 u = unpack2<E>(a.w[k]);
      const float2 y = turn2(u.x, u.y, cs[k]);
      a.w[k] = pack2<E>(y.x, y.y);
    }
  }
}

// kTwo: a rotated unit is two packs, V values and the V that turn with them
// (the half layout); otherwise one pack of V / 2 adjacent pairs.
template <typename E, int V, bool kTwo>
__device__ __forceinline__ void rotate_rows(const Params& p, const Tensor& w, int block) {
  constexpr int kPairs = kTwo ? V : V / 2;
  constexpr int kUnroll = kTwo ? 2 : 4;  // heads in flight
  const int tid = threadIdx.x;
  int k, r = 0;
  if (w.unit_blocks == 1) {
    r = tid / w.units;
    k = tid - r * w.units;
    if (r >= w.tok_rows * w.head_rows) return;
  } else {
    k = block % w.unit_blocks * kThreads + tid;
    block /= w.unit_blocks;
    if (k >= w.units) return;
  }
  const int dt = r / w.head_rows;
  const int64_t t = static_cast<int64_t>(block / w.head_blocks) * w.tok_rows + dt;
  const int h = block % w.head_blocks * w.passes * w.head_rows + (r - dt * w.head_rows);
  if (t >= p.T || h >= w.n_heads) return;
  const int n = min(w.passes, (w.n_heads - h + w.head_rows - 1) / w.head_rows);
  const bool rotated = k < w.rot_units;
  int d, pair0 = 0;
  if (rotated) {
    pair0 = k * kPairs;
    d = w.rot_off + (kTwo ? pair0 : 2 * pair0);
  } else {
    const int c = (k - w.rot_units) * V;  // copied values, in order
    d = c < w.rot_off ? c : c + 2 * p.pairs;
  }
  int64_t to = t;
  if (w.rows != nullptr) {
    to = __ldg(w.rows + t);
    if (to >= w.num_rows && k == 0 && h == 0) atomicOr(&g_rope_status, MLA_DEVICE_BAD_BLOCK);
    if (to < 0 || to >= w.num_rows) return;
  }
  const E* x = static_cast<const E*>(w.x) + t * w.xt + h * w.xh + d;
  E* out = static_cast<E*>(w.out) + to * w.ot + h * w.oh + d;
  const int64_t x_step = w.head_rows * w.xh, o_step = w.head_rows * w.oh;
  const int32_t pos = rotated ? __ldg(p.positions + t) : 0;
  Pack<E, V> a[kUnroll], b[kUnroll];
  float2 cs[kPairs];
  for (int it = 0; it < n; it += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (it + u < n) {
        a[u].load(x);
        if (kTwo && rotated) b[u].load(x + p.pairs);
      }
      x += x_step;
    }
    if (it == 0 && rotated) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        cs[i] = cos_sin(pos, p.f.turn[pair0 + i], p.f.mscale);
        if (p.inverse) cs[i].y = -cs[i].y;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (it + u < n) {
        if (rotated) {
          turn_unit<E, V, kTwo>(a[u], b[u], cs);
          if (kTwo) b[u].store(out + p.pairs);
        }
        a[u].store(out);
      }
      out += o_step;
    }
  }
}

// Both tensors in 16-byte units: 403 + 403 MB in 123 us, 98% of a copy's rate.
template <typename E>
__global__ void __launch_bounds__(kThreads, 2) rope_kernel(const __grid_constant__ Params p) {
  const int second = static_cast<int>(blockIdx.x) >= p.t[0].blocks;
  const int block = static_cast<int>(blockIdx.x) - (second ? p.t[0].blocks : 0);
  const Tensor& w = p.t[second];
  if (p.half) rotate_rows<E, 16 / sizeof(E), true>(p, w, block);
  else rotate_rows<E, 16 / sizeof(E), false>(p, w, block);
}

// Applies `body` to `n` heads, G at a time and the rest one by one.
template <int G, typename F>
__device__ __forceinline__ void walk_heads(int n, F&& body) {
  for (; n >= G; n -= G) body(std::integral_constant<int, G>());
  for (; n > 0; --n) body(std::integral_constant<int, 1>());
}

// Rows that are not 16-byte aligned: a thread takes one value, or the two of a
// pair.  Instructions bind it before memory does, so divisions are products with
// reciprocals, a thread walks all heads where there are tokens enough, and the
// heads that fill a group carry no tests: 30 + 30 MB in 18.4 us (the form above
// with single values 20.6, 2.5 times the instructions; 6 or 9 heads in flight
// 20.5 and 24.6, as fewer warps fit).
template <typename E>
__global__ void __launch_bounds__(kSingles, 8) rope_single_kernel(const __grid_constant__ Params p) {
  const int second = static_cast<int>(blockIdx.x) >= p.t[0].blocks;
  int block = static_cast<int>(blockIdx.x) - (second ? p.t[0].blocks : 0);
  const Tensor& w = p.t[second];
  const int tid = threadIdx.x;
  int k = tid, dt = 0, dh = 0;
  if (w.unit_blocks == 1) {
    const int r = static_cast<int>(tid * w.per_unit >> 22);
    k = tid - r * w.units;
    dt = static_cast<int>(r * w.per_head_row >> 22);
    dh = r - dt * w.head_rows;
  } else {
    k += block % w.unit_blocks * static_cast<int>(blockDim.x);
    block /= w.unit_blocks;
  }
  if (k >= w.units || dt >= w.tok_rows) return;
  int hb = 0;
  if (w.head_blocks > 1) {
    hb = block % w.head_blocks;
    block /= w.head_blocks;
  }
  const int64_t t = static_cast<int64_t>(block) * w.tok_rows + dt;
  const int h = hb * w.passes * w.head_rows + dh;
  if (t >= p.T || h >= w.n_heads) return;
  int n = w.passes;  // heads h, h + head_rows, ...
  if (w.head_rows > 1 || w.head_blocks > 1) n = min(n, (w.n_heads - h + w.head_rows - 1) / w.head_rows);
  const bool rotated = k < w.rot_units;
  int d;
  if (rotated) {
    d = w.rot_off + (p.half ? k : 2 * k);
  } else {
    d = k - w.rot_units;
    if (d >= w.rot_off) d += 2 * p.pairs;
  }
  int64_t to = t;
  if (w.rows != nullptr) {
    to = __ldg(w.rows + t);
    if (to >= w.num_rows && k == 0 && h == 0) atomicOr(&g_rope_status, MLA_DEVICE_BAD_BLOCK);
    if (to < 0 || to >= w.num_rows) return;
  }
  const char* x = static_cast<const char*>(w.x) + (t * w.xt + h * w.xh + d) * static_cast<int64_t>(sizeof(E));
  char* out = static_cast<char*>(w.out) + (to * w.ot + h * w.oh + d) * static_cast<int64_t>(sizeof(E));
  const int64_t x_step = w.head_rows * w.xh * static_cast<int64_t>(sizeof(E));
  const int64_t o_step = w.head_rows * w.oh * static_cast<int64_t>(sizeof(E));
  if (!rotated) {
    walk_heads<4>(n, [&](auto group) {
      constexpr int G = decltype(group)::value;
      Pack<E, 1> a[G];
#pragma unroll
      for (int u = 0; u < G; ++u, x += x_step) a[u].load(reinterpret_cast<const E*>(x));
#pragma unroll
      for (int u = 0; u < G; ++u, out += o_step) a[u].store(reinterpret_cast<E*>(out));
    });
    return;
  }
  float2 cs[1] = {cos_sin(__ldg(p.positions + t), p.f.turn[k], p.f.mscale)};
  if (p.inverse) cs[0].y = -cs[0].y;
  const int other = (p.half ? p.pairs : 1) * static_cast<int>(sizeof(E));  // the pair's other value
  walk_heads<3>(n, [&](auto group) {
    constexpr int G = decltype(group)::value;
    Pack<E, 1> a[G], b[G];
#pragma unroll
    for (int u = 0; u < G; ++u, x += x_step) {
      a[u].load(reinterpret_cast<const E*>(x));
      b[u].load(reinterpret_cast<const E*>(x + other));
    }
#pragma unroll
    for (int u = 0; u < G; ++u, out += o_step) {
      turn_unit<E, 1, true>(a[u], b[u], cs);
      a[u].store(reinterpret_cast<E*>(out));
      b[u].store(reinterpret_cast<E*>(out + other));
    }
  });
}

}  // namespace mlarp

namespace {

thread_local char g_rope_error[256] = "";

mla_status rope_fail(mla_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mla_status rope_fail(mla_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_rope_error, sizeof g_rope_error, fmt, ap);
  va_end(ap);
  return s;
}

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// What a call reads or writes: a run of bytes at each of n[0] x n[1] places.
struct Area {
  uintptr_t at;
  int64_t n[2], stride[2], bytes;  // strides in bytes
};
Area run(const void* ptr, int64_t bytes) { return {reinterpret_cast<uintptr_t>(ptr), {1, 1}, {0, 0}, bytes}; }
Area area_of(const mla_rope_tensor* q, const mla_rope_dims& d, bool out) {
  const int64_t size = d.dtype == MLA_ROPE_FP32 ? 4 : 2;
  const bool same = q->x == q->out;  // in place, the rotated part alone is touched
  const int64_t first = same ? q->rot_off : 0, values = same ? d.rot_dim : q->head_dim;
  return {reinterpret_cast<uintptr_t>(out ? q->out : q->x) + static_cast<uintptr_t>(first * size),
          {out && q->rows ? q->num_rows : d.T, q->n_heads},
          {(out ? q->out_token_stride : q->x_token_stride) * size, (out ? q->out_head_stride : q->x_head_stride) * size},
          values * size};
}

// Whether the areas have a byte in common.  Views of one tensor interleave, so
// areas whose stretches overlap are also told apart by their strides: runs of a
// and b bytes that repeat at multiples of g miss one another when the distance
// of their starts, modulo g, is at least a, and b short of g.  Tried for whole
// tokens, whole heads and single runs; what none of them tells apart counts as
// overlapping.
bool overlap(const Area& a, const Area& b) {
  typedef __int128 Wide;  // 2^40 places times a stride of 2^42
  const Wide delta = static_cast<Wide>(b.at) - static_cast<Wide>(a.at);
  auto stride = [](const Area& x, int i) { return x.n[i] > 1 ? static_cast<Wide>(x.stride[i]) : 0; };
  auto length = [&](const Area& x, int i) { return static_cast<Wide>(x.n[i] - 1) * stride(x, i) + x.bytes; };
  auto gcd = [](Wide x, Wide y) {
    while (y != 0) {
      const Wide r = x % y;
      x = y;
      y = r;
    }
    return x;
  };
  auto apart = [&](Wide g, Wide la, Wide lb) {
    if (g == 0) return false;  // nothing repeats: the stretches have been compared
    const Wide r = (delta % g + g) % g;
    return r >= la && g - r >= lb;
  };
  if (delta >= length(a, 0) + length(a, 1) - a.bytes || -delta >= length(b, 0) + length(b, 1) - b.bytes) return false;
  const Wide tokens = gcd(stride(a, 0), stride(b, 0)), heads = gcd(stride(a, 1), stride(b, 1));
  return !(apart(tokens, length(a, 1), length(b, 1)) || apart(heads, length(a, 0), length(b, 0)) ||
           apart(gcd(tokens, heads), a.bytes, b.bytes));
}

// Refuses outputs that overlap what the call reads, or one another: threads read and write in no order.
mla_status check_overlaps(const mla_rope_dims& d, const int32_t* positions, const mla_rope_tensor* q,
                          const mla_rope_tensor* k) {
  const mla_rope_tensor* t[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    if (t[i] == nullptr) continue;
    const Area out = area_of(t[i], d, true);
    bool hit = overlap(out, run(positions, 4ll * d.T));
    for (int j = 0; j < 2; ++j) {
      if (t[j] == nullptr) continue;
      hit = hit || ((i != j || t[i]->x != t[i]->out) && overlap(out, area_of(t[j], d, false)));
      hit = hit || (i < j && overlap(out, area_of(t[j], d, true)));
      hit = hit || (t[j]->rows != nullptr && overlap(out, run(t[j]->rows, 8ll * d.T)));
    }
    if (hit) return rope_fail(MLA_ERR_UNSUPPORTED, "%s's output overlaps an input or the other output", i ? "k" : "q");
  }
  return MLA_OK;
}

// Checks the scheme and fills the fixed-point turns per position.
mla_status make_freqs(const mla_rope_params* q, int rot, mlarp::Freqs* f) {
  if (q == nullptr) return rope_fail(MLA_ERR_NULL, "params is NULL");
  if (rot < 2 || rot > 2 * mlarp::kMaxPairs || (rot & 1))
    return rope_fail(MLA_ERR_SHAPE, "rot_dim=%d must be even, in [2, 256]", rot);
  if (q->scaling < MLA_ROPE_NONE || q->scaling > MLA_ROPE_YARN)
    return rope_fail(MLA_ERR_SHAPE, "scaling %d unknown", q->scaling);
  if (!(q->theta > 1.0) || !isfinite(q->theta)) return rope_fail(MLA_ERR_SHAPE, "theta must be finite and above 1");
  if (!(q->mscale > 0.0) || !isfinite(static_cast<float>(q->mscale)))
    return rope_fail(MLA_ERR_SHAPE, "mscale must be above 0 and finite in fp32");
  if (q->scaling != MLA_ROPE_NONE && (!(q->factor >= 1.0) || !isfinite(q->factor)))
    return rope_fail(MLA_ERR_SHAPE, "factor must be finite and at least 1");
  const bool yarn = q->scaling == MLA_ROPE_YARN;
  if (yarn && (!(q->orig_positions >= 1.0) || !isfinite(q->orig_positions) || !(q->beta_slow > 0.0) ||
               !(q->beta_fast >= q->beta_slow) || !isfinite(q->beta_fast)))
    return rope_fail(MLA_ERR_SHAPE, "orig_positions must be at least 1 and 0 < beta_slow <= beta_fast");
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

// Checks one tensor; *vec stays set if its rows and parts are 16-byte aligned.
mla_status check_tensor(const mla_rope_tensor* q, const mla_rope_dims& d, const char* name, bool* vec) {
  if (!q->x || !q->out) return rope_fail(MLA_ERR_NULL, "%s: a required pointer is NULL", name);
  if (q->n_heads < 1 || q->rot_off < 0 || static_cast<int64_t>(q->rot_off) + d.rot_dim > q->head_dim)
    return rope_fail(MLA_ERR_SHAPE, "%s: n_heads=%d must be >= 1 and the head's %d values hold [rot_off, rot_off + rot_dim)",
                     name, q->n_heads, q->head_dim);
  if (q->head_dim > (1 << 20) || static_cast<int64_t>(q->n_heads) * q->head_dim > (1 << 28))
    return rope_fail(MLA_ERR_SHAPE, "%s: heads of more than 2^20 values, or tokens of more than 2^28", name);
  if (q->x_token_stride < 0 || q->x_head_stride < 0 || q->out_token_stride < 0 || q->out_head_stride < 0)
    return rope_fail(MLA_ERR_SHAPE, "%s: strides must be >= 0", name);
  // rows and heads of out may not run into one another: heads lie within a token's stretch, or tokens within a head's
  const int64_t T = q->rows ? q->num_rows : d.T, H = q->n_heads, D = q->head_dim;
  const int64_t ts = q->out_token_stride, hs = q->out_head_stride;
  const int64_t most = int64_t(1) << 40;
  if (T > most || ts > most || hs > most || q->x_token_stride > most || q->x_head_stride > most)
    return rope_fail(MLA_ERR_SHAPE, "%s: strides and rows must be at most 2^40", name);
  const bool by_token = (H == 1 || hs >= D) && (T <= 1 || ts >= (H - 1) * hs + D);
  const bool by_head = ts >= D && H > 1 && hs / ts >= T - 1 && hs - (T - 1) * ts >= D;
  if (!by_token && !by_head) return rope_fail(MLA_ERR_SHAPE, "%s: out's strides make heads overlap", name);
  if (q->rows && q->num_rows < 1) return rope_fail(MLA_ERR_SHAPE, "%s: num_rows must be >= 1", name);
  if (q->rows && q->x == q->out) return rope_fail(MLA_ERR_UNSUPPORTED, "%s: rows of out cannot be x itself", name);
  const bool same = q->x == q->out;
  if (same && ((q->n_heads > 1 && q->x_head_stride != q->out_head_stride) ||
               (d.T > 1 && q->x_token_stride != q->out_token_stride)))
    return rope_fail(MLA_ERR_SHAPE, "%s: in place, x and out need the same strides", name);
  const int size = d.dtype == MLA_ROPE_FP32 ? 4 : 2, V = 16 / size;
  if (!aligned(q->x, size) || !aligned(q->out, size) || (q->rows && !aligned(q->rows, 8)))
    return rope_fail(MLA_ERR_ALIGN, "%s: tensors must be aligned to their elements", name);
  const bool heads = q->n_heads > 1, tokens = d.T > 1;  // strides that are taken
  const int64_t parts[] = {tokens ? q->x_token_stride : 0,
                           heads ? q->x_head_stride : 0,
                           tokens || q->rows ? q->out_token_stride : 0,
                           heads ? q->out_head_stride : 0,
                           q->head_dim,
                           q->rot_off,
                           d.half ? d.rot_dim / 2 : d.rot_dim};
  *vec = aligned(q->x, 16) && aligned(q->out, 16);
  for (int64_t v : parts) *vec = *vec && v % V == 0;
  return MLA_OK;
}

// Splits a checked tensor's rows into blocks.
mla_status split_tensor(const mla_rope_tensor* q, const mla_rope_dims& d, const char* name, bool vec, mlarp::Tensor* w) {
  const bool same = q->x == q->out;
  w->x = q->x;
  w->out = q->out;
  w->xt = q->x_token_stride;
  w->xh = q->x_head_stride;
  w->ot = q->out_token_stride;
  w->oh = q->out_head_stride;
  w->rows = q->rows;
  w->num_rows = q->num_rows;
  w->n_heads = q->n_heads;
  w->rot_off = q->rot_off;
  const int width = !vec ? 1 : (d.dtype == MLA_ROPE_FP32 ? 4 : 8);
  w->rot_units = vec && !d.half ? d.rot_dim / width : d.rot_dim / 2 / width;
  w->units = w->rot_units + (same ? 0 : (q->head_dim - d.rot_dim) / width);
  const int threads = vec ? mlarp::kThreads : mlarp::kSingles;
  w->unit_blocks = (w->units + threads - 1) / threads;
  const int rows = w->unit_blocks > 1 ? 1 : threads / w->units;
  w->tok_rows = std::min(rows, d.T);
  w->head_rows = std::min(rows / w->tok_rows, q->n_heads);
  // several heads per thread once there is a block for every SM twice over
  const int64_t toks = (static_cast<int64_t>(d.T) + w->tok_rows - 1) / w->tok_rows;
  const int turns = (q->n_heads + w->head_rows - 1) / w->head_rows;
  const int most = std::min(turns, vec ? mlarp::kMaxPasses : mlarp::kMaxSinglePasses);
  w->passes = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, toks * turns / (2 * 152))));
  w->head_blocks = (turns + w->passes - 1) / w->passes;
  w->passes = (turns + w->head_blocks - 1) / w->head_blocks;  // even shares
  // n * per_unit >> 22 is n / units for n and units up to 512: the product's excess is below n / 2^22
  w->per_unit = (1u << 22) / w->units + 1;
  w->per_head_row = (1u << 22) / w->head_rows + 1;
  const int64_t blocks = toks * w->head_blocks * w->unit_blocks;
  if (blocks >= (1ll << 30)) return rope_fail(MLA_ERR_SHAPE, "%s: T x heads too large", name);
  w->blocks = static_cast<int>(blocks);
  return MLA_OK;
}

}  // namespace

extern "C" {

mla_status mla_rope_table(const mla_rope_params* params, int32_t T, int32_t rot_dim, const int32_t* positions,
                          float* cos, float* sin, void* stream) {
  g_rope_error[0] = '\0';
  mlarp::TableParams p;
  const mla_status st = make_freqs(params, rot_dim, &p.f);
  if (st != MLA_OK) return st;
  if (T < 0) return rope_fail(MLA_ERR_SHAPE, "T=%d must be >= 0", T);
  if (T == 0) return MLA_OK;
  if (!positions || !cos || !sin) return rope_fail(MLA_ERR_NULL, "a required pointer is NULL");
  if (!aligned(positions, 4) || !aligned(cos, 4) || !aligned(sin, 4))
    return rope_fail(MLA_ERR_ALIGN, "tensors must be 4-byte aligned");
  const Area table[] = {run(cos, 2ll * T * rot_dim), run(sin, 2ll * T * rot_dim), run(positions, 4ll * T)};
  if (overlap(table[0], table[1]) || overlap(table[0], table[2]) || overlap(table[1], table[2]))
    return rope_fail(MLA_ERR_UNSUPPORTED, "cos, sin and positions overlap");
  p.positions = positions;
  p.cos = cos;
  p.sin = sin;
  p.T = T;
  p.pairs = rot_dim / 2;
  const int width = p.pairs % 4 == 0 && aligned(cos, 16) && aligned(sin, 16) ? 4 : 1;
  const dim3 block(p.pairs / width, mlarp::kTableThreads / (p.pairs / width));
  const int per_block = static_cast<int>(block.y) * (width == 4 ? mlarp::kTableTokens<4> : mlarp::kTableTokens<1>);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(T) + per_block - 1) / per_block);
  (width == 4 ? mlarp::rope_table_kernel<4> : mlarp::rope_table_kernel<1>)<<<grid, block, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return rope_fail(MLA_ERR_CUDA, "rope table launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

mla_status mla_rope_apply(const mla_rope_dims* dims, const mla_rope_params* params, const int32_t* positions,
                          const mla_rope_tensor* q, const mla_rope_tensor* k, void* stream) {
  g_rope_error[0] = '\0';
  if (dims == nullptr || q == nullptr) return rope_fail(MLA_ERR_NULL, "dims or q is NULL");
  const mla_rope_dims d = *dims;
  if (d.dtype < MLA_ROPE_BF16 || d.dtype > MLA_ROPE_FP32) return rope_fail(MLA_ERR_DTYPE, "dtype %d unknown", d.dtype);
  if (d.T < 0 || d.half < 0 || d.half > 1 || d.inverse < 0 || d.inverse > 1)
    return rope_fail(MLA_ERR_SHAPE, "T must be >= 0, half and inverse 0 or 1");
  mlarp::Params p;
  mla_status st = make_freqs(params, d.rot_dim, &p.f);
  if (st != MLA_OK) return st;
  if (d.T == 0) return MLA_OK;
  if (!positions) return rope_fail(MLA_ERR_NULL, "positions is NULL");
  if (!aligned(positions, 4)) return rope_fail(MLA_ERR_ALIGN, "positions must be 4-byte aligned");
  bool vec[2] = {true, true};
  mlarp::Tensor t[2];
  st = check_tensor(q, d, "q", &vec[0]);
  if (st == MLA_OK && k != nullptr) st = check_tensor(k, d, "k", &vec[1]);
  if (st == MLA_OK) st = check_overlaps(d, positions, q, k);
  if (st == MLA_OK) st = split_tensor(q, d, "q", vec[0], &t[0]);
  if (st == MLA_OK && k != nullptr) st = split_tensor(k, d, "k", vec[1], &t[1]);
  if (st != MLA_OK) return st;
  p.positions = positions;
  p.T = d.T;
  p.pairs = d.rot_dim / 2;
  p.half = d.half;
  p.inverse = d.inverse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void (*kernels[3][2])(mlarp::Params) = {{mlarp::rope_single_kernel<__nv_bfloat16>, mlarp::rope_kernel<__nv_bfloat16>},
                                          {mlarp::rope_single_kernel<__half>, mlarp::rope_kernel<__half>},
                                          {mlarp::rope_single_kernel<float>, mlarp::rope_kernel<float>}};
  // one launch, or one each where only one of the tensors has 16-byte rows (8192 tokens x 128 heads of 192 beside
  // an unaligned head of 64: 131 us, both value by value 228)
  const bool together = k != nullptr && vec[0] == vec[1];
  for (int i = 0; i < (k == nullptr || together ? 1 : 2); ++i) {
    p.t[0] = t[i];
    p.t[1] = t[together ? 1 : i];
    if (!together) p.t[1].blocks = 0;
    const unsigned grid = static_cast<unsigned>(p.t[0].blocks + p.t[1].blocks);
    kernels[d.dtype][vec[i] ? 1 : 0]<<<grid, vec[i] ? mlarp::kThreads : mlarp::kSingles, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return rope_fail(MLA_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
  }
  return MLA_OK;
}

const char* mla_rope_last_error(void) { return g_rope_error; }

mla_status mla_rope_device_status(void* stream, uint32_t* flags, int32_t clear) {
  g_rope_error[0] = '\0';
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return rope_fail(MLA_ERR_CUDA, "cudaStreamSynchronize: %s", cudaGetErrorString(e));
  unsigned int v = 0;
  e = cudaMemcpyFromSymbol(&v, mlarp::g_rope_status, sizeof v);
  if (e != cudaSuccess) return rope_fail(MLA_ERR_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  if (clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(mlarp::g_rope_status, &zero, sizeof zero);
    if (e != cudaSuccess) return rope_fail(MLA_ERR_CUDA, "clearing the status word: %s", cudaGetErrorString(e));
  }
  if (flags) *flags = v;
  if (v != 0) return rope_fail(MLA_ERR_DEVICE_STATUS, "rope device status 0x%x", v);
  return MLA_OK;
}

}  // extern "C"
