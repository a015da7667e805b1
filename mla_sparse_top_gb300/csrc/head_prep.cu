// Norms and rotation of heads, and the write of keys and values into a paged
// cache, for GB300 (sm_103a); formulas in mla_heads.h.
//
// A head is one group of 1 to 32 lanes: its units (16 bytes, two of them where
// the half layout pairs them, or single values where alignment forbids that)
// are spread over the group, the norm's sums go round it by shuffles, and the
// rotation needs no lane but its own.  A group keeps its token and walks over
// heads, so angles and weights are made once.  Everything is read once and
// written once: bound by memory.
// Measured (graph replay): 8192 tokens of 32 + 8 heads of 128 in bf16, RMS norms and
// rotation, 33 us (168 MB, 5.1 TB/s), with 64 + 8 heads 52 (5.8 TB/s); 16384 new tokens to
// the cache, 28 + 4 + 4 heads of 128 of which 64 turn, no norm, 54 us (302 MB, 5.6 TB/s); 64 new tokens 5.6 us, of which
// the launch is most; 4099 tokens of 17 fp32 heads of 107, LayerNorm, 35 us: single
// values and two sums that follow one another, bound by latency and instructions.
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "heads.h"
#include "rope_angles.cuh"

namespace mlaheads {

using mlarp::Freqs;
using mlarp::Pack;

constexpr int kThreads = 128;
constexpr int kMaxPasses = 16;  // heads of a group (8: 16384 new tokens to the cache 54 -> 57 us)
// Heads in flight and the one that is worked on, in shared memory: in registers, four ahead,
// norms of 8192 tokens took 42 us and 16384 new tokens to the cache 60.  2 / 3 / 4 / 6 / 8:
// 36 / 34 / 33 / 34 / 39 and 63 / 57 / 54 / 60 / 67.
constexpr int kStages = 4;
constexpr int kHeadsAhead = 2;  // of single values, in registers
// Blocks of an SM: 5 to 7 alike, 8 (64 registers) 38 and 54 us.  Of single values, with or
// without a mean: latency binds, so as many as the registers let go (5 and 6: 4099 tokens of 17
// fp32 heads of 107 25 us instead of 21, with LayerNorm 37 and 36).
constexpr int kBlocks = 5, kLayerBlocks = 7, kSingleBlocks = 8;

__device__ unsigned int g_prep_status = 0;

struct Tensor {
  const void* x;
  void* out;
  int64_t xt, xh;        // strides in elements
  int64_t ob, orow, oh;  // of a block of 128 rows, a row, a head
  const int64_t* rows;
  int64_t num_rows;
  const void* weight;
  const void* bias;
  float eps, inv_d;
  int kind, weight_fp32, weight_vec;  // vec: weights are read 16 bytes at a time
  int n_heads, rot_off;
  int pairs, half;     // of the rotation; 0 pairs: none
  int rot_units;       // units of a head that hold rotated values
  int units;           // all units of a head
  int per_lane;        // units of a lane
  int lanes;           // of a group, a power of two
  int chunks;          // times that the group's lanes go over a head
  int tok_rows;        // tokens of a block
  int head_rows;       // heads that a block takes at a time
  int passes;          // times that it does
  int head_blocks;     // blocks over the heads
  int blocks;
};

struct Params {
  Freqs f;
  const int32_t* positions;
  Tensor t[3];
  int T;
};

template <typename E, int V>
__device__ __forceinline__ void unpack(const Pack<E, V>& a, float* x) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __uint_as_float(a.w[i]);
  } else if constexpr (V == 1) {
    x[0] = mlarp::unpack2<E>(a.w[0]).x;
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 v = mlarp::unpack2<E>(a.w[i]);
      x[2 * i] = v.x;
      x[2 * i + 1] = v.y;
    }
  }
}
template <typename E, int V>
__device__ __forceinline__ void pack(Pack<E, V>& a, const float* x) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) a.w[i] = __float_as_uint(x[i]);
  } else if constexpr (V == 1) {
    a.w[0] = mlarp::pack2<E>(x[0], 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) a.w[i] = mlarp::pack2<E>(x[2 * i], x[2 * i + 1]);
  }
}

// V weights from `at` on, in 16-byte loads where `vec` says that they are so aligned.
template <typename E, int V>
__device__ __forceinline__ void values(const void* p, int at, int fp32, int vec, float* v) {
  if (fp32 || sizeof(E) == 4) {
    const float* f = static_cast<const float*>(p) + at;
    if (V >= 4 && vec) {
#pragma unroll
      for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(v + i) = __ldg(reinterpret_cast<const float4*>(f + i));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __ldg(f + i);
    }
  } else {
    const E* e = static_cast<const E*>(p) + at;
    Pack<E, V> a;
    if (V == 1 || vec) {
      a.load(e);
      unpack<E, V>(a, v);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        Pack<E, 1> one;
        one.load(e + i);
        unpack<E, 1>(one, v + i);
      }
    }
  }
}

// A lane's units of a head.  kTwo: a rotated unit is two packs, V values and the
// V that turn with them, and comes before those that are copied; otherwise units
// lie as the values do, V / 2 adjacent pairs of which any may turn.
template <typename E, int V, bool kTwo, int KU>
struct Lane {
  static constexpr int kVals = kTwo ? 2 * V : V;
  static constexpr int kPairs = kTwo ? V : V / 2;
  int d[KU];   // first value
  int second;  // distance of a rotated unit's other pack
  bool in[KU], rot[KU];
  uint32_t turns[KU];  // a bit for each of a unit's pairs
  __device__ __forceinline__ void place(const Tensor& w, int first_unit, int lane) {
    second = kTwo ? (w.half ? w.pairs : 1) : 0;
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      const int k = first_unit + lane + i * w.lanes;
      in[i] = k < w.units;
      if constexpr (!kTwo) {
        d[i] = k * V;
        // pairs [first, end) of the unit
        const int first = min(max((w.rot_off - d[i]) / 2, 0), kPairs), end = min(max((w.rot_off + 2 * w.pairs - d[i]) / 2, 0), kPairs);
        turns[i] = w.rot_units > 0 ? (1u << end) - (1u << min(first, end)) : 0u;
        rot[i] = turns[i] != 0;
        continue;
      }
      rot[i] = k < w.rot_units;
      if (rot[i]) {
        d[i] = w.rot_off + (w.half ? k * V : 2 * k);
      } else {
        const int c = (k - w.rot_units) * V;  // copied values, in order
        d[i] = c < w.rot_off ? c : c + 2 * w.pairs;
      }
    }
  }
  __device__ __forceinline__ void load(const E* x, bool live, Pack<E, V> (&a)[KU], Pack<E, V> (&b)[KU]) const {
    // what is never loaded holds zero from the start, which a norm's sums count on; behind the last head
    // there are another head's values, whose results go nowhere
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      if (live && in[i]) {
        a[i].load(x + d[i]);
        if (kTwo && rot[i]) b[i].load(x + d[i] + second);
      }
    }
  }
};

// fp32 pairs (one instruction for two lanes of arithmetic: instructions bind the
// kernel where memory does not).
typedef uint64_t Two;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(Two v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void copy_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}

// The rotation of a normed pair is linear in the pair: weights go into the cosines
// and sines, once for a token, the bias turns along, and the norm's factor comes last.
// Coefficients of two values each: of two pairs (of a pack, or of two units of single
// values), or of the two values of one.
//   two packs:  first' = first straight - second cross,  second' = first back + second other
//   one pack:   (u, v)' = (u, v) straight + (v, u) cross
struct Coef {
  Two straight, cross, back, other;
};

template <typename E, int V, bool kTwo, int KU, bool kLayer>
__device__ __forceinline__ void work(const Params& p, const Tensor& w, int block) {
  using L = Lane<E, V, kTwo, KU>;
  const int tid = threadIdx.x;
  const int r = tid / w.lanes, lane = tid & (w.lanes - 1);
  const int dt = r / w.head_rows;
  const int64_t t = static_cast<int64_t>(block / w.head_blocks) * w.tok_rows + dt;
  const int h0 = block % w.head_blocks * w.passes * w.head_rows + (r - dt * w.head_rows);
  bool live = dt < w.tok_rows && t < p.T && h0 < w.n_heads;  // every lane stays for the shuffles
  int64_t to = t;
  if (live && w.rows != nullptr) {
    to = __ldg(w.rows + t);
    if (to >= w.num_rows && lane == 0 && h0 == 0) atomicOr(&g_prep_status, MLA_DEVICE_BAD_BLOCK);
    live = to >= 0 && to < w.num_rows;
  }
  if (!live) to = 0;
  const E* x = static_cast<const E*>(w.x) + (live ? t * w.xt + h0 * w.xh : 0);
  E* out = static_cast<E*>(w.out) + (live ? (to >> 7) * w.ob + (to & 127) * w.orow + h0 * w.oh : 0);
  const int32_t pos = live && w.rot_units > 0 ? __ldg(p.positions + t) : 0;
  const bool normed = w.kind != MLA_NORM_NONE, layer = kLayer && w.kind == MLA_NORM_LAYER;
  L at;
  constexpr int kCoefs = KU * L::kPairs / (kTwo ? 2 : 1);
  static_assert(!kTwo || KU * V % 2 == 0, "pairs of pairs");
  Coef co[kCoefs];
  Two ba[kLayer ? kCoefs : 1], bb[kLayer && kTwo ? kCoefs : 1];
  auto coefficients = [&]() {
    float wt[KU][L::kVals], bi[KU][L::kVals];
#pragma unroll
    for (int i = 0; i < KU; ++i) {
#pragma unroll
      for (int j = 0; j < L::kVals; ++j) {
        wt[i][j] = 1.f;
        bi[i][j] = 0.f;
      }
      if (normed && at.in[i]) {
        if (w.weight != nullptr) {
          values<E, V>(w.weight, at.d[i], w.weight_fp32, w.weight_vec, wt[i]);
          if (kTwo && at.rot[i]) values<E, V>(w.weight, at.d[i] + at.second, w.weight_fp32, w.weight_vec, wt[i] + L::kVals - V);
        }
        if (kLayer && w.bias != nullptr) {
          values<E, V>(w.bias, at.d[i], w.weight_fp32, w.weight_vec, bi[i]);
          if (kTwo && at.rot[i]) values<E, V>(w.bias, at.d[i] + at.second, w.weight_fp32, w.weight_vec, bi[i] + L::kVals - V);
        }
      }
    }
    auto angle = [&](int i, int j) {
      return (kTwo ? at.rot[i] : (at.turns[i] >> j & 1u) != 0)
                 ? mlarp::cos_sin(pos, p.f.turn[(at.d[i] - w.rot_off) / (kTwo && w.half ? 1 : 2) + j], p.f.mscale)
                 : make_float2(1.f, 0.f);
    };
#pragma unroll
    for (int k = 0; k < kCoefs; ++k) {
      if constexpr (kTwo) {
        const int i = 2 * k / V, j = 2 * k % V, i2 = (2 * k + 1) / V, j2 = (2 * k + 1) % V;
        const float2 c = angle(i, j), d = angle(i2, j2);
        co[k] = {two(wt[i][j] * c.x, wt[i2][j2] * d.x), two(-wt[i][V + j] * c.y, -wt[i2][V + j2] * d.y),
                 two(wt[i][j] * c.y, wt[i2][j2] * d.y), two(wt[i][V + j] * c.x, wt[i2][V + j2] * d.x)};
        if constexpr (kLayer) {
          const float2 y = mlarp::turn2(bi[i][j], bi[i][V + j], c), z = mlarp::turn2(bi[i2][j2], bi[i2][V + j2], d);
          ba[k] = two(y.x, z.x);
          bb[k] = two(y.y, z.y);
        }
      } else {
        const int i = k / L::kPairs, j = k % L::kPairs;
        const float2 c = angle(i, j);
        co[k].straight = two(wt[i][2 * j] * c.x, wt[i][2 * j + 1] * c.x);
        co[k].cross = two(-wt[i][2 * j + 1] * c.y, wt[i][2 * j] * c.y);
        if constexpr (kLayer) {
          const float2 y = mlarp::turn2(bi[i][2 * j], bi[i][2 * j + 1], c);
          ba[k] = two(y.x, y.y);
        }
      }
    }
  };
  at.place(w, 0, lane);
  // a chunk's part of sum (x - mean) or its squares
  auto part = [&](const Pack<E, V>(&a)[KU], const Pack<E, V>(&b)[KU], float mean, bool square) {
    Two s = two(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      float v[L::kVals];
      unpack<E, V>(a[i], v);
      if constexpr (kTwo) unpack<E, V>(b[i], v + V);
      if constexpr (kLayer) {
#pragma unroll
        for (int j = 0; j < L::kVals; ++j) v[j] = at.in[i] && (j < V || at.rot[i]) ? v[j] - mean : 0.f;
      }
#pragma unroll
      for (int j = 0; j < L::kVals; j += 2) {  // places without a value hold zero
        const Two c = two(v[j], v[j + 1]);
        s = square ? fma2(c, c, s) : add2(s, c);
      }
    }
    const float2 h = halves(s);
    return h.x + h.y;
  };
  // norm, rotation and store of a chunk
  auto finish = [&](const Pack<E, V>(&a)[KU], const Pack<E, V>(&b)[KU], float mean, float inv, E* o, bool put) {
    const Two inv2 = two(inv, inv);
    float v[KU][L::kVals];
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      unpack<E, V>(a[i], v[i]);
      if constexpr (kTwo) unpack<E, V>(b[i], v[i] + V);
      if constexpr (kLayer) {
#pragma unroll
        for (int j = 0; j < L::kVals; ++j) v[i][j] -= mean;
      }
    }
#pragma unroll
    for (int k = 0; k < kCoefs; ++k) {
      if constexpr (kTwo) {
        const int i = 2 * k / V, j = 2 * k % V, i2 = (2 * k + 1) / V, j2 = (2 * k + 1) % V;
        const Two x = two(v[i][j], v[i2][j2]);
        // a unit that does not turn has no second pack: nothing of it may reach the first
        const Two y = kLayer ? two(at.rot[i] ? v[i][V + j] : 0.f, at.rot[i2] ? v[i2][V + j2] : 0.f) : two(v[i][V + j], v[i2][V + j2]);
        Two first = fma2(y, co[k].cross, mul2(x, co[k].straight)), second = fma2(x, co[k].back, mul2(y, co[k].other));
        if constexpr (kLayer) {
          first = fma2(first, inv2, ba[k]);
          second = fma2(second, inv2, bb[k]);
        } else {
          first = mul2(first, inv2);
          second = mul2(second, inv2);
        }
        const float2 f = halves(first), g = halves(second);
        v[i][j] = f.x;
        v[i2][j2] = f.y;
        v[i][V + j] = g.x;
        v[i2][V + j2] = g.y;
      } else {
        const int i = k / L::kPairs, j = k % L::kPairs;
        const Two x = two(v[i][2 * j], v[i][2 * j + 1]), y = two(v[i][2 * j + 1], v[i][2 * j]);
        // what does not turn keeps apart from its neighbour
        Two r = (at.turns[i] >> j & 1u) != 0 ? fma2(y, co[k].cross, mul2(x, co[k].straight)) : mul2(x, co[k].straight);
        if constexpr (kLayer) r = fma2(r, inv2, ba[k]);
        else r = mul2(r, inv2);
        const float2 f = halves(r);
        v[i][2 * j] = f.x;
        v[i][2 * j + 1] = f.y;
      }
    }
    // a and b stay as they came: a place that no load fills holds its zero for the heads that follow
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      Pack<E, V> first = a[i], second = b[i];
      if (normed || at.rot[i]) {  // else the values go as they came
        pack<E, V>(first, v[i]);
        if constexpr (kTwo) pack<E, V>(second, v[i] + V);
      }
      if (put && at.in[i]) {
        first.store(o + at.d[i]);
        if (kTwo && at.rot[i]) second.store(o + at.d[i] + at.second);
      }
    }
  };
  // mean and 1 / root from a head's sums
  auto root = [&](float sum) {
    const float m = fmaf(sum, w.inv_d, w.eps), r = rsqrtf(m);
    // one step of Newton's takes the approximation's two steps off; not for 0 and infinity
    return m > 1e-36f && m < 1e36f ? fmaf(fmaf(-m * r, r, 1.f), 0.5f * r, r) : r;
  };
  auto group_sum = [&](float v) {
    for (int o = w.lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  const int64_t x_step = w.head_rows * w.xh, o_step = w.head_rows * w.oh;
  const int heads = live ? min(w.passes, (w.n_heads - h0 + w.head_rows - 1) / w.head_rows) : 0;  // of this group
  if (w.chunks == 1) {
    float mean = 0.f, inv = 1.f;
    auto sums = [&](const Pack<E, V>(&a)[KU], const Pack<E, V>(&b)[KU]) {
      if (layer) mean = group_sum(part(a, b, 0.f, false)) * w.inv_d;
      if (normed) inv = root(group_sum(part(a, b, mean, true)));
    };
    if constexpr (V > 1) {
      // copies ahead of the head that is worked on, each lane's into places of its own
      __shared__ uint4 stage[kStages][2][kThreads];
      static_assert(KU == 1 && sizeof(Pack<E, V>) == 16, "a unit of a lane");
      auto fetch = [&](int slot, bool on) {
        if (on && at.in[0]) {
          copy_async(&stage[slot][0][tid], x + at.d[0]);
          if (kTwo && at.rot[0]) copy_async(&stage[slot][1][tid], x + at.d[0] + at.second);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        x += x_step;
      };
      auto fetched = [&](const uint4& from, bool on, Pack<E, V>& a) {  // what was not copied is zero
        const uint4 v = on ? from : make_uint4(0, 0, 0, 0);
        a.w[0] = v.x;
        a.w[1] = v.y;
        a.w[2] = v.z;
        a.w[3] = v.w;
      };
      for (int u = 0; u < kStages - 1; ++u) fetch(u, u < heads);
      if (normed || w.rot_units > 0) coefficients();  // while the copies are on their way
#pragma unroll 1
      for (int it = 0; it < w.passes; ++it, out += o_step) {
        fetch((it + kStages - 1) % kStages, it + kStages - 1 < heads);
        asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 1) : "memory");
        Pack<E, V> a[1], b[1];
        fetched(stage[it % kStages][0][tid], at.in[0], a[0]);
        fetched(stage[it % kStages][1][tid], kTwo && at.rot[0], b[0]);
        sums(a, b);
        finish(a, b, mean, inv, out, it < heads);
      }
    } else {
      // single values may be too small to copy: heads ahead in registers
      constexpr int kSets = kHeadsAhead + 1;
      Pack<E, V> a[kSets][KU], b[kSets][KU];
#pragma unroll
      for (int u = 0; u < kSets; ++u)
#pragma unroll
        for (int i = 0; i < KU; ++i)
#pragma unroll
          for (int k = 0; k < Pack<E, V>::W; ++k) a[u][i].w[k] = b[u][i].w[k] = 0;
#pragma unroll
      for (int u = 0; u < kSets - 1; ++u, x += x_step) at.load(x, u < heads, a[u], b[u]);
      if (normed || w.rot_units > 0) coefficients();
      for (int it = 0; it < w.passes; it += kSets) {
#pragma unroll
        for (int u = 0; u < kSets; ++u, x += x_step, out += o_step) {
          if (it + u >= w.passes) break;
          at.load(x, it + u + kSets - 1 < heads, a[(u + kSets - 1) % kSets], b[(u + kSets - 1) % kSets]);
          sums(a[u], b[u]);
          finish(a[u], b[u], mean, inv, out, it + u < heads);
        }
      }
    }
    return;
  }
  // heads of more values than the group holds, chunk by chunk
  auto clear = [&](Pack<E, V>(&a)[KU], Pack<E, V>(&b)[KU]) {
#pragma unroll
    for (int i = 0; i < KU; ++i)
#pragma unroll
      for (int k = 0; k < Pack<E, V>::W; ++k) a[i].w[k] = b[i].w[k] = 0;
  };
  for (int it = 0; it < w.passes; ++it, x += x_step, out += o_step) {
    Pack<E, V> a[KU], b[KU];
    float mean = 0.f, inv = 1.f;
    for (int step = layer ? 0 : 1; step < 2 && normed; ++step) {
      float sum = 0.f;
      for (int c = 0; c < w.chunks; ++c) {
        at.place(w, c * KU * w.lanes, lane);
        clear(a, b);
        at.load(x, it < heads, a, b);
        sum += part(a, b, mean, step == 1);
      }
      sum = group_sum(sum);
      if (step == 0) mean = sum * w.inv_d;
      else inv = root(sum);
    }
    for (int c = 0; c < w.chunks; ++c) {  // in place, a lane has read and written its own values alone
      at.place(w, c * KU * w.lanes, lane);
      coefficients();
      clear(a, b);
      at.load(x, it < heads, a, b);
      finish(a, b, mean, inv, out, it < heads);
    }
  }
}

// One block works on one of the tensors.
template <typename E, int V, int KU, bool kLayer>
__global__ void __launch_bounds__(kThreads, V > 1 ? kBlocks : kLayer ? kLayerBlocks : kSingleBlocks) head_prep_kernel(const __grid_constant__ Params p) {
  int block = static_cast<int>(blockIdx.x), i = 0;
  while (i < 2 && block >= p.t[i].blocks) block -= p.t[i++].blocks;
  const Tensor& w = p.t[i];
  if constexpr (V > 1) {
    if (!w.half) return work<E, V, false, KU, kLayer>(p, w, block);
  }
  work<E, V, true, KU, kLayer>(p, w, block);
}

thread_local char g_error[256] = "";

mla_status fail(mla_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_error, sizeof g_error, fmt, ap);
  va_end(ap);
  return s;
}
void no_error() { g_error[0] = '\0'; }

cudaError_t prep_status(unsigned int* v, bool clear) { return read_status(g_prep_status, v, clear); }

namespace {

// One tensor of a call as the host sees it.
struct Job {
  const char* name;
  const void* x;
  int64_t xt, xh;
  void* out;
  int64_t ob, orow, oh;  // block, row and head strides of out
  const int64_t* rows;
  int64_t num_rows;  // rows of out
  int n_heads, head_dim, rot_off, rot_dim;
  mla_head_norm norm;
  bool vec;
  Area in, to;
};

constexpr int64_t kMost = int64_t(1) << 40;

// Strides and layout; *job.vec is set where 16-byte accesses fit.
mla_status check_job(Job& j, int T, int dtype, bool half, bool paged) {
  if (!j.x || !j.out) return fail(MLA_ERR_NULL, "%s: a required pointer is NULL", j.name);
  if (j.n_heads < 1 || j.head_dim < 1 || j.rot_off < 0 || static_cast<int64_t>(j.rot_off) + j.rot_dim > j.head_dim)
    return fail(MLA_ERR_SHAPE, "%s: n_heads=%d must be >= 1 and the head's %d values hold [rot_off, rot_off + rot_dim)",
                j.name, j.n_heads, j.head_dim);
  if (j.head_dim > (1 << 20) || static_cast<int64_t>(j.n_heads) * j.head_dim > (1 << 28))
    return fail(MLA_ERR_SHAPE, "%s: heads of more than 2^20 values, or tokens of more than 2^28", j.name);
  for (int64_t s : {j.xt, j.xh, j.ob, j.orow, j.oh})
    if (s < 0 || s > kMost) return fail(MLA_ERR_SHAPE, "%s: strides must be in [0, 2^40]", j.name);
  if (j.num_rows < 1 || j.num_rows > kMost) return fail(MLA_ERR_SHAPE, "%s: rows must be in [1, 2^40]", j.name);
  const mla_head_norm& n = j.norm;
  if (n.kind < MLA_NORM_NONE || n.kind > MLA_NORM_LAYER || n.fp32 < 0 || n.fp32 > 1)
    return fail(MLA_ERR_SHAPE, "%s: norm kind %d unknown, or its fp32 neither 0 nor 1", j.name, n.kind);
  if (n.kind != MLA_NORM_NONE && (!(n.eps >= 0.f) || !(n.eps < 3.4e38f)))
    return fail(MLA_ERR_SHAPE, "%s: eps must be finite and >= 0", j.name);
  if (n.kind == MLA_NORM_RMS && n.bias) return fail(MLA_ERR_UNSUPPORTED, "%s: the RMS norm has no bias", j.name);
  const int size = dtype == MLA_ROPE_FP32 ? 4 : 2, V = 16 / size;
  const uintptr_t wsize = n.fp32 ? 4 : static_cast<uintptr_t>(size);
  if (!aligned(j.x, size) || !aligned(j.out, size) || (j.rows && !aligned(j.rows, 8)) ||
      (n.kind != MLA_NORM_NONE && (!aligned(n.weight, wsize) || !aligned(n.bias, wsize))))
    return fail(MLA_ERR_ALIGN, "%s: tensors must be aligned to their elements", j.name);
  const bool same = j.x == j.out;
  if (same && j.rows) return fail(MLA_ERR_UNSUPPORTED, "%s: rows of out cannot be x itself", j.name);
  if (same && ((j.n_heads > 1 && j.xh != j.oh) || (T > 1 && j.xt != j.orow)))
    return fail(MLA_ERR_SHAPE, "%s: in place, x and out need the same strides", j.name);
  const int64_t bytes = static_cast<int64_t>(j.head_dim) * size;
  j.in = {reinterpret_cast<uintptr_t>(j.x), {1, T, j.n_heads}, {0, j.xt * size, j.xh * size}, bytes};
  if (paged)
    j.to = {reinterpret_cast<uintptr_t>(j.out), {j.num_rows / 128, 128, j.n_heads}, {j.ob * size, j.orow * size, j.oh * size}, bytes};
  else
    j.to = {reinterpret_cast<uintptr_t>(j.out), {1, j.rows ? j.num_rows : T, j.n_heads}, {0, j.orow * size, j.oh * size}, bytes};
  if (!mlasp::distinct(j.to)) return fail(MLA_ERR_SHAPE, "%s: the output's strides make heads overlap", j.name);
  const bool heads = j.n_heads > 1, tokens = T > 1;  // strides that are taken
  // interleaved pairs may begin and end anywhere, but not lie in two units
  const int64_t parts[] = {tokens ? j.xt : 0, heads ? j.xh : 0, tokens || j.rows ? j.orow : 0, j.rows ? j.ob : 0,
                           heads ? j.oh : 0, j.head_dim, half ? j.rot_off : 0, half ? j.rot_dim / 2 : 0};
  j.vec = aligned(j.x, 16) && aligned(j.out, 16) && (half || j.rot_dim == 0 || j.rot_off % 2 == 0);
  for (int64_t v : parts) j.vec = j.vec && v % V == 0;
  return MLA_OK;
}

// Refuses outputs that overlap what the call reads, or one another: blocks read and write in no order.
mla_status check_overlaps(const Job* jobs, int n, int T, const int32_t* positions, const int64_t* rows, int dtype) {
  const int size = dtype == MLA_ROPE_FP32 ? 4 : 2;
  for (int i = 0; i < n; ++i) {
    bool hit = overlap(jobs[i].to, mlasp::run(positions, 4ll * T)) || overlap(jobs[i].to, mlasp::run(rows, 8ll * T));
    for (int k = 0; k < n; ++k) {
      const mla_head_norm& norm = jobs[k].norm;
      hit = hit || ((i != k || jobs[i].x != jobs[i].out) && overlap(jobs[i].to, jobs[k].in));
      hit = hit || (i < k && overlap(jobs[i].to, jobs[k].to));
      if (norm.kind != MLA_NORM_NONE) {
        const int64_t bytes = static_cast<int64_t>(jobs[k].head_dim) * (norm.fp32 ? 4 : size);
        hit = hit || overlap(jobs[i].to, mlasp::run(norm.weight, bytes)) || overlap(jobs[i].to, mlasp::run(norm.bias, bytes));
      }
    }
    if (hit) return fail(MLA_ERR_UNSUPPORTED, "%s's output overlaps an input or another output", jobs[i].name);
  }
  return MLA_OK;
}

// Units of a lane: one of 16 bytes; of single values two where 64 hold a head, else four (4096
// tokens of 32 bf16 heads of 128, unaligned: 46 us with four, 30 with two).
constexpr int kUnits = 1, kFewUnits = 2, kSingleUnits = 4;

// Splits a checked tensor's heads into groups and blocks.
mla_status split_job(const Job& j, int T, int dtype, bool half, Tensor* w) {
  w->x = j.x;
  w->out = j.out;
  w->xt = j.xt;
  w->xh = j.xh;
  w->ob = j.ob;
  w->orow = j.orow;
  w->oh = j.oh;
  w->rows = j.rows;
  w->num_rows = j.num_rows;
  w->weight = j.norm.weight;
  w->bias = j.norm.bias;
  w->eps = j.norm.eps;
  w->inv_d = 1.f / static_cast<float>(j.head_dim);
  w->kind = j.norm.kind;
  w->weight_fp32 = j.norm.fp32;
  w->weight_vec = j.vec && aligned(j.norm.weight, 16) && aligned(j.norm.bias, 16) ? 1 : 0;
  w->n_heads = j.n_heads;
  w->rot_off = j.rot_off;
  w->pairs = j.rot_dim / 2;
  w->half = half ? 1 : 0;
  const int width = !j.vec ? 1 : (dtype == MLA_ROPE_FP32 ? 4 : 8);
  if (j.vec && !half) {
    w->rot_units = j.rot_dim > 0 ? 1 : 0;  // there are some
    w->units = j.head_dim / width;
  } else {
    w->rot_units = j.rot_dim / 2 / width;
    w->units = w->rot_units + (j.head_dim - j.rot_dim) / width;
  }
  w->per_lane = j.vec ? kUnits : w->units <= 32 * kFewUnits ? kFewUnits : kSingleUnits;
  w->lanes = 1;
  while (w->lanes < 32 && w->lanes < w->units) w->lanes *= 2;
  w->chunks = (w->units + w->lanes * w->per_lane - 1) / (w->lanes * w->per_lane);
  const int rows = kThreads / w->lanes;
  w->tok_rows = std::min(rows, T);
  w->head_rows = std::min(rows / w->tok_rows, j.n_heads);
  // several heads per group once there are blocks for all places of the GPU
  const int64_t toks = (static_cast<int64_t>(T) + w->tok_rows - 1) / w->tok_rows;
  const int turns = (j.n_heads + w->head_rows - 1) / w->head_rows;
  const int most = std::min(turns, kMaxPasses);
  w->passes = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, (toks * turns + 607) / 608)));
  w->head_blocks = std::max(std::max(1, (turns + w->passes / 2) / w->passes), (turns + kMaxPasses - 1) / kMaxPasses);
  w->passes = (turns + w->head_blocks - 1) / w->head_blocks;  // even shares
  const int64_t blocks = toks * w->head_blocks;
  if (blocks >= (1ll << 29)) return fail(MLA_ERR_SHAPE, "%s: T x heads too large", j.name);
  w->blocks = static_cast<int>(blocks);
  return MLA_OK;
}

typedef void (*Kernel)(Params);
template <typename E>
Kernel kernel_of(int per_lane, bool layer) {
  constexpr int V = 16 / sizeof(E);
  if (per_lane == kUnits) return layer ? head_prep_kernel<E, V, kUnits, true> : head_prep_kernel<E, V, kUnits, false>;
  if (per_lane == kFewUnits) return layer ? head_prep_kernel<E, 1, kFewUnits, true> : head_prep_kernel<E, 1, kFewUnits, false>;
  return layer ? head_prep_kernel<E, 1, kSingleUnits, true> : head_prep_kernel<E, 1, kSingleUnits, false>;
}

mla_status launch(const Job* jobs, int n, int T, int dtype, bool half, Params& p, cudaStream_t s) {
  p.T = T;
  // a launch for the tensors of each kind of access
  for (int per_lane : {kUnits, kSingleUnits, kFewUnits}) {
    int taken = 0, by[3] = {0, 1, 2};
    int64_t grid = 0;
    bool layer = false;
    // those of most heads first: their blocks take longest
    std::sort(by, by + n, [&](int a, int b) { return jobs[a].n_heads > jobs[b].n_heads; });
    for (int i = 0; i < 3; ++i) p.t[i].blocks = 0;
    for (int o = 0; o < n; ++o) {
      const Job& j = jobs[by[o]];
      Tensor w = {};
      const mla_status st = split_job(j, T, dtype, half, &w);
      if (st != MLA_OK) return st;
      if (w.per_lane != per_lane) continue;
      layer = layer || j.norm.kind == MLA_NORM_LAYER;
      grid += w.blocks;
      p.t[taken++] = w;
    }
    if (taken == 0) continue;
    const Kernel kernel = dtype == MLA_ROPE_BF16   ? kernel_of<__nv_bfloat16>(per_lane, layer)
                          : dtype == MLA_ROPE_FP16 ? kernel_of<__half>(per_lane, layer)
                                                   : kernel_of<float>(per_lane, layer);
    kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    HEADS_CUDA(cudaGetLastError(), "launch");
  }
  return MLA_OK;
}

mla_head_norm norm_of(const mla_head_norm* n) {
  mla_head_norm none = {nullptr, nullptr, MLA_NORM_NONE, 0, 0.f, 0};
  return n != nullptr ? *n : none;
}

Job rope_job(const char* name, const mla_rope_tensor& q, const mla_head_norm* norm, int T, int rot_dim) {
  Job j;
  j.name = name;
  j.x = q.x;
  j.xt = q.x_token_stride;
  j.xh = q.x_head_stride;
  j.out = q.out;
  j.orow = q.out_token_stride;
  j.ob = q.out_token_stride <= kMost / 128 ? 128 * q.out_token_stride : kMost + 1;
  j.oh = q.out_head_stride;
  j.rows = q.rows;
  j.num_rows = q.rows ? q.num_rows : T;
  j.n_heads = q.n_heads;
  j.head_dim = q.head_dim;
  j.rot_off = q.rot_off;
  j.rot_dim = rot_dim;
  j.norm = norm_of(norm);
  j.vec = false;
  return j;
}

// The scheme of a call that may rotate nothing.
mla_status make_scheme(const mla_rope_params* params, int rot_dim, Freqs* f) {
  return rot_dim == 0 ? MLA_OK : mlarp::make_freqs(params, rot_dim, f, fail);
}

}  // namespace
}  // namespace mlaheads

extern "C" {

mla_status mla_norm_rope(const mla_rope_dims* dims, const mla_rope_params* params, const int32_t* positions,
                         const mla_rope_tensor* q, const mla_head_norm* q_norm, const mla_rope_tensor* k,
                         const mla_head_norm* k_norm, void* stream) {
  using namespace mlaheads;
  no_error();
  if (dims == nullptr || q == nullptr) return fail(MLA_ERR_NULL, "dims or q is NULL");
  const mla_rope_dims d = *dims;
  if (d.dtype < MLA_ROPE_BF16 || d.dtype > MLA_ROPE_FP32) return fail(MLA_ERR_DTYPE, "dtype %d unknown", d.dtype);
  if (d.T < 0 || d.half < 0 || d.half > 1) return fail(MLA_ERR_SHAPE, "T must be >= 0, half 0 or 1");
  if (d.inverse != 0) return fail(MLA_ERR_UNSUPPORTED, "inverse must be 0");
  Params p;
  mla_status st = make_scheme(params, d.rot_dim, &p.f);
  if (st != MLA_OK) return st;
  if (d.T == 0) return MLA_OK;
  if (d.rot_dim > 0 && !positions) return fail(MLA_ERR_NULL, "positions is NULL");
  if (!aligned(positions, 4)) return fail(MLA_ERR_ALIGN, "positions must be 4-byte aligned");
  Job jobs[2] = {rope_job("q", *q, q_norm, d.T, d.rot_dim), {}};
  const int n = k != nullptr ? 2 : 1;
  if (n == 2) jobs[1] = rope_job("k", *k, k_norm, d.T, d.rot_dim);
  for (int i = 0; i < n && st == MLA_OK; ++i) st = check_job(jobs[i], d.T, d.dtype, d.half != 0, false);
  if (st == MLA_OK) st = check_overlaps(jobs, n, d.T, d.rot_dim ? positions : nullptr, q->rows, d.dtype);
  if (st == MLA_OK && n == 2 && k->rows) st = check_overlaps(jobs, n, d.T, nullptr, k->rows, d.dtype);
  if (st != MLA_OK) return st;
  p.positions = positions;
  return launch(jobs, n, d.T, d.dtype, d.half != 0, p, static_cast<cudaStream_t>(stream));
}

mla_status mla_kv_append(const mla_append_dims* dims, const mla_rope_params* params, const int32_t* positions,
                         const int64_t* rows, const mla_append_input* k, const mla_head_norm* k_norm,
                         const mla_kv_cache* k_cache, const mla_append_input* v, const mla_kv_cache* v_cache,
                         const mla_rope_tensor* q, const mla_head_norm* q_norm, void* stream) {
  using namespace mlaheads;
  no_error();
  if (!dims || !k || !k_cache || !v || !v_cache) return fail(MLA_ERR_NULL, "dims, k, v or a cache is NULL");
  const mla_append_dims d = *dims;
  if (d.dtype < MLA_ROPE_BF16 || d.dtype > MLA_ROPE_FP32) return fail(MLA_ERR_DTYPE, "dtype %d unknown", d.dtype);
  if (d.T < 0 || d.half < 0 || d.half > 1) return fail(MLA_ERR_SHAPE, "T must be >= 0, half 0 or 1");
  if (d.num_blocks < 1 || d.num_blocks >= (1 << 24))
    return fail(MLA_ERR_SHAPE, "num_blocks=%d outside [1, 2^24)", d.num_blocks);
  if (q != nullptr && q->rows != nullptr) return fail(MLA_ERR_UNSUPPORTED, "q's rows must be NULL");
  Params p;
  mla_status st = make_scheme(params, d.rot_dim, &p.f);
  if (st != MLA_OK) return st;
  if (d.T == 0) return MLA_OK;
  if (!rows || (d.rot_dim > 0 && !positions)) return fail(MLA_ERR_NULL, "rows or positions is NULL");
  if (!aligned(positions, 4)) return fail(MLA_ERR_ALIGN, "positions must be 4-byte aligned");
  Job jobs[3];
  const mla_append_input* in[2] = {k, v};
  const mla_kv_cache* cache[2] = {k_cache, v_cache};
  for (int i = 0; i < 2; ++i) {
    Job& j = jobs[i];
    j.name = i == 0 ? "k" : "v";
    j.x = in[i]->x;
    j.xt = in[i]->token_stride;
    j.xh = in[i]->head_stride;
    j.out = cache[i]->data;
    j.ob = cache[i]->block_stride;
    j.orow = cache[i]->row_stride;
    j.oh = cache[i]->head_stride;
    j.rows = rows;
    j.num_rows = 128ll * d.num_blocks;
    j.n_heads = d.n_kv;
    j.head_dim = i == 0 ? d.d_qk : d.d_v;
    j.rot_off = i == 0 ? d.rot_off : 0;
    j.rot_dim = i == 0 ? d.rot_dim : 0;
    j.norm = norm_of(i == 0 ? k_norm : nullptr);
    j.vec = false;
  }
  int n = 2;
  if (q != nullptr) jobs[n++] = rope_job("q", *q, q_norm, d.T, d.rot_dim);
  for (int i = 0; i < n && st == MLA_OK; ++i) st = check_job(jobs[i], d.T, d.dtype, d.half != 0, i < 2);
  if (st == MLA_OK) st = check_overlaps(jobs, n, d.T, d.rot_dim ? positions : nullptr, rows, d.dtype);
  if (st != MLA_OK) return st;
  p.positions = positions;
  return launch(jobs, n, d.T, d.dtype, d.half != 0, p, static_cast<cudaStream_t>(stream));
}

const char* mla_heads_last_error(void) { return mlaheads::g_error; }

mla_status mla_heads_device_status(void* stream, uint32_t* flags, int32_t clear) {
  using namespace mlaheads;
  no_error();
  HEADS_CUDA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)), "cudaStreamSynchronize");
  unsigned int all = 0;
  for (auto read : {prep_status, prompt_status, paged_status}) {
    unsigned int v = 0;
    HEADS_CUDA(read(&v, clear != 0), "the status word");
    all |= v;
  }
  if (flags) *flags = all;
  if (all != 0) return fail(MLA_ERR_DEVICE_STATUS, "heads device status 0x%x", all);
  return MLA_OK;
}

}  // extern "C"
