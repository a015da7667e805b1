// Rotary positions for GB300 (sm_103a): cosine / sine tables and the rotation
// of heads (formulas in mla_rope.h).
//
// Angles.  A pair's frequency is kept as a 64-bit fixed-point fraction of a
// turn per position, so position * frequency modulo 2^64 is the angle modulo
// whole turns, exactly, at the cost of one 64-bit multiply: no fp64 (slow
// here) and no loss at far positions.  Read as a signed fraction of a turn it
// converts to fp32 with full relative precision, and sincospif takes it.
//
// The rotation is bound by memory.  A block takes some tokens (their angles go
// to shared memory once, for all heads) and some heads; each thread moves four
// 16-byte units per pass, loaded before the angles are needed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "../../include/mla_rope.h"

namespace mlarp {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;      // rot_dim <= 256
constexpr int kMaxBlockPairs = 1024;  // (token, pair) angles of a block
constexpr int kUnroll = 4;

__device__ unsigned int g_rope_status = 0;

struct Freqs {
  uint64_t turn[kMaxPairs];  // turns per position, 64-bit fraction
  float mscale;
};

// cos and sin of position * frequency, times mscale.
__device__ __forceinline__ float2 cos_sin(int32_t pos, uint64_t turn, float mscale) {
  const int64_t frac = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(pos)) * turn);
  float s, c;
  sincospif(static_cast<float>(frac) * 0x1p-63f, &s, &c);
  return make_float2(c * mscale, s * mscale);
}

struct TableParams {
  Freqs f;
  const int32_t* positions;
  float* cos;
  float* sin;
  int T, pairs;
};

__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ TableParams p) {
  __shared__ uint64_t turn[kMaxPairs];
  if (threadIdx.x < p.pairs) turn[threadIdx.x] = p.f.turn[threadIdx.x];
  __syncthreads();
  const int64_t n = static_cast<int64_t>(p.T) * p.pairs;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e < n;
       e += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int t = static_cast<int>(e / p.pairs), i = static_cast<int>(e - static_cast<int64_t>(t) * p.pairs);
    const float2 v = cos_sin(__ldg(p.positions + t), turn[i], p.f.mscale);
    p.cos[e] = v.x;
    p.sin[e] = v.y;
  }
}

struct Tensor {
  const void* x;
  void* out;
  int64_t xt, xh, ot, oh;  // strides in elements
  const int64_t* rows;
  int64_t num_rows;
  int n_heads, head_dim, rot_off;
  int vec;          // 16-byte units
  int in_place;     // the part outside the rotation is left alone
  int rot_units;    // units of a head that hold rotated values
  int units;        // all units of a head
  int tokens;       // tokens of a block
  int heads;        // heads of a block
  int head_blocks;  // blocks per group of tokens
  int blocks;
};

struct Params {
  Freqs f;
  const int32_t* positions;
  Tensor t[2];
  int T, pairs, half, inverse;
};

template <typename E>
__device__ __forceinline__ float to_f(E v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E>
__device__ __forceinline__ E from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

template <typename E, int V>
struct alignas(sizeof(E) * V) Pack {
  E e[V];
};

// A unit of the half layout (both layouts for V = 1) is two packs: V values of
// the first half and the V that turn with them; any other unit is one pack.
template <typename E, int V>
struct Unit {
  Pack<E, V> a, b;
};

template <typename E, int V>
__device__ void rotate_block(const Params& p, const Tensor& w, int block, float2* angles) {
  const int tid = threadIdx.x;
  const int t0 = block / w.head_blocks * w.tokens, h0 = block % w.head_blocks * w.heads;
  const int nt = min(w.tokens, p.T - t0), nh = min(w.heads, w.n_heads - h0);
  const bool two = V == 1 || p.half;  // rotated units are two packs
  const int rot = w.rot_off, pairs = p.pairs;
  const int n = nt * nh * w.units;
  const int second = p.half ? pairs : 1;  // distance of a pair's values

  // where unit u of this block starts: element offsets in x and out, its token
  // and rotated pair (-1: copied)
  struct Place {
    int64_t x, o;
    int at;  // index of its first angle, -1 when copied
  };
  auto place = [&](int u) {
    const int k = u % w.units, r = u / w.units;
    const int h = r % nh, t = r / nh;
    Place q;
    int d;
    if (k < w.rot_units) {
      const int pr = V == 1 ? k : (p.half ? k * V : k * V / 2);  // first pair
      d = rot + (p.half ? pr : 2 * pr);
      q.at = t * pairs + pr;
    } else {
      const int c = (k - w.rot_units) * V;  // copied values, in order
      d = c < rot ? c : c + 2 * pairs;
      q.at = -1;
    }
    const int64_t tok = t0 + t;
    q.x = tok * w.xt + static_cast<int64_t>(h0 + h) * w.xh + d;
    int64_t row = tok;
    if (w.rows != nullptr) row = __ldg(w.rows + tok);
    q.o = row < 0 || (w.rows != nullptr && row >= w.num_rows)
              ? -1
              : row * w.ot + static_cast<int64_t>(h0 + h) * w.oh + d;
    return q;
  };
  const E* x = static_cast<const E*>(w.x);
  E* out = static_cast<E*>(w.out);
  auto load = [&](const Place& q) {
    Unit<E, V> v;
    v.a = *reinterpret_cast<const Pack<E, V>*>(x + q.x);
    v.b = v.a;
    if (two && q.at >= 0) v.b = *reinterpret_cast<const Pack<E, V>*>(x + q.x + second);
    return v;
  };

  // the first units are on their way while the angles are made
  Place q[kUnroll];
  Unit<E, V> v[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k)
    if (tid + k * kThreads < n) {
      q[k] = place(tid + k * kThreads);
      v[k] = load(q[k]);
    }
  if (w.rows != nullptr && h0 == 0)
    for (int t = tid; t < nt; t += kThreads)
      if (__ldg(w.rows + t0 + t) >= w.num_rows) atomicOr(&g_rope_status, MLA_DEVICE_BAD_BLOCK);
  for (int e = tid; e < nt * pairs; e += kThreads) {
    const int t = e / pairs;
    float2 cs = cos_sin(__ldg(p.positions + t0 + t), p.f.turn[e - t * pairs], p.f.mscale);
    if (p.inverse) cs.y = -cs.y;
    angles[e] = cs;
  }
  __syncthreads();
  for (int u0 = tid; u0 < n; u0 += kUnroll * kThreads) {
    if (u0 != tid) {
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (u0 + k * kThreads < n) {
          q[k] = place(u0 + k * kThreads);
          v[k] = load(q[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (u0 + k * kThreads >= n || q[k].o < 0) continue;
      if (q[k].at < 0) {
        *reinterpret_cast<Pack<E, V>*>(out + q[k].o) = v[k].a;
        continue;
      }
      if (two) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 cs = angles[q[k].at + i];
          const float a = to_f(v[k].a.e[i]), b = to_f(v[k].b.e[i]);
          v[k].a.e[i] = from_f<E>(a * cs.x - b * cs.y);
          v[k].b.e[i] = from_f<E>(a * cs.y + b * cs.x);
        }
        *reinterpret_cast<Pack<E, V>*>(out + q[k].o) = v[k].a;
        *reinterpret_cast<Pack<E, V>*>(out + q[k].o + second) = v[k].b;
      } else {
#pragma unroll
        for (int i = 0; i + 1 < V; i += 2) {
          const float2 cs = angles[q[k].at + i / 2];
          const float a = to_f(v[k].a.e[i]), b = to_f(v[k].a.e[i + 1]);
          v[k].a.e[i] = from_f<E>(a * cs.x - b * cs.y);
          v[k].a.e[i + 1] = from_f<E>(a * cs.y + b * cs.x);
        }
        *reinterpret_cast<Pack<E, V>*>(out + q[k].o) = v[k].a;
      }
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Params p) {
  __shared__ float2 angles[kMaxBlockPairs];
  const int second = static_cast<int>(blockIdx.x) >= p.t[0].blocks;
  const int block = static_cast<int>(blockIdx.x) - (second ? p.t[0].blocks : 0);
  const Tensor& w = p.t[second];
  if (w.vec) rotate_block<E, 16 / sizeof(E)>(p, w, block, angles);
  else rotate_block<E, 1>(p, w, block, angles);
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

// Checks the scheme and fills the fixed-point turns per position.
mla_status make_freqs(const mla_rope_params* q, int rot, mlarp::Freqs* f) {
  if (q == nullptr) return rope_fail(MLA_ERR_NULL, "params is NULL");
  if (rot < 2 || rot > 2 * mlarp::kMaxPairs || (rot & 1))
    return rope_fail(MLA_ERR_SHAPE, "rot_dim=%d must be even, in [2, 256]", rot);
  if (q->scaling < MLA_ROPE_NONE || q->scaling > MLA_ROPE_YARN)
    return rope_fail(MLA_ERR_SHAPE, "scaling %d unknown", q->scaling);
  if (!(q->theta > 1.0) || !isfinite(q->theta)) return rope_fail(MLA_ERR_SHAPE, "theta must be finite and above 1");
  if (!(q->mscale > 0.0) || !isfinite(q->mscale)) return rope_fail(MLA_ERR_SHAPE, "mscale must be finite and above 0");
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

// Checks one tensor and splits its work into blocks of about kThreads * kUnroll units.
mla_status make_tensor(const mla_rope_tensor* q, const mla_rope_dims& d, const char* name, mlarp::Tensor* w) {
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
  const int64_t parts[] = {q->x_token_stride, q->x_head_stride,  q->out_token_stride, q->out_head_stride,
                           q->head_dim,       q->rot_off,        d.half ? d.rot_dim / 2 : d.rot_dim};
  w->vec = aligned(q->x, 16) && aligned(q->out, 16);
  for (int64_t v : parts) w->vec = w->vec && v % V == 0;
  w->x = q->x;
  w->out = q->out;
  w->xt = q->x_token_stride;
  w->xh = q->x_head_stride;
  w->ot = q->out_token_stride;
  w->oh = q->out_head_stride;
  w->rows = q->rows;
  w->num_rows = q->num_rows;
  w->n_heads = q->n_heads;
  w->head_dim = q->head_dim;
  w->rot_off = q->rot_off;
  w->in_place = same;
  const int width = w->vec ? V : 1;
  w->rot_units = w->vec && !d.half ? d.rot_dim / V : d.rot_dim / 2 / width;
  w->units = w->rot_units + (same ? 0 : (q->head_dim - d.rot_dim) / width);
  const int goal = mlarp::kThreads * mlarp::kUnroll;
  w->heads = std::min(q->n_heads, std::max(1, goal / w->units));
  w->head_blocks = (q->n_heads + w->heads - 1) / w->heads;
  w->tokens = w->head_blocks > 1 ? 1 : std::max(1, goal / (w->units * w->heads));
  w->tokens = std::min({w->tokens, mlarp::kMaxBlockPairs / (d.rot_dim / 2), d.T});
  const int64_t blocks = (static_cast<int64_t>(d.T) + w->tokens - 1) / w->tokens * w->head_blocks;
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
  p.positions = positions;
  p.cos = cos;
  p.sin = sin;
  p.T = T;
  p.pairs = rot_dim / 2;
  const int64_t n = static_cast<int64_t>(T) * p.pairs;
  const int64_t want = (n + mlarp::kThreads - 1) / mlarp::kThreads;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(want, 152 * 8));
  mlarp::rope_table_kernel<<<grid, mlarp::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
  st = make_tensor(q, d, "q", &p.t[0]);
  if (st != MLA_OK) return st;
  p.t[1] = p.t[0];
  p.t[1].blocks = 0;
  if (k != nullptr) {
    st = make_tensor(k, d, "k", &p.t[1]);
    if (st != MLA_OK) return st;
  }
  p.positions = positions;
  p.T = d.T;
  p.pairs = d.rot_dim / 2;
  p.half = d.half;
  p.inverse = d.inverse;
  const unsigned grid = static_cast<unsigned>(p.t[0].blocks + p.t[1].blocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d.dtype == MLA_ROPE_BF16) mlarp::rope_kernel<__nv_bfloat16><<<grid, mlarp::kThreads, 0, s>>>(p);
  else if (d.dtype == MLA_ROPE_FP16) mlarp::rope_kernel<__half><<<grid, mlarp::kThreads, 0, s>>>(p);
  else mlarp::rope_kernel<float><<<grid, mlarp::kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return rope_fail(MLA_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
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
