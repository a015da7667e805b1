// Attention of new tokens over a paged cache of keys and values for GB300
// (sm_103a); formulas in mla_heads.h.
//
// The keys and values of a sequence are read once and meet few rows (the S1 new
// tokens of the G heads that share them), so memory binds.  One warp of a CTA
// streams units of 64 keys, key and value together, by TMA through a ring that
// fills shared memory, on and on across sequences and heads; two groups of four
// warps take units in turn.  The warps of a group split a unit: by 16 rows, and
// by keys where there are fewer than 64 rows.  Each keeps its rows' running
// maximum, sum and output in registers, as accumulators of mma.sync (m16n8k16:
// with 16 rows the 128-row tiles of tcgen05 would be an eighth full, and a
// unit's products take a third of the time that its bytes take to arrive); they
// meet in shared memory when a sequence's head is through.
//
// The units of all sequences and heads are one stream of which every CTA takes
// an equal share.  A head cut between CTAs leaves partial states in the
// workspace, and a second launch joins them.  Which CTA takes what follows from
// the lengths alone, so results do not depend on timing.  Calls of more than 64
// rows to a key head go through the 128-row tiles of prompts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "heads.h"
#include "heads_device.cuh"

namespace mlaheads {
namespace paged {

__device__ unsigned int g_paged_status = 0;

constexpr int kUnit = 64;        // keys
constexpr int kConsumers = 8;    // warps
constexpr int kGroups = 2;
constexpr int kLoadWarp = 8;
constexpr int kThreads = 288;
constexpr int kChunk = 8192;     // 64 rows of 128 bytes
constexpr int kMaxStages = 16;
constexpr int kMaxRows = 64;
constexpr int kCols = 32;        // columns that the warps join at a time
constexpr int kPitch = kCols + 4;

constexpr int kFull = 0;                      // [kMaxStages]
constexpr int kEmpty = kFull + kMaxStages;    // [kMaxStages]
constexpr int kSegFull = kEmpty + kMaxStages; // [2] a segment's Q has landed, its description is written
constexpr int kSegEmpty = kSegFull + 2;       // [2]
constexpr int kJoin = kSegEmpty + 2;          // the consumers have come this far
constexpr int kNumBars = kJoin + 1;

// A run of units of one sequence and key head.
struct Segment {
  int b, hk;         // b < 0: no more
  int u0, u1, units; // units [u0, u1) of `units`
  int n, len, pos;   // query tokens, keys within the table, position of token 0
};

constexpr int kOffJoin = 0;                                              // float [kConsumers][16][kPitch]
constexpr int kOffMl = kOffJoin + kConsumers * 16 * kPitch * 4;          // float2 [kConsumers][16]
constexpr int kOffScan = kOffMl + kConsumers * 16 * 8;                   // int64 [kThreads / 32]
constexpr int kOffWalk = kOffScan + kThreads / 32 * 8;                   // int64 [2]
constexpr int kOffSeg = kOffWalk + 16;                                   // Segment [2]
constexpr int kOffGood = kOffSeg + 2 * static_cast<int>(sizeof(Segment));  // int [kMaxStages]
constexpr int kOffBars = kOffGood + kMaxStages * 4;
constexpr int kOffAbort = kOffBars + 8 * kNumBars;
constexpr int kOffMended = kOffAbort + 4;
constexpr int kOffTiles = (kOffMended + 4 + 1023) & ~1023;  // Q twice, then the ring
constexpr int kSmemMost = 232448;
static_assert(kOffBars % 8 == 0 && kOffWalk % 8 == 0, "alignment");

struct Params {
  Problem x;
  float* parts;    // [CTAs][2][part_floats]
  int4* records;   // [CTAs] the head whose first part is the CTA's last: sequence, key head, parts behind it
  int part_floats;
  int G, rows;     // heads to a key head, rows of a key head
  int kc, vc;      // 64-column chunks of keys and values
  int ks, vs;      // 16-column steps
  int stages, stage_bytes, q_bytes;
  int ctas;
  unsigned long long wait_ns;
};
struct Maps {
  CUtensorMap q, k, v;
};

struct Seq {
  int n, len, pos, units;
  bool cut_table;
};
__device__ __forceinline__ Seq load_seq(const Params& p, int b) {
  Seq s;
  const int act = max(0, __ldg(p.x.act_seqs + b));
  s.n = p.x.q_lens != nullptr ? min(p.x.S1, max(0, __ldg(p.x.q_lens + b))) : p.x.S1;
  s.len = min(act, p.x.W * kPage);
  s.cut_table = s.len < act && s.n > 0;
  s.pos = act - s.n;
  s.units = s.n > 0 ? max(1, (s.len + kUnit - 1) / kUnit) : 1;  // rows that see nothing are written too
  return s;
}

struct Ctx {
  uint32_t sb;
  uint8_t* smem;
  uint64_t wait_ns;
  volatile uint32_t* abort;
  __device__ uint32_t bar(int i) const { return sb + kOffBars + 8 * i; }
  __device__ volatile uint32_t* mended() const { return reinterpret_cast<volatile uint32_t*>(smem + kOffMended); }
};

// Units of a CTA at least: fewer parts to join where there is little to read.
constexpr int kMinUnits = 2;

__device__ __forceinline__ int ctas_of(const Params& p, int64_t total) {
  return static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(p.ctas), total / kMinUnits)));
}

// Where the CTA's share of the stream begins; false when it has none.
__device__ bool start(const Params& p, const Ctx& c, int& b0, int64_t& base, int64_t& from, int64_t& to, int64_t& total, int& ctas) {
  int64_t* part = reinterpret_cast<int64_t*>(c.smem + kOffScan);
  int64_t* at = reinterpret_cast<int64_t*>(c.smem + kOffWalk);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.x.B;
  const int chunks = (B + kThreads - 1) / kThreads;
  auto scan = [&](int64_t v, int64_t& sum) {  // over the threads before this one, and over the block
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int64_t before = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += part[w];
      sum += part[w];
    }
    return before + x - v;
  };
  int64_t mine = 0, len = 0, pre = 0;
  bool cut = false;
  for (int k = 0; k < chunks; ++k) {
    const int b = k * kThreads + tid;
    len = 0;
    if (b < B) {
      const Seq s = load_seq(p, b);
      len = static_cast<int64_t>(s.units) * p.x.n_kv;
      cut = cut || s.cut_table;
    }
    mine += len;
  }
  if (cut) atomicOr(&g_paged_status, MLA_DEVICE_BAD_BLOCK);
  pre = scan(mine, total);
  ctas = ctas_of(p, total);
  const int cid = blockIdx.x;
  if (cid >= ctas) return false;
  from = cid * total / ctas;
  to = (cid + 1) * total / ctas;
  int64_t carry = 0;
  for (int k = 0; k < chunks; ++k) {
    const int b = k * kThreads + tid;
    int64_t sum = total;
    if (chunks > 1) {
      len = b < B ? static_cast<int64_t>(load_seq(p, b).units) * p.x.n_kv : 0;
      pre = carry + scan(len, sum);
    }
    if (b < B && from >= pre && from < pre + len) {
      at[0] = b;
      at[1] = pre;
    }
    carry += sum;
    if (carry > from) break;
  }
  __syncthreads();
  b0 = static_cast<int>(at[0]);
  base = at[1];
  return from < to;
}

__device__ void load_role(const Params& p, const Ctx& c, const Maps& maps, int b, int64_t base, int64_t from, int64_t to) {
  const int lane = threadIdx.x & 31;
  const uint32_t ring = c.sb + kOffTiles + 2 * p.q_bytes;
  int stage = 0;
  uint32_t phase = 1, segs = 0;
  bool bad = false;
  auto publish = [&](const Segment& s) {
    const int k = segs & 1;
    if (!warp_wait(c, kSegEmpty + k, ((segs >> 1) & 1) ^ 1)) return false;
    if (lane == 0) {
      reinterpret_cast<Segment*>(c.smem + kOffSeg)[k] = s;
      if (s.b >= 0) {
        mbar_arrive_expect_tx(c.bar(kSegFull + k), p.kc * p.rows * 128);
        for (int i = 0; i < p.kc; ++i)
          tma_3d(c.sb + kOffTiles + k * p.q_bytes + i * (p.q_bytes / p.kc), &maps.q, 64 * i, s.hk * p.G, s.b * p.x.S1, c.bar(kSegFull + k));
      } else {
        mbar_arrive(c.bar(kSegFull + k));
      }
    }
    __syncwarp();
    ++segs;
    return true;
  };
  while (from < to) {
    const Seq q = load_seq(p, b);
    const int64_t len = static_cast<int64_t>(q.units) * p.x.n_kv;
    if (from - base >= len) {
      base += len;
      ++b;
      continue;
    }
    Segment s;
    s.b = b;
    s.hk = static_cast<int>((from - base) / q.units);
    s.units = q.units;
    s.u0 = static_cast<int>(from - base - static_cast<int64_t>(s.hk) * q.units);
    s.u1 = static_cast<int>(min(static_cast<int64_t>(q.units), s.u0 + to - from));
    s.n = q.n;
    s.len = q.len;
    s.pos = q.pos;
    if (!publish(s)) return;
    int ids = -1;
    for (int u = s.u0; u < s.u1; ++u) {
      const int page = u >> 1;
      if (u == s.u0 || ((u & 1) == 0 && ((page - (s.u0 >> 1)) & 31) == 0)) {  // the next 32 pages
        const int at = page + lane;
        ids = at < p.x.W && at * kPage < q.len ? __ldg(p.x.block_table + static_cast<int64_t>(b) * p.x.W + at) : -1;
      }
      const int id = __shfl_sync(0xffffffffu, ids, (page - (s.u0 >> 1)) & 31);
      const bool good = id >= 0 && id < p.x.num_blocks;
      bad = bad || (!good && u * kUnit < q.len && q.n > 0);
      if (!warp_wait(c, kEmpty + stage, phase)) return;
      if (lane == 0) {
        reinterpret_cast<volatile int*>(c.smem + kOffGood)[stage] = good ? 1 : 0;
        const uint32_t bar = c.bar(kFull + stage), dst = ring + stage * p.stage_bytes;
        const int row = (u & 1) * kUnit, block = good ? id : p.x.num_blocks;  // beyond the pool: zeros
        mbar_arrive_expect_tx(bar, p.stage_bytes);
        for (int i = 0; i < p.kc; ++i) tma_4d(dst + i * kChunk, &maps.k, 64 * i, row, s.hk, block, bar);
        for (int i = 0; i < p.vc; ++i) tma_4d(dst + (p.kc + i) * kChunk, &maps.v, 64 * i, row, s.hk, block, bar);
      }
      __syncwarp();
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    from += s.u1 - s.u0;
  }
  Segment none = {};
  none.b = -1;
  publish(none);
  if (bad && lane == 0) atomicOr(&g_paged_status, MLA_DEVICE_BAD_BLOCK);
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
template <typename E>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (__is_same(E, __half))
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether column `col` of a value that a row sees, key by key in [lo, hi), is not finite.
template <typename E>
__device__ __noinline__ bool infinite_column(const Params& p, const Segment& s, int lo, int hi, int col) {
  constexpr uint32_t kExp = __is_same(E, __half) ? 0x7C00u : 0x7F80u;
  for (int key = lo; key < hi; ++key) {
    const int id = __ldg(p.x.block_table + static_cast<int64_t>(s.b) * p.x.W + key / kPage);
    if (id < 0 || id >= p.x.num_blocks) continue;
    const uint16_t v = __ldg(static_cast<const uint16_t*>(p.x.v.data) + id * p.x.v.block_stride + (key % kPage) * p.x.v.row_stride +
                             s.hk * p.x.v.head_stride + col);
    if ((v & kExp) == kExp) return true;
  }
  return false;
}

// kTiles: 16-row tiles of a key head's rows, 1, 2 or 4.  kV: 8-column tiles of the values, 8 or 16.
template <typename E, int kTiles, int kV>
__device__ void consume_role(const Params& p, const Ctx& c, int warp, int lane, int ctas, int64_t total) {
  constexpr int kSplits = 4 / kTiles;        // warps of a group that share a row tile
  constexpr int kKeys = kUnit / kSplits;     // keys of a warp
  constexpr int kN = kKeys / 8;              // 8-key tiles of a warp
  constexpr int kStates = kGroups * kSplits; // states of a row
  const int group = warp >> 2, tile = (warp & 3) % kTiles, split = (warp & 3) / kTiles;
  const int quad = lane & 3, row0 = lane >> 2;  // the thread's rows: row0 and row0 + 8 of the tile
  const float scale = p.x.scale_log2;
  const bool raw = scale > 0.f;
  const float mul = raw ? scale : 1.f;
  const uint32_t ring = c.sb + kOffTiles + 2 * p.q_bytes;
  float* join = reinterpret_cast<float*>(c.smem + kOffJoin);
  float2* ml = reinterpret_cast<float2*>(c.smem + kOffMl);
  uint32_t unit_count = 0, joins = 0;  // of the CTA
  auto meet = [&]() {  // of the consumers; bounded like every wait
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(kJoin));
    return warp_wait(c, kJoin, joins++ & 1);
  };
  int stage = 0;
  uint32_t phase = 0;
  for (uint32_t segs = 0;; ++segs) {
    const int k2 = segs & 1;
    if (!warp_wait(c, kSegFull + k2, (segs >> 1) & 1)) return;
    const Segment s = reinterpret_cast<const Segment*>(c.smem + kOffSeg)[k2];
    if (s.b < 0) return;
    int vis[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tok = (tile * 16 + row0 + 8 * i) / p.G;
      vis[i] = tile * 16 + row0 + 8 * i < p.rows && tok < s.n ? min(s.len, max(0, s.pos + tok + 1)) : 0;
    }
    const int lo = min(s.len, max(0, s.pos + 1));  // keys that every token sees
    const uint32_t qs = c.sb + kOffTiles + k2 * p.q_bytes;
    float o[kV][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kV; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    for (int u = s.u0; u < s.u1; ++u, ++unit_count) {
      const int at_stage = stage;
      const uint32_t at_phase = phase;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
      if ((unit_count & 1) != static_cast<uint32_t>(group)) continue;
      if (!warp_wait(c, kFull + at_stage, at_phase)) return;
      const uint32_t ks = ring + at_stage * p.stage_bytes, vs = ks + p.kc * kChunk;
      const bool good = reinterpret_cast<volatile int*>(c.smem + kOffGood)[at_stage] != 0;
      const int key0 = split * kKeys;            // within the unit
      const int first = u * kUnit + key0;        // key of column 0
      const bool edge = !good || first + kKeys > lo;
      float z[kN][4];
#pragma unroll
      for (int n = 0; n < kN; ++n) z[n][0] = z[n][1] = z[n][2] = z[n][3] = 0.f;
      // scores: rows of Q against rows of K, 16 values at a time
      const int q_row = tile * 16 + (lane & 15), q_half = lane >> 4;
      const int k_row = key0 + (lane & 7) + ((lane >> 4) << 3), k_half = (lane >> 3) & 1;
#pragma unroll 4
      for (int k = 0; k < p.ks; ++k) {
        uint32_t a[4];
        ldsm(a, qs + (k >> 2) * (kTiles * 16 * 128) + q_row * 128 + (((2 * (k & 3) + q_half) ^ (q_row & 7)) << 4));
#pragma unroll
        for (int n = 0; n < kN; n += 2) {
          uint32_t b[4];
          const int r = k_row + 8 * n;
          ldsm(b, ks + (k >> 2) * kChunk + r * 128 + (((2 * (k & 3) + k_half) ^ (r & 7)) << 4));
          mma<E>(z[n], a, b[0], b[1]);
          mma<E>(z[n + 1], a, b[2], b[3]);
        }
      }
      if (!raw) {
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) z[n][j] *= scale;
      }
      if (edge) {
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!good || first + 8 * n + 2 * quad + (j & 1) >= vis[j >> 1]) z[n][j] = -INFINITY;
      }
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        top[0] = fmaxf(top[0], fmaxf(z[n][0], z[n][1]));
        top[1] = fmaxf(top[1], fmaxf(z[n][2], z[n][3]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2)) * mul;
      }
      // the maximum moves only when a unit exceeds it by more than 2^8: weights stay below 2^8
      const bool grow0 = top[0] > m[0] + 8.f, grow1 = top[1] > m[1] + 8.f;
      if (__any_sync(0xffffffffu, grow0 || grow1)) {
        const float f0 = grow0 ? fast_exp2(m[0] - top[0]) : 1.f, f1 = grow1 ? fast_exp2(m[1] - top[1]) : 1.f;
        if (grow0) m[0] = top[0];
        if (grow1) m[1] = top[1];
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
      }
      const float mm[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
      uint32_t w[kN][2];
#pragma unroll
      for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[n][j] = fast_exp2(fmaf(z[n][j], mul, -mm[j >> 1]));
        l[0] += z[n][0] + z[n][1];
        l[1] += z[n][2] + z[n][3];
        w[n][0] = pack16<E>(z[n][0], z[n][1]);
        w[n][1] = pack16<E>(z[n][2], z[n][3]);
      }
      // the weighted sum of rows of V, 16 keys at a time
      const int v_row = key0 + (lane & 15), v_half = lane >> 4;
#pragma unroll
      for (int g = 0; g < kN / 2; ++g) {
        const uint32_t a[4] = {w[2 * g][0], w[2 * g][1], w[2 * g + 1][0], w[2 * g + 1][1]};
        const int r = v_row + 16 * g;
        const uint32_t row_at = vs + r * 128;
        const int key = first + 16 * g + 2 * quad;  // the keys of a register: key and key + 1, 8 further on
        const bool mend = edge && first + 16 * g + 16 > lo;
#pragma unroll
        for (int j = 0; j < kV; j += 2) {
          uint32_t b[4];
          ldsm_t(b, row_at + (j >> 3) * kChunk + ((((j & 7) + v_half) ^ (r & 7)) << 4));
          if (mend) {  // a weight of 0 would carry NaN and infinities into the product
            bool found = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kk = key + 8 * (i & 1);
              uint32_t x = b[i];
              if (kk >= s.len) x &= 0xFFFF0000u;
              if (kk + 1 >= s.len) x &= 0x0000FFFFu;
              const uint32_t y = finite2<E>(x);
              found = found || (y != x && good);
              if (kk >= lo) x = (x & 0xFFFF0000u) | (y & 0x0000FFFFu);
              if (kk + 1 >= lo) x = (x & 0x0000FFFFu) | (y & 0xFFFF0000u);
              b[i] = x;
            }
            if (found) *c.mended() = 1u;
          }
          mma<E>(o[j], a, b[0], b[1]);
          mma<E>(o[j + 1], a, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar(kEmpty + at_stage));
    }
    // ---- the warps' states meet
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (quad == 0) ml[warp * 16 + row0 + 8 * i] = make_float2(m[i], l[i]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(kSegEmpty + k2));  // Q and the description have been read
    if (!meet()) return;
    // state k of row tile t: group k / kSplits, split k % kSplits
    auto state_warp = [&](int t, int k) { return (k / kSplits) * 4 + (k % kSplits) * kTiles + t; };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float most = -INFINITY;
#pragma unroll
      for (int k = 0; k < kStates; ++k) most = fmaxf(most, ml[state_warp(tile, k) * 16 + row0 + 8 * i].x);
      const float f = m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - most);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        o[j][2 * i] *= f;
        o[j][2 * i + 1] *= f;
      }
    }
    const bool whole = s.u0 == 0 && s.u1 == s.units;
    const int slot = s.u0 > 0 ? 0 : 1;
    float* part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * p.part_floats;
    const bool mended = *c.mended() != 0;
#pragma unroll
    for (int ch = 0; ch < kV / 4; ++ch) {
      if (ch * kCols >= p.x.d_v) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = 8 * j + 2 * quad;
        float* dst = join + (warp * 16 + row0) * kPitch + col;
        *reinterpret_cast<float2*>(dst) = make_float2(o[4 * ch + j][0], o[4 * ch + j][1]);
        *reinterpret_cast<float2*>(dst + 8 * kPitch) = make_float2(o[4 * ch + j][2], o[4 * ch + j][3]);
      }
      if (!meet()) return;
      const int tid = warp * 32 + lane, col = (tid & 7) * 4, d = ch * kCols + col;
      for (int r = tid >> 3; r < p.rows; r += 32) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float most = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kStates; ++k) most = fmaxf(most, ml[state_warp(r >> 4, k) * 16 + (r & 15)].x);
#pragma unroll
        for (int k = 0; k < kStates; ++k) {
          const int w = state_warp(r >> 4, k);
          const float4 x = *reinterpret_cast<const float4*>(join + (w * 16 + (r & 15)) * kPitch + col);
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
          const float2 t = ml[w * 16 + (r & 15)];
          if (t.x != -INFINITY) sum += t.y * fast_exp2(t.x - most);
          else sum += t.y;  // 0, or the NaN of a score
        }
        if (d >= p.x.d_v) continue;
        const int tok = r / p.G, head = s.hk * p.G + (r - tok * p.G);
        const int seen = tok < s.n ? min(s.len, max(0, s.pos + tok + 1)) : 0;
        if (tok >= s.n) {  // padding: its scores were made, and are dropped here
          sum = 0.f;
          most = -INFINITY;
        }
        if (mended && lo < seen) {
          const int a = max(lo, s.u0 * kUnit), e = min(seen, s.u1 * kUnit);
          float* y = &v.x;
          for (int i = 0; i < 4; ++i)
            if (infinite_column<E>(p, s, a, e, d + i)) y[i] = __uint_as_float(0x7FC00000u);
        }
        if (whole) {
          const int64_t at = (static_cast<int64_t>(s.b) * p.x.S1 + tok) * p.x.n_q + head;
          const bool nothing = sum == 0.f;
          const float inv = nothing ? 0.f : 1.f / sum;
          uint2 y = make_uint2(pack16<E>(v.x * inv, v.y * inv), pack16<E>(v.z * inv, v.w * inv));
          if (nothing) y = make_uint2(0u, 0u);
          *reinterpret_cast<uint2*>(static_cast<E*>(p.x.out) + at * p.x.d_v + d) = y;
          if (d == 0 && p.x.lse != nullptr) p.x.lse[at] = nothing ? -INFINITY : (most + log2f(sum)) * 0.69314718055994530942f;
        } else {
          *reinterpret_cast<float4*>(part + r * p.x.d_v + d) = v;
          // the lowest maximum joins with weight 0 and brings along the NaN of infinite values whose scores are all -inf
          if (d == 0) *reinterpret_cast<float2*>(part + p.rows * p.x.d_v + 2 * r) = make_float2(seen > 0 ? fmaxf(most, -3.402823466e38f) : most, sum);
        }
      }
      if (!meet()) return;
    }
    if (!whole && slot == 1 && warp == 0 && lane == 0) {
      // the CTAs that hold the rest: up to the one whose share has the head's last unit
      const int64_t end = static_cast<int64_t>(blockIdx.x + 1) * total / ctas + (s.units - s.u1);  // one behind it
      int last = static_cast<int>((end * ctas + total - 1) / total) - 1;
      p.records[blockIdx.x] = make_int4(s.b, s.hk, last - static_cast<int>(blockIdx.x), 1);
    }
  }
}

template <typename E, int kTiles, int kV>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ uint8_t raw[];
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  Ctx c;
  c.sb = (smem_u32(raw) + 1023u) & ~1023u;  // swizzled tiles
  c.smem = raw + (c.sb - smem_u32(raw));
  c.wait_ns = p.wait_ns;
  c.abort = reinterpret_cast<volatile uint32_t*>(c.smem + kOffAbort);
  if (tid == 0) {
    *c.abort = 0u;
    *c.mended() = 0u;
    p.records[blockIdx.x] = make_int4(0, 0, 0, 0);  // nothing to join, until this CTA finds a cut
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(c.bar(kFull + i), 1);
      mbar_init(c.bar(kEmpty + i), kConsumers / kGroups);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(c.bar(kSegFull + i), 1);
      mbar_init(c.bar(kSegEmpty + i), kConsumers);
    }
    mbar_init(c.bar(kJoin), kConsumers);
    fence_mbarrier_init_cluster();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int b = 0, ctas = 1;
  int64_t base = 0, from = 0, to = 0, total = 0;
  __syncthreads();
  const bool busy = start(p, c, b, base, from, to, total, ctas);
  __syncthreads();
  if (busy) {
    if (warp == kLoadWarp) load_role(p, c, maps, b, base, from, to);
    else consume_role<E, kTiles, kV>(p, c, warp, lane, ctas, total);
  }
  if (*c.abort) {
    if (lane == 0) atomicOr(&g_paged_status, MLA_DEVICE_TIMEOUT);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000) {  // loads in flight to shared memory take microseconds
    }
  }
}

// ------------------------------------------------------------------ merge
// Joins the parts of a head that was cut: block i those of the head whose first part is CTA i's last.
constexpr int kMergeThreads = 256;
constexpr int kAhead = 4;  // parts in flight
template <typename E>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 rec = __ldcg(p.records + blockIdx.x);
  if (rec.w == 0) return;
  const int quads = p.x.d_v / 4;
  for (int i = threadIdx.x; i < p.rows * quads; i += kMergeThreads) {
    const int r = i / quads, d = (i - r * quads) * 4;
    float top = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 <= rec.z; k0 += kAhead) {
      float2 ml[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = min(k0 + u, rec.z);
        const float* src = p.parts + ((static_cast<int64_t>(blockIdx.x) + k) * 2 + (k > 0 ? 0 : 1)) * p.part_floats;
        ml[u] = __ldcg(reinterpret_cast<const float2*>(src + p.rows * p.x.d_v + 2 * r));
        v[u] = __ldcg(reinterpret_cast<const float4*>(src + r * p.x.d_v + d));
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (k0 + u > rec.z || (ml[u].x == -INFINITY && ml[u].y == 0.f)) continue;  // a part in which the row sees nothing
        const float next = fmaxf(top, ml[u].x), f = top == -INFINITY ? 0.f : exp2f(top - next), w = exp2f(ml[u].x - next);
        top = next;
        l = l * f + ml[u].y * w;
        o[0] = o[0] * f + v[u].x * w;
        o[1] = o[1] * f + v[u].y * w;
        o[2] = o[2] * f + v[u].z * w;
        o[3] = o[3] * f + v[u].w * w;
      }
    }
    const bool nothing = l == 0.f;
    const float inv = nothing ? 0.f : 1.f / l;
    const int tok = r / p.G;
    const int64_t at = (static_cast<int64_t>(rec.x) * p.x.S1 + tok) * p.x.n_q + rec.y * p.G + (r - tok * p.G);
    uint2 y = make_uint2(pack16<E>(o[0] * inv, o[1] * inv), pack16<E>(o[2] * inv, o[3] * inv));
    if (nothing) y = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(static_cast<E*>(p.x.out) + at * p.x.d_v + d) = y;
    if (d == 0 && p.x.lse != nullptr) p.x.lse[at] = nothing ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
  }
}

// ------------------------------------------------------------------ host side
constexpr int kMaxDevices = 64, kMaxCtas = 160;
struct Device {
  bool ready = false;
  int sms = 0;
};
Device g_dev[kMaxDevices];
std::mutex g_lock;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

typedef void (*Kernel)(const Maps, const Params);
template <typename E>
Kernel kernel_of(int tiles, bool wide) {
  static const Kernel all[3][2] = {{paged_attn_kernel<E, 1, 8>, paged_attn_kernel<E, 1, 16>},
                                   {paged_attn_kernel<E, 2, 8>, paged_attn_kernel<E, 2, 16>},
                                   {paged_attn_kernel<E, 4, 8>, paged_attn_kernel<E, 4, 16>}};
  return all[tiles / 2][wide ? 1 : 0];
}

// Kernel attributes and the tensor-map encoder; the first call on a device.
mla_status init_device(int* sms) {
  int dev = 0;
  HEADS_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(MLA_ERR_UNSUPPORTED, "device ordinal %d too large", dev);
  std::lock_guard<std::mutex> guard(g_lock);
  Device& d = g_dev[dev];
  if (!d.ready) {
    const mla_status st = tensor_map_encoder(&g_encode);
    if (st != MLA_OK) return st;
    HEADS_CUDA(cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev), "device attributes");
    for (int tiles : {1, 2, 4})
      for (bool wide : {false, true})
        for (Kernel k : {kernel_of<__nv_bfloat16>(tiles, wide), kernel_of<__half>(tiles, wide)})
          HEADS_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost), "kernel set-up");
    d.ready = true;
  }
  *sms = d.sms;
  return MLA_OK;
}

// Rows of a key head; up to kMaxRows of them go through the kernel above.
int rows_of(const Problem& p) { return static_cast<int>(std::min<int64_t>(1 << 30, static_cast<int64_t>(p.S1) * (p.n_q / p.n_kv))); }
int part_floats(const Problem& p) { return (rows_of(p) * (p.d_v + 2) + 3) & ~3; }
// CTAs that the longest stream of these dims feeds.
int64_t most_ctas(const Problem& p) {
  const int64_t heads = std::min<int64_t>(int64_t(1) << 20, static_cast<int64_t>(p.B) * p.n_kv);
  return std::max<int64_t>(1, std::min<int64_t>(kMaxCtas, heads * 2 * p.W / kMinUnits));
}
size_t records_bytes(const Problem& p) { return (most_ctas(p) * sizeof(int4) + 255) & ~size_t(255); }
size_t workspace_of(const Problem& p) { return records_bytes(p) + static_cast<size_t>(most_ctas(p)) * 2 * part_floats(p) * sizeof(float); }

mla_status launch(const Problem& x, cudaStream_t s) {
  int sms = 0;
  const mla_status st = init_device(&sms);
  if (st != MLA_OK) return st;
  Params p;
  p.x = x;
  p.records = static_cast<int4*>(x.workspace);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(x.workspace) + records_bytes(x));
  p.part_floats = part_floats(x);
  p.G = x.n_q / x.n_kv;
  p.rows = rows_of(x);
  const int tiles = p.rows <= 16 ? 1 : p.rows <= 32 ? 2 : 4;
  p.kc = (x.d_qk + 63) / 64;
  p.vc = (x.d_v + 63) / 64;
  p.ks = (x.d_qk + 15) / 16;
  p.q_bytes = p.kc * tiles * 16 * 128;
  p.stage_bytes = (p.kc + p.vc) * kChunk;
  p.stages = std::min(kMaxStages, (kSmemMost - 1024 - kOffTiles - 2 * p.q_bytes) / p.stage_bytes);
  p.ctas = static_cast<int>(std::min<int64_t>(std::min(sms, kMaxCtas), most_ctas(x)));
  p.wait_ns = host_wait_limit_ns();
  Maps maps;
  {
    const int64_t size[3] = {x.d_qk, x.n_q, x.T}, stride[2] = {x.q.head_stride, x.q.token_stride};
    const int box[3] = {64, p.G, x.S1};
    const mla_status ms = tmap(g_encode, &maps.q, x.dtype, x.q.data, 3, size, stride, box, "q");
    if (ms != MLA_OK) return ms;
  }
  for (int i = 0; i < 2; ++i) {
    const mla_kv_cache& c = i == 0 ? x.k : x.v;
    const int64_t size[4] = {i == 0 ? x.d_qk : x.d_v, kPage, x.n_kv, x.num_blocks};
    const int64_t stride[3] = {c.row_stride, c.head_stride, c.block_stride};
    const int box[4] = {64, kUnit, 1, 1};
    const mla_status ms = tmap(g_encode, i == 0 ? &maps.k : &maps.v, x.dtype, c.data, 4, size, stride, box, i == 0 ? "k" : "v");
    if (ms != MLA_OK) return ms;
  }
  const bool bf = x.dtype == MLA_ROPE_BF16;
  const Kernel kernel = bf ? kernel_of<__nv_bfloat16>(tiles, p.vc == 2) : kernel_of<__half>(tiles, p.vc == 2);
  const size_t smem = 1024 + kOffTiles + 2 * p.q_bytes + static_cast<size_t>(p.stages) * p.stage_bytes;
  kernel<<<static_cast<unsigned>(p.ctas), kThreads, smem, s>>>(maps, p);
  HEADS_CUDA(cudaGetLastError(), "kernel launch");
  if (p.ctas > 1)
    HEADS_CUDA(bf ? launch_after(paged_merge_kernel<__nv_bfloat16>, dim3(static_cast<unsigned>(p.ctas)), kMergeThreads, 0, s, p)
                  : launch_after(paged_merge_kernel<__half>, dim3(static_cast<unsigned>(p.ctas)), kMergeThreads, 0, s, p),
               "merge launch");
  return MLA_OK;
}

}  // namespace paged

cudaError_t paged_status(unsigned int* v, bool clear) { return read_status(paged::g_paged_status, v, clear); }

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

// Which kernel: memory binds the one above for as long as its products keep up.
bool few_rows(const Problem& p) { return paged::rows_of(p) <= paged::kMaxRows; }
size_t workspace_of(const Problem& p) { return few_rows(p) ? paged::workspace_of(p) : tiles_workspace(p); }

}  // namespace
}  // namespace mlaheads

extern "C" {

size_t mla_paged_workspace_bytes(const mla_paged_dims* dims) {
  using namespace mlaheads;
  no_error();
  if (dims == nullptr || check_dims(*dims) != MLA_OK) return 0;
  return workspace_of(problem_of(*dims));
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
  const mla_status cst = check_problem(p, workspace_bytes, workspace_of(p));
  if (cst != MLA_OK) return cst;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return few_rows(p) ? paged::launch(p, s) : launch_tiles(p, s);
}

}  // extern "C"
