// Attention of new tokens over a paged cache of keys and values for GB300
// (sm_103a); formulas in mla_heads.h.
//
// The keys and values of a sequence are read once and meet few rows (the S1 new
// tokens of the G heads that share them), so memory binds.  A CTA holds up to eight
// pipelines of two warps (as many as get two slots each: eight where keys and values
// have at most three 64-column chunks together, seven at 128 and 128, five at 192 and
// 128; the warps left over idle): one streams units of 32 keys, keys and values together,
// by TMA into slots of shared memory that no other pipeline touches, the other
// takes 16 rows through them with the running maximum, sum and output in
// registers, as accumulators of mma.sync (m16n8k16: the 128-row tiles of tcgen05
// would be an eighth full, and the products of a unit take less time than its
// bytes take to arrive).  No pipeline waits for another, and a head that one has
// through goes from its registers to memory.  More than 16 rows go to two or four
// pipelines side by side, which read the same units, from L2 but for the first.
//
// The units of all sequences and heads, and what a head costs beside them, are one
// stream of which every pipeline (or group of them side by side) takes an equal
// share.  A head cut between them leaves partial states in the workspace, and a
// second launch joins them.  Who takes what follows from the lengths alone, so
// results do not depend on timing.
// Calls of more than 64 rows to a key head go through the 128-row tiles of prompts.
//
// Measured (graph replay): 64 sequences of 8192, 32 heads on 8 key heads of 128, 317 to 325 us
// (6.6 to 6.8 TB/s, the copy rate); of 100 to 8192 87 us (5.6 TB/s); chains of up to five
// tokens, 24 sequences of 500 to 20000, heads of 96, 61 us (4.8 TB/s); one token of one
// sequence of 1000 9.5 to 10.9 us, of 100000 76.  Some 12 us of a call are launches, first loads
// and the join.
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

constexpr int kUnit = 32;        // keys
constexpr int kWarps = 8;        // that compute, and as many that load
constexpr int kThreads = 2 * 32 * kWarps;
constexpr int kRegs = 128, kConsumerRegs = 192, kLoadRegs = 64;
static_assert(32 * kWarps * (kConsumerRegs + kLoadRegs) <= kThreads * kRegs, "register budget");
constexpr int kChunk = kUnit * 128;  // a unit's rows of 128 bytes
constexpr int kMaxSlots = 48;    // of a CTA
constexpr int kMaxRows = 64;
constexpr int kLeastSlots = 2;   // of a pipeline

constexpr int kBars = kMaxSlots;
constexpr int kOffScan = 0;                          // int64 [kThreads / 32]
constexpr int kOffWalk = kOffScan + kThreads / 32 * 8;  // int64 [kWarps][2]: a share's first sequence and its stream position
constexpr int kOffBars = kOffWalk + kWarps * 16;     // [kBars] the slot's bytes have landed, [kBars] they have been read
constexpr int kOffGood = kOffBars + 2 * 8 * kBars;   // int [kBars] the slot's page exists
constexpr int kOffAbort = kOffGood + 4 * kBars;
constexpr int kOffMended = kOffAbort + 4;            // a value that not every token sees was NaN or infinite
constexpr int kOffSlots = 2048;
static_assert(kOffMended + 4 <= kOffSlots, "shared memory");
constexpr int kSmemMost = 232448;

struct Params {
  Problem x;
  float* parts;    // [groups][tiles][2][part_floats]
  // [groups] the cut head that a group begins, or holds a middle part of: sequence, key head,
  // parts behind the first, 1 + the part that the group has of it (0: there is none)
  int4* records;
  int part_floats;
  int G, rows;     // heads to a key head, rows of a key head
  int tiles;       // 16-row tiles of them
  int kc, vc;      // 64-column chunks of keys and values
  int slots, unit_bytes;  // of a pipeline
  int pipes;       // pipelines of a CTA, each of a load warp and `tiles` others
  int groups;      // pipelines of the GPU that take part
  unsigned long long wait_ns;
};
struct Maps {
  CUtensorMap k, v;
};

// What a head costs beside its units, in units: queries on their way in, rows on their way out.
// Shares are equal in both: 24 sequences of 500 to 20000 keys, some without new tokens, 71 us
// -> 61 (0 / 1 / 2 / 3 / 4: 71 / 67 / 62 / 61 / 61), 64 of 100 to 8192 90 -> 87.
constexpr int kHeadCost = 3;

struct Seq {
  int n, len, pos, units;  // query tokens, keys within the table, position of token 0, units of a head
  bool cut_table;
  __device__ __forceinline__ int steps() const { return units + kHeadCost; }  // of the stream, of a head
};
__device__ __forceinline__ Seq make_seq(const Params& p, int act, int q_len) {
  Seq s;
  act = max(0, act);
  s.n = min(p.x.S1, max(0, q_len));
  s.len = min(act, p.x.W * kPage);
  s.cut_table = s.len < act && s.n > 0;
  s.pos = act - s.n;
  s.units = s.n > 0 ? max(1, (s.len + kUnit - 1) / kUnit) : 1;  // rows that see nothing are written too
  return s;
}
__device__ __forceinline__ Seq load_seq(const Params& p, int b) {
  return make_seq(p, __ldg(p.x.act_seqs + b), p.x.q_lens != nullptr ? __ldg(p.x.q_lens + b) : p.x.S1);
}

struct Ctx {
  uint32_t sb;
  uint8_t* smem;
  uint64_t wait_ns;
  volatile uint32_t* abort;
  __device__ uint32_t bar(int i) const { return sb + kOffBars + 8 * i; }
  __device__ volatile uint32_t* mended() const { return reinterpret_cast<volatile uint32_t*>(smem + kOffMended); }
};

// The stream in equal shares: the first `more` of them have `each` + 1 steps, the others `each`.
struct Split {
  int64_t each, more;
  int groups;
  __device__ __forceinline__ int64_t begin(int g) const { return g * each + min(static_cast<int64_t>(g), more); }
  __device__ __forceinline__ int group_of(int64_t step) const {
    int64_t rest;
    const int64_t wide = more * (each + 1);
    return static_cast<int>(step < wide ? divide(step, each + 1, rest) : more + divide(step - wide, each, rest));
  }
};

// Steps of a share at least: fewer parts to join where there is little to read.  4 / 5 / 6 / 8:
// one token over 1000 keys 9.4 / 10.4 / 10.8 / 10.7 us, 16 sequences of 100 9.7 / 14.5 / 15.9 / 15.
constexpr int kMinSteps = 4;
static_assert(kMinSteps > kHeadCost, "a share has a unit");

__device__ __forceinline__ Split split_of(const Params& p, int64_t total) {
  Split s;
  s.groups = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(p.groups), total / kMinSteps)));
  s.each = divide(total, s.groups, s.more);
  return s;
}
// A pipeline's number: neighbours in the stream lie in different CTAs, so that few of them use many SMs.
__device__ __forceinline__ int group_id(int pipe) { return pipe * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x); }

// Finds where the shares of the CTA's pipelines begin, and how the stream is split.
__device__ Split find_shares(const Params& p, const Ctx& c) {
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
  int64_t mine = 0, len = 0, total;
  bool cut = false;
  for (int k = 0; k < chunks; ++k) {
    const int b = k * kThreads + tid;
    len = 0;
    if (b < B) {
      const Seq s = load_seq(p, b);
      len = static_cast<int64_t>(s.steps()) * p.x.n_kv;
      cut = cut || s.cut_table;
    }
    mine += len;
  }
  if (cut) atomicOr(&g_paged_status, MLA_DEVICE_BAD_BLOCK);
  int64_t pre = scan(mine, total);
  const Split split = split_of(p, total);
  int64_t carry = 0;
  for (int k = 0; k < chunks; ++k) {
    const int b = k * kThreads + tid;
    int64_t sum = total;
    if (chunks > 1) {
      len = b < B ? static_cast<int64_t>(load_seq(p, b).steps()) * p.x.n_kv : 0;
      pre = carry + scan(len, sum);
    }
    if (b < B) {
      for (int w = 0; w < p.pipes; ++w) {
        const int g = group_id(w);
        const int64_t from = g < split.groups ? split.begin(g) : -1;
        if (from >= pre && from < pre + len) {
          at[2 * w] = b;
          at[2 * w + 1] = pre;
        }
      }
    }
    carry += sum;
  }
  __syncthreads();
  return split;
}

// A share of the stream, head by head.  Lane i keeps the lengths of sequence b0 + i.
struct Walk {
  int b, b0, act, q_len;
  int hk, at;      // the share goes on at this step of sequence b's key head hk
  int64_t left;    // steps that follow, this one among them
  Seq s;
  __device__ __forceinline__ void load_lengths(const Params& p, int lane) {
    const int i = min(b0 + lane, p.x.B - 1);
    act = __ldg(p.x.act_seqs + i);
    q_len = p.x.q_lens != nullptr ? __ldg(p.x.q_lens + i) : p.x.S1;
  }
  __device__ __forceinline__ void begin(const Params& p, int lane, int b_, int64_t off, int64_t count) {
    b = b0 = b_;
    left = count;
    load_lengths(p, lane);
    s = make_seq(p, uniform(act), uniform(q_len));
    int64_t rest;
    hk = static_cast<int>(divide(off, s.steps(), rest));
    at = static_cast<int>(rest);
  }
  // The share's units [u0, u1) of the head; none where it ends before the first.
  __device__ __forceinline__ void take(int& u0, int& u1) {
    const int end = static_cast<int>(min(static_cast<int64_t>(s.steps()), at + left));
    left -= end - at;
    u0 = max(0, at - kHeadCost);
    u1 = max(0, end - kHeadCost);
  }
  // the head behind the current one
  __device__ __forceinline__ void next_head(const Params& p, int lane) {
    at = 0;
    if (++hk < p.x.n_kv) return;
    hk = 0;
    if (++b >= p.x.B) return;  // the end of the stream
    if (b - b0 == 32) {
      b0 = b;
      load_lengths(p, lane);
    }
    s = make_seq(p, __shfl_sync(0xffffffffu, act, b - b0), __shfl_sync(0xffffffffu, q_len, b - b0));
  }
};

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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether column `col` of a value, key by key in [lo, hi), is not finite.
template <typename E>
__device__ __noinline__ bool infinite_column(const Params& p, int b, int hk, int lo, int hi, int col) {
  constexpr uint32_t kExp = __is_same(E, __half) ? 0x7C00u : 0x7F80u;
  for (int key = lo; key < hi; ++key) {
    const int id = __ldg(p.x.block_table + static_cast<int64_t>(b) * p.x.W + key / kPage);
    if (id < 0 || id >= p.x.num_blocks) continue;
    const uint16_t v = __ldg(static_cast<const uint16_t*>(p.x.v.data) + id * p.x.v.block_stride + (key % kPage) * p.x.v.row_stride +
                             hk * p.x.v.head_stride + col);
    if ((v & kExp) == kExp) return true;
  }
  return false;
}

// Rows of a unit's values that not every token sees, from row `first` on (which may
// lie far behind the unit: a page that does not exist): those
// behind the sequence (from row `live` on) become zero, the others lose their NaN
// and infinities, which a weight of 0 would carry into the product.  Warps that
// share a unit write the same; the flag is up before a value is gone.
template <typename E>
__device__ __noinline__ void mend_values(const Ctx& c, uint32_t vs, int chunks, int first, int live, int lane) {
  const int units = 8 * chunks;
  first = max(0, min(first, kUnit));  // before it is multiplied: a sequence may have 2^30 keys
  live = max(first, min(live, kUnit));
  auto at = [&](int i) {
    const int r = i / units, col = i - r * units;
    return vs + (col >> 3) * kChunk + r * 128 + (((col & 7) ^ (r & 7)) << 4);
  };
  auto load = [&](int i) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at(i)));
    return v;
  };
  auto store = [&](int i, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at(i)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
  };
  const int begin = first * units, middle = live * units;
  bool good = true;
  for (int i = begin + lane; i < middle; i += 32) good = good && finite4<E>(load(i));
  if (__any_sync(0xffffffffu, !good)) {
    *c.mended() = 1u;
    __threadfence_block();
    for (int i = begin + lane; i < middle; i += 32) {
      const uint4 v = load(i);
      store(i, make_uint4(finite2<E>(v.x), finite2<E>(v.y), finite2<E>(v.z), finite2<E>(v.w)));
    }
  }
  for (int i = middle + lane; i < kUnit * units; i += 32) store(i, make_uint4(0, 0, 0, 0));
  fence_proxy_async_smem();  // before the slot's next load
  __syncwarp();
}

// The share of a pipeline.
struct Share {
  int g, b;                  // b < 0: there is none
  int64_t from, count, off;  // in steps, of the stream, of sequence b
};
// `b` and `at`: the sequence in which the share begins, and where that sequence does.
__device__ __forceinline__ Share share_of(const Params& p, int pipe, const Split& split, int b, int64_t at) {
  Share s;
  s.g = group_id(pipe);
  s.b = pipe < p.pipes && s.g < split.groups ? b : -1;
  if (s.b < 0) return s;
  s.from = split.begin(s.g);
  s.count = split.begin(s.g + 1) - s.from;
  s.off = s.from - at;
  return s;
}
__device__ __forceinline__ Share share_of(const Params& p, const Ctx& c, int pipe, const Split& split) {
  const int64_t* at = reinterpret_cast<const int64_t*>(c.smem + kOffWalk) + 2 * min(pipe, kWarps - 1);
  return share_of(p, pipe, split, static_cast<int>(at[0]), at[1]);
}
// Of up to 32 sequences, one to a lane: every warp finds its pipeline's share, without the block.
__device__ __forceinline__ Share find_share(const Params& p, int pipe, int lane, Split& split) {
  int64_t len = 0;
  if (lane < p.x.B) {
    const Seq s = load_seq(p, lane);
    len = static_cast<int64_t>(s.steps()) * p.x.n_kv;
    if (s.cut_table && blockIdx.x == 0 && threadIdx.x < 32) atomicOr(&g_paged_status, MLA_DEVICE_BAD_BLOCK);
  }
  int64_t upto = len;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  split = split_of(p, __shfl_sync(0xffffffffu, upto, 31));
  const int64_t from = split.begin(group_id(pipe));
  const int b = max(0, __ffs(__ballot_sync(0xffffffffu, from >= upto - len && from < upto)) - 1);
  return share_of(p, pipe, split, b, __shfl_sync(0xffffffffu, upto - len, b));
}

__device__ void load_role(const Params& p, const Ctx& c, const Maps& maps, int pipe, int lane, const Share& sh) {
  const int slot0 = pipe * p.slots;
  const uint32_t slots = c.sb + kOffSlots + slot0 * p.unit_bytes;
  volatile int* good_of = reinterpret_cast<volatile int*>(c.smem + kOffGood) + slot0;
  Walk w;
  w.begin(p, lane, sh.b, sh.off, sh.count);
  int ids = -1, slot = 0;
  uint32_t phase = 1;
  bool bad = false;
  while (w.left > 0) {
    int u0, end;
    w.take(u0, end);
    const int page0 = u0 / (kPage / kUnit);
    for (int u = u0; u < end; ++u) {
      const int page = u / (kPage / kUnit) - page0;
      if (u == u0 || (page % 32 == 0 && u % (kPage / kUnit) == 0)) {  // the next 32 pages, one to a lane
        const int i = page0 + page + lane;
        ids = i < p.x.W && i * kPage < w.s.len ? __ldg(p.x.block_table + static_cast<int64_t>(w.b) * p.x.W + i) : -1;
      }
      const int id = __shfl_sync(0xffffffffu, ids, page % 32);
      const bool good = id >= 0 && id < p.x.num_blocks;
      bad = bad || (!good && u * kUnit < w.s.len && w.s.n > 0);
      const int bar = slot0 + slot;
      if (!warp_wait(c, kBars + bar, phase)) return;
      if (elect_one()) {
        const uint32_t full = c.bar(bar), dst = slots + slot * p.unit_bytes;
        const int row = u * kUnit % kPage, block = good ? id : p.x.num_blocks;  // beyond the pool: zeros
        good_of[slot] = good ? 1 : 0;
        mbar_arrive_expect_tx(full, p.unit_bytes);
        for (int i = 0; i < p.kc; ++i) tma_4d(dst + i * kChunk, &maps.k, 64 * i, row, w.hk, block, full);
        for (int i = 0; i < p.vc; ++i) tma_4d(dst + (p.kc + i) * kChunk, &maps.v, 64 * i, row, w.hk, block, full);
      }
      __syncwarp();
      if (++slot == p.slots) {
        slot = 0;
        phase ^= 1;
      }
    }
    w.next_head(p, lane);
  }
  if (bad && lane == 0) atomicOr(&g_paged_status, MLA_DEVICE_BAD_BLOCK);
}

// kS: 16-column steps of keys, kV: 8-column tiles of values.
template <typename E, int kS, int kV>
__device__ void consume_role(const Params& p, const Ctx& c, int warp, int lane, const Split& split, const Share& sh) {
  const int pipe = warp / p.tiles, tile = warp % p.tiles;
  const int quad = lane & 3, row0 = lane >> 2;  // the thread's rows: row0 and row0 + 8 of the tile
  const int rows = min(16, p.rows - tile * 16);
  const float scale = p.x.scale_log2;
  const bool raw = scale > 0.f;
  const float mul = raw ? scale : 1.f;
  const int slot0 = pipe * p.slots;
  const uint32_t slots = c.sb + kOffSlots + slot0 * p.unit_bytes;
  const volatile int* good_of = reinterpret_cast<const volatile int*>(c.smem + kOffGood) + slot0;

  // ---- heads of the share
  Walk w;
  w.begin(p, lane, sh.b, sh.off, sh.count);
  int slot = 0;
  uint32_t phase = 0;
  while (w.left > 0) {
    const Seq s = w.s;
    const int b = w.b, hk = w.hk;
    const int64_t begin = sh.from + (sh.count - w.left) - w.at;  // of the head in the stream
    int u0, u1;
    w.take(u0, u1);
    if (u0 == u1) break;  // the share ends before the head's first unit
    int vis[2], tok[2];
    uint32_t q[kS][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = tile * 16 + row0 + 8 * i;
      tok[i] = r / p.G;
      const bool live = r < p.rows && tok[i] < s.n;
      vis[i] = live ? min(s.len, max(0, s.pos + tok[i] + 1)) : 0;
      const uint16_t* src = static_cast<const uint16_t*>(p.x.q.data) + (static_cast<int64_t>(b) * p.x.S1 + tok[i]) * p.x.q.token_stride +
                            (hk * p.G + r - tok[i] * p.G) * p.x.q.head_stride + 2 * quad;
#pragma unroll
      for (int k = 0; k < kS; ++k) {
        q[k][i] = live && 16 * k < p.x.d_qk ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k)) : 0u;
        q[k][i + 2] = live && 16 * k + 8 < p.x.d_qk ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8)) : 0u;
      }
    }
    const int lo = min(s.len, max(0, s.pos + 1));  // keys that every token sees
    float o[kV][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kV; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    for (int u = u0; u < u1; ++u) {
      if (!warp_wait(c, slot0 + slot, phase)) return;
      const uint32_t ks = slots + slot * p.unit_bytes, vs = ks + p.kc * kChunk;
      const bool good = good_of[slot] != 0;
      const int first = u * kUnit;  // key of column 0
      constexpr int kN = kUnit / 8;
      float z[kN][4];
#pragma unroll
      for (int n = 0; n < kN; ++n) z[n][0] = z[n][1] = z[n][2] = z[n][3] = 0.f;
      const int k_row = (lane & 7) + ((lane >> 4) << 3), k_half = (lane >> 3) & 1;
      // fragments are loaded a step ahead of the products that take them
      uint32_t t[2][kN / 2][4];
      auto load_keys = [&](int k) {
#pragma unroll
        for (int n = 0; n < kN / 2; ++n)
          ldsm(t[k & 1][n], ks + (k >> 2) * kChunk + (k_row + 16 * n) * 128 + (((2 * (k & 3) + k_half) ^ (k_row & 7)) << 4));
      };
      load_keys(0);
#pragma unroll
      for (int k = 0; k < kS; ++k) {
        if (k + 1 < kS) load_keys(k + 1);
#pragma unroll
        for (int n = 0; n < kN / 2; ++n) {
          mma<E>(z[2 * n], q[k], t[k & 1][n][0], t[k & 1][n][1]);
          mma<E>(z[2 * n + 1], q[k], t[k & 1][n][2], t[k & 1][n][3]);
        }
      }
      if (!raw) {
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) z[n][j] *= scale;
      }
      if (!good || first + kUnit > lo) {
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!good || first + 8 * n + 2 * quad + (j & 1) >= vis[j >> 1]) z[n][j] = -INFINITY;
        mend_values<E>(c, vs, p.vc, lo - first, s.len - first, lane);
      }
      const int v_row = lane & 15, v_half = lane >> 4;
      auto load_values = [&](int j) {
#pragma unroll
        for (int g = 0; g < kN / 2; ++g)
          ldsm_t(t[j & 1][g], vs + (j >> 2) * kChunk + (v_row + 16 * g) * 128 + (((2 * (j & 3) + v_half) ^ (v_row & 7)) << 4));
      };
      load_values(0);
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
      // the maximum moves only when a unit exceeds it by more than 2^8: weights stay below 2^8 (lifted, 2^15)
      const bool grow0 = top[0] > m[0] + (8.f + kLift<E>), grow1 = top[1] > m[1] + (8.f + kLift<E>);
      if (__any_sync(0xffffffffu, grow0 || grow1)) {
        const float m0 = top[0] - kLift<E>, m1 = top[1] - kLift<E>;
        const float f0 = grow0 ? fast_exp2(m[0] - m0) : 1.f, f1 = grow1 ? fast_exp2(m[1] - m1) : 1.f;
        if (grow0) m[0] = m0;
        if (grow1) m[1] = m1;
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
      uint32_t a[kN / 2][4];
#pragma unroll
      for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[n][j] = fast_exp2(fmaf(z[n][j], mul, -mm[j >> 1]));
        l[0] += z[n][0] + z[n][1];
        l[1] += z[n][2] + z[n][3];
        a[n / 2][2 * (n & 1)] = pack16<E>(z[n][0], z[n][1]);
        a[n / 2][2 * (n & 1) + 1] = pack16<E>(z[n][2], z[n][3]);
      }
#pragma unroll
      for (int j = 0; j < kV / 2; ++j) {
        if (j + 1 < kV / 2) load_values(j + 1);
#pragma unroll
        for (int g = 0; g < kN / 2; ++g) {
          mma<E>(o[2 * j], a[g], t[j & 1][g][0], t[j & 1][g][1]);
          mma<E>(o[2 * j + 1], a[g], t[j & 1][g][2], t[j & 1][g][3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar(kBars + slot0 + slot));
      if (++slot == p.slots) {
        slot = 0;
        phase ^= 1;
      }
    }
    // ---- the head's rows, or this part of them, leave the registers
    const bool whole = u0 == 0 && u1 == s.units, mended = *c.mended() != 0;
    const int part = u0 > 0 ? 0 : 1;
    float* dst = p.parts + (static_cast<int64_t>(sh.g * p.tiles + tile) * 2 + part) * p.part_floats;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int r = row0 + 8 * i;
      if (r >= rows) continue;
      if (tok[i] >= s.n) {  // padding
        l[i] = 0.f;
        m[i] = -INFINITY;
      }
      const bool nothing = l[i] == 0.f;
      const float inv = nothing ? 0.f : 1.f / l[i];
      const int64_t row = (static_cast<int64_t>(b) * p.x.S1 + tok[i]) * p.x.n_q + hk * p.G + (tile * 16 + r - tok[i] * p.G);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const int d = 8 * j + 2 * quad;
        if (d >= p.x.d_v) continue;
        float x = o[j][2 * i], y = o[j][2 * i + 1];
        if (mended && !(whole && nothing)) {
          const int k0 = max(lo, u0 * kUnit), k1 = min(vis[i], u1 * kUnit);
          if (infinite_column<E>(p, b, hk, k0, k1, d)) x = __uint_as_float(0x7FC00000u);
          if (infinite_column<E>(p, b, hk, k0, k1, d + 1)) y = __uint_as_float(0x7FC00000u);
        }
        if (whole)
          *reinterpret_cast<uint32_t*>(static_cast<E*>(p.x.out) + row * p.x.d_v + d) = nothing ? 0u : pack16<E>(x * inv, y * inv);
        else
          *reinterpret_cast<float2*>(dst + r * p.x.d_v + d) = make_float2(x, y);
      }
      if (quad == 0) {
        if (whole) {
          if (p.x.lse != nullptr) p.x.lse[row] = nothing ? -INFINITY : (m[i] + log2f(l[i])) * 0.69314718055994530942f;
        } else {
          // the lowest maximum joins with weight 0 and brings along the NaN of infinite values whose scores are all -inf
          *reinterpret_cast<float2*>(dst + rows * p.x.d_v + 2 * r) = make_float2(vis[i] > 0 ? fmaxf(m[i], -3.402823466e38f) : m[i], l[i]);
        }
      }
    }
    if (u1 < s.units && tile == 0 && lane == 0) {  // the share ends inside the head
      const int first = u0 > 0 ? split.group_of(begin + kHeadCost) : sh.g;
      p.records[sh.g] = make_int4(b, hk, split.group_of(begin + s.steps() - 1) - first, 1 + sh.g - first);
    }
    w.next_head(p, lane);
  }
}

template <typename E, int kS, int kV>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ uint8_t raw[];
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  Ctx c;
  c.sb = (smem_u32(raw) + 1023u) & ~1023u;  // swizzled tiles
  c.smem = raw + (c.sb - smem_u32(raw));
  c.wait_ns = p.wait_ns;
  c.abort = reinterpret_cast<volatile uint32_t*>(c.smem + kOffAbort);
  if (tid == 0) *c.abort = *c.mended() = 0u;
  if (tid < 2 * kBars) mbar_init(c.bar(tid), tid < kBars ? 1 : p.tiles);
  if (tid < p.pipes && group_id(tid) < p.groups) p.records[group_id(tid)] = make_int4(0, 0, 0, 0);
  fence_mbarrier_init_cluster();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();
  const int pipe = warp < kWarps ? warp / p.tiles : warp - kWarps;
  Split split;
  Share sh;
  if (p.x.B <= 32) {
    sh = find_share(p, pipe, lane, split);
  } else {
    split = find_shares(p, c);
    sh = share_of(p, c, pipe, split);
  }
  if (warp < kWarps) {
    regs_increase<kConsumerRegs>();
    if (sh.b >= 0) consume_role<E, kS, kV>(p, c, warp, lane, split, sh);
  } else {
    regs_decrease<kLoadRegs>();
    if (sh.b >= 0) load_role(p, c, maps, pipe, lane, sh);
  }
  if (*c.abort) {
    if (lane == 0) atomicOr(&g_paged_status, MLA_DEVICE_TIMEOUT);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000) {  // loads in flight to shared memory take microseconds
    }
  }
}

// ------------------------------------------------------------------ merge
// Joins the parts of the heads that were cut, 32 quads of columns of a row tile at a
// time: a block to each group, whose record says what it has to do, so that nothing is
// searched for.  Few parts are a warp's work, the head's first group has it; many are
// shared out among a block's warps, and their slices among the groups that hold them.
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
constexpr int kAhead = 4;        // parts in flight
constexpr int kFewParts = 8;     // 4 / 8 / 16: 24 chains of 500 to 20000 62 / 60.5 / 63 us
constexpr int kMaxGroups = 152 * kWarps;

struct State {
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void join(float m2, float l2, const float (&v)[4]) {
    if (m2 == -INFINITY && l2 == 0.f) return;  // a part in which the row sees nothing
    const float top = fmaxf(m, m2), f = m == -INFINITY ? 0.f : exp2f(m - top), w = exp2f(m2 - top);
    m = top;
    l = l * f + l2 * w;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = o[j] * f + v[j] * w;
  }
};

template <typename E>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ Params p) {
  __shared__ float sm[kMergeWarps][6][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tile = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 rec = __ldcg(p.records + blockIdx.x);
  if (rec.w == 0) return;
  const int parts = rec.z + 1, mine = rec.w - 1, group0 = static_cast<int>(blockIdx.x) - mine;
  const bool few = parts <= kFewParts;
  if (few && mine > 0) return;
  const int rows = min(16, p.rows - tile * 16), quads = p.x.d_v / 4, slices = (rows * quads + 31) / 32;
  // parts first, first + step, ... of slice `i`
  auto gather = [&](int i, int first, int step, State& st, int& r, int& d) {
    const int quad = i * 32 + lane;
    r = quad / quads;
    d = (quad - r * quads) * 4;
    const bool in = r < rows;
    if (!in) r = 0;
    for (int k0 = first; k0 < parts; k0 += kAhead * step) {
      float2 ml[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * step < parts ? k0 + u * step : first;
        const float* src = p.parts + ((static_cast<int64_t>(group0 + k) * p.tiles + tile) * 2 + (k > 0 ? 0 : 1)) * p.part_floats;
        ml[u] = __ldcg(reinterpret_cast<const float2*>(src + rows * p.x.d_v + 2 * r));
        v[u] = __ldcg(reinterpret_cast<const float4*>(src + r * p.x.d_v + d));
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (k0 + u * step < parts) st.join(ml[u].x, ml[u].y, {v[u].x, v[u].y, v[u].z, v[u].w});
    }
    r = in ? tile * 16 + r : -1;
  };
  auto put = [&](const State& st, int r, int d) {
    if (r < 0) return;
    const bool nothing = st.l == 0.f;
    const float inv = nothing ? 0.f : 1.f / st.l;
    const int tok = r / p.G;
    const int64_t at = (static_cast<int64_t>(rec.x) * p.x.S1 + tok) * p.x.n_q + rec.y * p.G + (r - tok * p.G);
    uint2 y = make_uint2(pack16<E>(st.o[0] * inv, st.o[1] * inv), pack16<E>(st.o[2] * inv, st.o[3] * inv));
    if (nothing) y = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(static_cast<E*>(p.x.out) + at * p.x.d_v + d) = y;
    if (d == 0 && p.x.lse != nullptr) p.x.lse[at] = nothing ? -INFINITY : (st.m + log2f(st.l)) * 0.69314718055994530942f;
  };
  if (few) {
    for (int i = warp; i < slices; i += kMergeWarps) {
      State st;
      int r, d;
      gather(i, 0, 1, st, r, d);
      put(st, r, d);
    }
    return;
  }
  for (int i = mine; i < slices; i += rec.z) {  // the first rec.z parts have groups with this record
    State st;
    int r, d;
    gather(i, warp, kMergeWarps, st, r, d);
    __syncthreads();  // the last slice's states have been read
    sm[warp][0][lane] = st.m;
    sm[warp][1][lane] = st.l;
#pragma unroll
    for (int j = 0; j < 4; ++j) sm[warp][2 + j][lane] = st.o[j];
    __syncthreads();
    if (warp != 0) continue;
    for (int k = 1; k < kMergeWarps; ++k)
      st.join(sm[k][0][lane], sm[k][1][lane], {sm[k][2][lane], sm[k][3][lane], sm[k][4][lane], sm[k][5][lane]});
    put(st, r, d);
  }
}

// ------------------------------------------------------------------ host side
constexpr int kMaxDevices = 64;
struct Device {
  bool ready = false;
  int sms = 0;
};
Device g_dev[kMaxDevices];
std::mutex g_lock;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

typedef void (*Kernel)(const Maps, const Params);
// The kernels, and the sizes of keys and values up to which each goes.
constexpr int kKernels = 7;
template <typename E>
Kernel kernel_of(int i) {
  static const Kernel all[kKernels] = {paged_attn_kernel<E, 4, 8>, paged_attn_kernel<E, 4, 16>,  paged_attn_kernel<E, 6, 12>, paged_attn_kernel<E, 6, 16>,
                                       paged_attn_kernel<E, 8, 8>, paged_attn_kernel<E, 8, 16>, paged_attn_kernel<E, 12, 16>};
  return all[i];
}
constexpr int kKernelSize[kKernels][2] = {{64, 64}, {64, 128}, {96, 96}, {96, 128}, {128, 64}, {128, 128}, {192, 128}};

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
    for (int i = 0; i < kKernels; ++i) {
      for (Kernel k : {kernel_of<__nv_bfloat16>(i), kernel_of<__half>(i)}) {
        HEADS_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost), "kernel set-up");
        cudaFuncAttributes fa;
        HEADS_CUDA(cudaFuncGetAttributes(&fa, k), "kernel attributes");
        if (fa.numRegs < kRegs) return fail(MLA_ERR_CUDA, "the kernel was built with %d registers", fa.numRegs);  // what the warps divide
      }
    }
    d.ready = true;
  }
  *sms = d.sms;
  return MLA_OK;
}

// Rows of a key head; up to kMaxRows of them go through the kernel above.
int rows_of(const Problem& p) { return static_cast<int>(std::min<int64_t>(1 << 30, static_cast<int64_t>(p.S1) * (p.n_q / p.n_kv))); }
int tiles_of(const Problem& p) { return rows_of(p) <= 16 ? 1 : rows_of(p) <= 32 ? 2 : 4; }
int part_floats(const Problem& p) { return (std::min(16, rows_of(p)) * (p.d_v + 2) + 3) & ~3; }
// Groups that the longest stream of these dims feeds.
int64_t most_groups(const Problem& p) {
  const int64_t heads = std::min<int64_t>(int64_t(1) << 20, static_cast<int64_t>(p.B) * p.n_kv);
  return std::max<int64_t>(1, std::min<int64_t>(kMaxGroups / tiles_of(p), heads * (kPage / kUnit) * p.W / kMinSteps));
}
size_t records_bytes(const Problem& p) { return (most_groups(p) * sizeof(int4) + 255) & ~size_t(255); }
size_t workspace_of(const Problem& p) {
  return records_bytes(p) + static_cast<size_t>(most_groups(p)) * tiles_of(p) * 2 * part_floats(p) * sizeof(float);
}

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
  p.tiles = tiles_of(x);
  int kind = 0;
  while (x.d_qk > kKernelSize[kind][0] || x.d_v > kKernelSize[kind][1]) ++kind;
  p.kc = (kKernelSize[kind][0] + 63) / 64;
  p.vc = (kKernelSize[kind][1] + 63) / 64;
  p.unit_bytes = (p.kc + p.vc) * kChunk;
  p.wait_ns = host_wait_limit_ns();
  const int fit = std::min(kMaxSlots, (kSmemMost - 1024 - kOffSlots) / p.unit_bytes);
  p.pipes = std::min(kWarps / p.tiles, std::max(1, fit / kLeastSlots));
  p.slots = fit / p.pipes;
  p.groups = static_cast<int>(std::min<int64_t>(most_groups(x), static_cast<int64_t>(sms) * p.pipes));
  const int ctas = std::min(sms, p.groups);
  Maps maps;
  for (int i = 0; i < 2; ++i) {
    const mla_kv_cache& c = i == 0 ? x.k : x.v;
    const int64_t size[4] = {i == 0 ? x.d_qk : x.d_v, kPage, x.n_kv, x.num_blocks};
    const int64_t stride[3] = {c.row_stride, c.head_stride, c.block_stride};
    const int box[4] = {64, kUnit, 1, 1};
    const mla_status ms = tmap(g_encode, i == 0 ? &maps.k : &maps.v, x.dtype, c.data, 4, size, stride, box, i == 0 ? "k" : "v");
    if (ms != MLA_OK) return ms;
  }
  const bool bf = x.dtype == MLA_ROPE_BF16;
  const Kernel kernel = bf ? kernel_of<__nv_bfloat16>(kind) : kernel_of<__half>(kind);
  const size_t smem = 1024 + kOffSlots + static_cast<size_t>(p.pipes) * p.slots * p.unit_bytes;
  kernel<<<static_cast<unsigned>(ctas), kThreads, smem, s>>>(maps, p);
  HEADS_CUDA(cudaGetLastError(), "kernel launch");
  if (p.groups > 1) {
    const dim3 grid(static_cast<unsigned>(p.groups), static_cast<unsigned>(p.tiles));
    HEADS_CUDA(bf ? launch_after(paged_merge_kernel<__nv_bfloat16>, grid, kMergeThreads, 0, s, p)
                  : launch_after(paged_merge_kernel<__half>, grid, kMergeThreads, 0, s, p),
               "merge launch");
  }
  return MLA_OK;
}

}  // namespace paged

cudaError_t paged_status(unsigned int* v, bool clear) { return read_status(paged::g_paged_status, v, clear); }

namespace {

mla_status check_dims(const mla_paged_dims& d) {
  const mla_status st = check_head_dims(d.n_q, d.n_kv, d.d_qk, d.d_v, d.dtype);
  if (st != MLA_OK) return st;
  if (d.B < 0 || d.S1 < 1 || d.S1 > (1 << 20)) return fail(MLA_ERR_SHAPE, "B must be >= 0, S1 in [1, 2^20]");
  if (static_cast<int64_t>(d.B) * d.S1 * d.n_q >= (1ll << 31) - 1024 || d.B > (1 << 24))
    return fail(MLA_ERR_SHAPE, "B * S1 * n_q must be below 2^31 - 1024, B at most 2^24");
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
