// Dense MLA attention over the whole paged cache for GB300 (sm_103a): single
// tokens, chains and trees of drafted tokens (formulas in mla_tree.h).
//
// All query heads and all drafted tokens of a sequence share its keys, so the
// rows of the problem are (token, head) pairs packed 128 to a block, and a
// cluster of two CTAs takes one block through a range of 256-key tiles.  A
// block's output, 128 x 512 in fp32, is half the tensor memory of two SMs;
// the pair's MMAs (cta_group::2, M = 128, N = 256, the shape that runs at the
// full rate of both SMs) leave rows 0-63 in CTA 0 and rows 64-127 in CTA 1,
// each as 128 lanes: lane m holds row m for the first half of the columns and
// lane 64 + m for the second.  No score crosses between the CTAs.
//
// Operands.  Q (64 rows x 576) stays in shared memory.  Keys and values stream
// through a ring of seven 16 KB slots, each four MMAs long (259 clocks):
//   key slot    64 dims of the CTA's 128 keys: CTA r takes page 2 t + r of tile t
//   value slot  64 keys of the CTA's 128 output dims
// The MMA reads a value from the CTA that owns its output column but a key
// from the CTA that owns the key, so every latent value comes in twice (once
// as a key half, once as a value half): 2176 bytes per key and pair, 62 bytes
// per clock and SM at the full MMA rate, below the ~77 that an SM's loads from
// L2 reach.
//
// Warps of a CTA:
//   0-7   softmax: S (64 x 256 scores as 128 lanes x 128 columns) from tensor
//         memory, mask, running maximum (lazily moved, shared by the four
//         threads of a row) and sum, P in bf16 to shared memory, rescaling
//         of O, the epilogue
//   bf16: 8-14  producers, one per ring slot: TMA; where a tile holds drafted
//         or unwritten rows, the values are mended in shared memory, since NaN
//         or infinity behind a weight of 0 would reach the second product
//   INT8: 8-15  converters, one warp that loads codes and scales (Conf<true>)
//   the last but INT8's load warp: MMA issue (CTA 0) and the loads of Q (each CTA)
// S is double buffered: S(t + 1) is computed while the softmax of tile t runs.
//
// Schedule.  Clusters form teams of g that take g row blocks of a sequence
// through the same keys side by side, so a key is read from HBM once per team;
// every team takes an equal share of the stream of tiles over all sequences.
// A row block cut between teams leaves partial states in the workspace, and a
// second launch merges them.  Which cluster takes what follows from the
// lengths alone, so results do not depend on timing.
//
// Measured (bf16).  64 sequences x 8 drafts x 128 heads over 8192 positions:
// 736 us from a cool start (1.59 PFLOP/s, 81% of the measured bf16 rate), 790 to
// 820 us back to back, where the SM clock falls to ~1.6 GHz under the power cap;
// one sequence, 64 drafts, 131072 positions: 1.51 ms, 1.55 PFLOP/s.  Bound by
// shared memory: counted once each, a tile of 256 keys moves 279 KB in, 279 KB out
// as B, 139 KB as A and 33 KB of P, 5700 clocks at 128 bytes a clock, against 4406
// clocks of MMA; ~5900 by the cycle counter of a small case, set-up taken off.
// Single tokens, 64 sequences of 8192: 145 to 154 us for 604 MB, 4.1 TB/s or 61% of
// the copy rate, ~8000 clocks a tile: neither memory nor the tensor cores (40%
// active) bind, but the latency from a load to its use over seven ring slots.
// Prefetching the next tile's keys into L2 gained nothing there, without an
// eviction priority it lost 8%, two tiles ahead 35% (lines leave L2 before their
// use: 1.04 GB read instead of 0.68).
// What shaped the kernel, at the largest case (us): arrivals on the other CTA's
// barriers with release at CTA scope instead of cluster scope 2018 -> 1682; a
// converged warp around an elected issuer instead of one running thread 2584 ->
// 2081; uniform control and two ring slots per turn 1682 -> 1575.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "../../include/mla_tree.h"
#include "ptx.cuh"

namespace mlasp {
unsigned long long host_wait_limit_ns();
}

namespace mlatree {

using namespace mlasp;

constexpr int kSoftmaxWarps = 8;
constexpr int kProducerWarp0 = 8;
// bf16: seven ring slots, a producer warp each.  INT8: four slots, filled from
// three raw slots of two items each by two groups of four converter warps, and a
// load warp.
template <bool kInt8>
struct Conf {
  static constexpr int kSlots = kInt8 ? 4 : 7;
  static constexpr int kProducers = kInt8 ? 8 : 7;
  static constexpr int kMmaWarp = kProducerWarp0 + kProducers;
  static constexpr int kThreads = (kMmaWarp + (kInt8 ? 2 : 1)) * 32;
  static constexpr int kFillers = kInt8 ? 4 : 1;  // warps of a CTA that fill one slot together
  // INT8: the softmax warps take registers over from the converters (112 and 80: 188 us instead of 183)
  static constexpr int kRegs = kInt8 ? 96 : 128, kSoftmaxRegs = 104, kConvertRegs = 88;
  static_assert(256 * kSoftmaxRegs + 256 * kConvertRegs <= 512 * 96, "register budget");
};
constexpr int kRawSlots = 3;
constexpr int kMaxThreads = 576;
static_assert(Conf<false>::kThreads == 512 && Conf<true>::kThreads == kMaxThreads, "roles");

constexpr int kRowBlock = 128;
constexpr int kTile = 256;
constexpr int kPage = 128;
constexpr int kKeyItems = 9;  // 64-dim slices of 576
constexpr int kSlotBytes = 16384;
constexpr int kRawCodes = 16384;  // two items: 128 keys x 128 codes, or twice 64 keys x 128 codes
constexpr int kRawBytes = kRawCodes + 128 * 16;  // and the rows' four scales
constexpr int kChunk = 8192;  // 64 rows of 128 bytes
constexpr int kOffQ = 0;
constexpr int kOffP = kOffQ + kKeyItems * kChunk;
constexpr int kOffRing = kOffP + 4 * kChunk;
constexpr int kOffRaw = kOffRing + Conf<true>::kSlots * kSlotBytes;  // INT8
constexpr int kOffExch = kOffRaw + kRawSlots * kRawBytes;            // float [2][4][64]
static_assert(kOffExch >= kOffRing + Conf<false>::kSlots * kSlotBytes, "ring");
static_assert(kOffRing % 1024 == 0 && kOffRaw % 1024 == 0 && kRawBytes % 1024 == 0, "swizzled tiles");
constexpr int kOffScan = kOffExch + 2048;                    // int64 [warps]
constexpr int kOffWalk = kOffScan + kMaxThreads / 32 * 8;  // int64 [4]: a share's first sequence and its stream position
constexpr int kOffBars = kOffWalk + 32;
constexpr int kMaxSlots = 7;
constexpr int kFull = 0;                   // [kMaxSlots], in CTA 0: both CTAs have filled the slot
constexpr int kEmpty = kFull + kMaxSlots;  // [kMaxSlots] the MMAs that read the slot are complete
constexpr int kSFull = kEmpty + kMaxSlots;  // [2]
constexpr int kSFree = kSFull + 2;       // [2], in CTA 0: the softmax warps have read S
constexpr int kPReady = kSFree + 2;      // in CTA 0: P is written, O may be added to
constexpr int kPvDone = kPReady + 1;
constexpr int kQFull = kPvDone + 1;  // in CTA 0
constexpr int kQFree = kQFull + 1;   // the segment's score MMAs are complete
constexpr int kMax = kQFree + 1;     // [2] the four warps of rows 0-31 / 32-63 have posted
constexpr int kFinal = kMax + 2;
constexpr int kLocal = kFinal + 1;  // [kMaxSlots] bf16: a slot's bytes have landed that the producer still has to mend
constexpr int kRawFull = kLocal + kMaxSlots;     // [kRawSlots] INT8: codes and scales have landed
constexpr int kRawEmpty = kRawFull + kRawSlots;  // [kRawSlots] INT8: they have been read
constexpr int kNumBars = kRawEmpty + kRawSlots;
constexpr int kOffTmem = kOffBars + 8 * kNumBars;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffMended = kOffAbort + 4;  // a drafted value of either CTA was NaN or infinite
constexpr int kSmemBytes = kOffMended + 4 + 1024;  // 1024: the base is aligned by hand
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kOffRing % 1024 == 0 && kOffP % 1024 == 0 && kOffBars % 8 == 0, "alignment");

constexpr uint32_t kTmemO = 0;    // two blocks of 128 columns: output dims [0, 256) and [256, 512)
constexpr uint32_t kTmemS = 256;  // two buffers of 128 columns
constexpr int kPartFloats = 128 * 256 + 128;  // one CTA's partial state: O, then m[64], l[64]
constexpr int kMaxClusters = 76;
constexpr uint64_t kDrainNs = 500ull * 1000 * 1000;

__device__ unsigned int g_tree_status = 0;

struct Params {
  const uint8_t* kv_nope;
  const float* kv_scales;
  const int32_t* block_table;
  const int32_t* act_seqs;
  const int32_t* tree_lens;
  const uint64_t* tree_mask;
  uint16_t* out;
  float* lse;
  float* parts;   // [clusters][2][2 CTAs][kPartFloats]
  int4* records;  // [clusters] what the merge has to do for a row block that starts in this cluster
  int B, S1, n_q, W, num_blocks;
  int rows;         // rows of a sequence
  int team, teams;  // clusters of a team, teams
  float scale_log2;
  int out32;
  int once;  // one cluster reads a key, once as a key and once as a value: 2% where memory binds
  unsigned long long wait_ns;
};

// ------------------------------------------------------------------ schedule
struct Seq {
  int act, n;         // cached positions, drafted tokens
  int blocks, tiles;  // row blocks that hold a drafted token, key tiles
  bool cut_table;     // positions beyond the table
  // tiles that a team goes through: passes over groups of row blocks
  __device__ int64_t len(const Params& p) const { return static_cast<int64_t>((blocks + p.team - 1) / p.team) * tiles; }
};

__device__ __forceinline__ Seq load_seq(const Params& p, int b) {
  Seq s;
  // far beyond the table a length says no more (W * 128 + S1 < 2^31)
  s.act = min(max(0, __ldg(p.act_seqs + b)), p.W * kPage + p.S1);
  s.n = p.tree_lens != nullptr ? min(p.S1, max(0, __ldg(p.tree_lens + b))) : p.S1;
  const int in_table = min(s.act, p.W * kPage);
  s.cut_table = in_table < s.act;
  s.tiles = max(1, (in_table + kTile - 1) / kTile);
  s.blocks = static_cast<int>((static_cast<int64_t>(s.n) * p.n_q + kRowBlock - 1) / kRowBlock);
  return s;
}

struct Segment {
  int b, rb;          // sequence, row block
  int t0, t1, tiles;  // tiles [t0, t1) of the row block's `tiles`
  int act, n;
  int ctx;            // first drafted position, may be negative
  int64_t first;      // stream position of the row block's first tile
};

// A team's share of the stream, walked row block by row block.
struct Walk {
  int b;
  int64_t base;       // stream position of sequence b
  int64_t off, left;  // position within sequence b, tiles left
  int member;
  __device__ bool next(const Params& p, Segment& s) {
    while (left > 0) {
      const Seq q = load_seq(p, b);
      const int64_t len = q.len(p);
      if (off >= len) {
        ++b;
        base += len;
        off = 0;
        continue;
      }
      const int pass = static_cast<int>(off / q.tiles);
      s.b = b;
      s.tiles = q.tiles;
      s.t0 = static_cast<int>(off - static_cast<int64_t>(pass) * q.tiles);
      s.t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), s.t0 + left));
      s.first = base + off - s.t0;
      s.act = q.act;
      s.n = q.n;
      s.ctx = s.act - s.n;
      s.rb = pass * p.team + member;
      off += s.t1 - s.t0;
      left -= s.t1 - s.t0;
      if (s.rb < q.blocks) return true;
    }
    return false;
  }
};

struct Ctx {
  uint32_t sb;
  uint8_t* smem;
  uint32_t tmem, rank;
  uint64_t wait_ns;
  volatile uint32_t* abort;
  __device__ volatile uint32_t* mended() const { return reinterpret_cast<volatile uint32_t*>(smem + kOffMended); }
  __device__ uint32_t bar(int i) const { return sb + kOffBars + 8 * i; }
  __device__ uint32_t lead(int i) const { return mapa_shared(bar(i), 0); }  // the barrier in CTA 0
};

__device__ __forceinline__ bool warp_wait(const Ctx& c, int i, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait<false>(c.bar(i), parity, c.abort, c.wait_ns));
}
// Arrivals on a barrier of CTA 0, with release at CTA scope: what they hand over
// is tensor memory or shared memory of the arriving CTA itself, already ordered
// for the tensor core (tcgen05.wait, fence.proxy.async), so nothing has to be
// made visible to threads of the other CTA.  Release at cluster scope waits for
// a round trip to L2, ~1500 clocks under load, in the softmax's critical path.
__device__ __forceinline__ void arrive_lead(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_lead_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cluster.b64 _, [%0], %1;"
               :: "r"(bar), "r"(bytes) : "memory");
}
// TMA load whose bytes count on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_pair(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
// The same for a box that is not read again: L2 gives its lines up first.
__device__ __forceinline__ void tma_pair_last(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void umma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// Arrive on the barrier at this offset in both CTAs when the MMAs issued so far are complete.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ int page_id(const Params& p, int b, int lb) {
  return lb < p.W ? __ldg(p.block_table + static_cast<int64_t>(b) * p.W + lb) : -1;
}
__device__ __forceinline__ bool good(const Params& p, int id) { return id >= 0 && id < p.num_blocks; }
// Key groups of 64 that tile t of a segment has to go through.
__device__ __forceinline__ int groups_of(const Segment& s, int t) {
  return min(4, max(1, (s.act - kTile * t + 63) >> 6));
}

// Sum over the threads before this one, and over the whole block.
template <int kThreads>
__device__ __forceinline__ int64_t block_sum_scan(const Ctx& c, int64_t v, int64_t& total) {
  int64_t* part = reinterpret_cast<int64_t*>(c.smem + kOffScan);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  return before + x - v;
}

// Teams that take a stream of `total` tiles: one for each tile as far as they go
// (one sequence of 16000 positions 26.9 us, with two tiles a team at least 29.0;
// 16 of 300 to 2000 25.2 and 29.4).  Of short shares no more than the longest
// needs: fewer cuts for the merge (8 sequences x 8 row blocks x 1000 positions
// 36.9 -> 29.3, 64 single tokens over 100 to 500 32.8 -> 30.7).
__device__ __forceinline__ int teams_of(const Params& p, int64_t total) {
  const int64_t teams = max(static_cast<int64_t>(1), min(static_cast<int64_t>(p.teams), total));
  const int64_t share = (total + teams - 1) / teams;
  return static_cast<int>(share > 0 && share < 8 ? (total + share - 1) / share : teams);
}

// The walk of cluster `cid`; false when it has nothing to do.
template <int kThreads>
__device__ bool start_walk(const Params& p, const Ctx& c, int cid, Walk& w, int64_t& total, int& teams) {
  int64_t* at = reinterpret_cast<int64_t*>(c.smem + kOffWalk);
  const int tid = threadIdx.x;
  const int chunks = (p.B + kThreads - 1) / kThreads;
  int64_t mine = 0, len = 0, pre = 0;
  bool beyond = false;  // positions outside the table
  for (int k = 0; k < chunks; ++k) {
    const int b = k * kThreads + tid;
    len = 0;
    if (b < p.B) {
      const Seq q = load_seq(p, b);
      len = q.len(p);
      beyond = beyond || (q.cut_table && q.n > 0);
    }
    mine += len;
  }
  if (beyond) atomicOr(&g_tree_status, MLA_DEVICE_BAD_BLOCK);
  pre = block_sum_scan<kThreads>(c, mine, total);
  teams = teams_of(p, total);
  const int team = cid / p.team;
  const bool busy = team < teams;
  const int64_t start = busy ? team * total / teams : 0, end = busy ? (team + 1) * total / teams : 0;
  if (busy) {
    int64_t carry = 0;
    for (int k = 0; k < chunks; ++k) {
      const int b = k * kThreads + tid;
      int64_t sum = total;
      if (chunks > 1) {
        len = b < p.B ? load_seq(p, b).len(p) : 0;
        pre = carry + block_sum_scan<kThreads>(c, len, sum);
      }
      if (b < p.B && start >= pre && start < pre + len) {
        at[0] = b;
        at[1] = pre;
      }
      carry += sum;
      if (carry > start) break;
    }
  }
  __syncthreads();
  w.b = static_cast<int>(at[0]);
  w.base = at[1];
  w.off = start - at[1];
  w.left = end - start;
  w.member = cid - team * p.team;
  return busy;
}

// ------------------------------------------------------------------ producers
struct Maps {
  CUtensorMap q_nope, q_rope, key, val, rope;  // key, val: of bf16 rows, or of codes
  CUtensorMap key_scale, val_scale;            // INT8
};

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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Four codes of a word times the scale, rounded to bf16: bytes enter the
// mantissa of 2^23 + 128 + code by a byte permutation (codes biased to
// unsigned), which is exact and cheaper than four conversions.
__device__ __forceinline__ void dequant4(uint32_t w, float sc, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const uint64_t bias = pair(-8388736.f, -8388736.f), s2 = pair(sc, sc);  // 2^23 + 128
  const uint64_t a = pair(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)),
                          __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441)));
  const uint64_t b = pair(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442)),
                          __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443)));
  const float2 x = unpair(mul2(add2(a, bias), s2)), y = unpair(mul2(add2(b, bias), s2));
  lo = pack_bf16x2(x.x, x.y);
  hi = pack_bf16x2(y.x, y.y);
}
// NaN and infinities of a bf16 pair become zero.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}
__device__ __forceinline__ uint4 finite8(uint4 v, bool& mended) {
  const uint4 f = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
  mended = mended || ((f.x ^ v.x) | (f.y ^ v.y) | (f.z ^ v.z) | (f.w ^ v.w)) != 0;
  return f;
}
// Tells the softmax warps of both CTAs, before the barrier that hands the values
// on: the fence returns when the other CTA's shared memory has the word.
__device__ __noinline__ void post_mended(uint32_t sb) {
#pragma unroll
  for (int r = 0; r < 2; ++r)
    asm volatile("st.shared::cluster.u32 [%0], 1;" :: "r"(mapa_shared(sb + kOffMended, r)) : "memory");
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

// First row of page `lb` of the sequence; one beyond the cache, where TMA fills
// zeros, for a page that is not used or not good.
__device__ __forceinline__ int page_row(const Params& p, const Segment& s, int lb) {
  const int id = lb * kPage < s.act ? page_id(p, s.b, lb) : -1;
  return (good(p, id) ? id : p.num_blocks) * kPage;
}

// One filling of a ring slot.
struct Item {
  int row, rows;  // first cache row (beyond the cache for a bad page), rows that exist
  int dim0;       // first dim
  bool value, rope;
  int first_draft;  // rows from here on may hold what some tokens must not see (values only)
};

// The fillings in the order in which the MMAs take them, keys of tile t + 1
// before values of tile t: every kStride-th from item k on.
template <int kStride>
struct Items {
  Walk walk;
  Segment s;
  bool open = false, values = false;
  int u = 0, k;  // tile that the keys come from; the next item, counted within the current group
  __device__ Items(const Walk& from, int first) : walk(from), k(first) {}
  __device__ bool next(const Params& p, int rank, Item& it) {
    while (true) {
      if (!open) {
        if (!walk.next(p, s)) return false;
        open = true;
        u = s.t0;
        values = false;
      }
      const int items = values ? (u > s.t0 ? 2 * groups_of(s, u - 1) : 0) : (u < s.t1 ? kKeyItems : 0);
      if (k < items) break;
      k -= items;
      if (values && ++u > s.t1) open = false;
      values = !values;
    }
    const int t = values ? u - 1 : u;
    const int lb = 2 * t + (values ? k >> 2 : rank), sub = values ? ((k >> 1) & 1) * 64 : 0;
    const int base = lb * kPage + sub;
    it.rows = max(0, min(values ? 64 : kPage, s.act - base));
    it.row = page_row(p, s, lb);
    if (it.row >= p.num_blocks * kPage) it.rows = 0;
    it.row += sub;
    it.dim0 = values ? (k & 1) * 256 + rank * 128 : 64 * k;
    it.value = values;
    it.rope = !values && k == 8;
    it.first_draft = s.ctx - base;
    k += kStride;
    return true;
  }
};

// Rows of a value item (64 keys x 128 dims, bf16, in the slot) that the second
// product must not see as they are: unwritten ones become zero, drafted ones
// lose their NaN and infinities, which a weight of 0 would carry to tokens that
// do not see them.  A token that sees such a row gets its NaN through the score,
// or, where an infinity scores -inf, from infinite_columns().
__device__ __forceinline__ void mend_values(const Ctx& c, uint32_t slot, const Item& it, int lane) {
  const int unit = lane & 15;
  bool mended = false;
  for (int r = max(0, min(it.first_draft, it.rows)) + (lane >> 4); r < 64; r += 2) {
    const uint32_t at = slot + (unit >> 3) * kChunk + r * 128 + (((unit & 7) ^ (r & 7)) << 4);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < it.rows) {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
      v = finite8(v, mended);
    }
    sts16(at, v);
  }
  if (mended) post_mended(c.sb);
}

// bf16: producer warp w fills ring slot w.
__device__ void producer_role(const Params& p, const Ctx& c, const Maps& maps, const Walk& walk, int w, int lane) {
  constexpr int kSlots = Conf<false>::kSlots;
  const uint32_t slot = c.sb + kOffRing + w * kSlotBytes;
  const uint32_t full = c.lead(kFull + w);
  const int rank = static_cast<int>(c.rank);
  uint32_t fills = 0, mended = 0;
  Items<kSlots> items(walk, w);
  Item cur, nxt;
  bool have = items.next(p, rank, cur);
  while (have) {
    const bool more = items.next(p, rank, nxt);  // its table entry is on its way while this one waits
    if (!warp_wait(c, kEmpty + w, (fills++ & 1) ^ 1)) return;
    if (cur.value) {
      const bool mend = cur.first_draft < 64 || cur.rows < 64;
      const uint32_t bar = mend ? c.bar(kLocal + w) : full;
      if (lane == 0) {
        if (mend) mbar_arrive_expect_tx(bar, kSlotBytes);
        else arrive_lead_tx(bar, kSlotBytes);
        if (p.once) {
          tma_pair_last(slot, &maps.val, cur.dim0, cur.row, bar);
          tma_pair_last(slot + kChunk, &maps.val, cur.dim0 + 64, cur.row, bar);
        } else {
          tma_pair(slot, &maps.val, cur.dim0, cur.row, bar);
          tma_pair(slot + kChunk, &maps.val, cur.dim0 + 64, cur.row, bar);
        }
      }
      __syncwarp();
      if (mend) {
        if (!warp_wait(c, kLocal + w, mended++ & 1)) return;
        mend_values(c, slot, cur, lane);
        fence_proxy_async_smem();  // generic-proxy stores -> tensor-core reads
        __syncwarp();
        if (lane == 0) arrive_lead(full);
      }
    } else {
      if (lane == 0) {
        arrive_lead_tx(full, kSlotBytes);
        if (cur.rope) tma_pair(slot, &maps.rope, 0, cur.row, full);
        else tma_pair(slot, &maps.key, cur.dim0, cur.row, full);
      }
      __syncwarp();
    }
    cur = nxt;
    have = more;
  }
}

// INT8: one warp requests the codes and scales, two items at a time (rows of
// 128 bytes: with 64 the load engine's rate per row would bind).
__device__ void raw_load_role(const Params& p, const Ctx& c, const Maps& maps, Walk walk, int lane) {
  const int rank = static_cast<int>(c.rank);
  int slot = 0;
  uint32_t phase = 1;
  // keys: 128 rows, dims [dim0, dim0 + 128); values: 64 rows, both halves of the output dims
  auto load = [&](bool value, int dim0, int row) {
    if (!warp_wait(c, kRawEmpty + slot, phase)) return false;
    if (lane == 0) {
      const uint32_t bar = c.bar(kRawFull + slot), dst = c.sb + kOffRaw + slot * kRawBytes;
      mbar_arrive_expect_tx(bar, kRawCodes + (value ? 64 : 128) * 16);
      tma_pair(dst, value ? &maps.val : &maps.key, dim0, row, bar);
      if (value) tma_pair(dst + kChunk, &maps.val, dim0 + 256, row, bar);
      tma_pair(dst + kRawCodes, value ? &maps.val_scale : &maps.key_scale, 0, row >> 6, bar);
    }
    __syncwarp();
    if (++slot == kRawSlots) {
      slot = 0;
      phase ^= 1;
    }
    return true;
  };
  Segment s;
  while (walk.next(p, s)) {
    int rows[2] = {0, 0};  // pages of the tile before
    for (int u = s.t0; u <= s.t1; ++u) {
      int next[2] = {0, 0};
      if (u < s.t1) {
        next[0] = page_row(p, s, 2 * u);
        next[1] = page_row(p, s, 2 * u + 1);
        for (int k = 0; k < 4; ++k)
          if (!load(false, 128 * k, next[rank])) return;
      }
      if (u > s.t0) {
        const int groups = groups_of(s, u - 1);
        for (int g = 0; g < groups; ++g)
          if (!load(true, rank * 128, rows[g >> 1] + (g & 1) * 64)) return;
      }
      rows[0] = next[0];
      rows[1] = next[1];
    }
  }
}

// INT8: converter warp w belongs to group w / 4 and turns a quarter of one of a
// raw slot's two items into bf16, 16 codes of a lane at a time.  Shared memory
// binds the INT8 kernel (64 single tokens over 8192 positions: 183 us, 344 MB;
// bf16 148 us, 604 MB): codes in and out, bf16 values in and the MMA's operands
// out are 990 KB a tile, 7.7 thousand clocks of the measured 11.6 (162 us with
// the arithmetic left out, 136 with the stores left out).  So eight lanes' 16
// bytes always lie in eight different banks; with two-way conflicts it took 193
// us.  Twice the warps a group 193 us, a third group 201, all arithmetic before
// the wait for the slot 197, loads by the converters themselves 274.
__device__ void convert_role(const Params& p, const Ctx& c, const Maps& maps, Walk walk, int w, int lane) {
  static_assert(Conf<true>::kSlots == 4 && Conf<true>::kProducers == 8, "two groups, four slots");
  const int rank = static_cast<int>(c.rank), group = w >> 2, quarter = w & 3;
  uint32_t item = group;  // the group's next item, counted over all items
  int raw = 0;
  uint32_t raw_phase = 0;
  auto free_slot = [&](uint32_t i) { return warp_wait(c, kEmpty + (i & 3), ((i >> 2) & 1) ^ 1); };
  // rows of 64 (us = 2) or 128 codes (us = 3); from row `mend` on the value rows
  // lose their NaN and infinities, from row `end` on they are zero
  auto convert = [&](auto us_, int scale, int mend, int end) {
    constexpr int us = decltype(us_)::value;
    if (!warp_wait(c, kRawFull + raw, raw_phase)) return false;
    const uint32_t src = c.sb + kOffRaw + raw * kRawBytes;
    // eight lanes take four 16-byte units of each of two rows, whose swizzles put
    // the loads and the stores into different banks: rows r and r ^ 5 (us = 2),
    // or r and r ^ 1 with the other half of the columns; k moves 8 or 4 rows on
    const int pair_row = lane >> 3, odd = (lane >> 2) & 1;
    const int r0 = us == 2 ? quarter * 32 + (odd ? pair_row ^ 5 : pair_row) : quarter * 16 + 2 * (pair_row >> 1) + odd;
    const int col = us == 2 ? lane & 3 : (lane & 3) + 4 * (odd ^ (pair_row & 1));
    const uint32_t codes = src + (us == 2 ? 0 : group * kChunk) + r0 * 128;
    const int unit = us == 2 ? 4 * group + col : col;
    uint4 v[4];
    float sc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int dr = (32 * k) >> us;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w) : "r"(codes + dr * 128 + ((unit ^ ((r0 + dr) & 7)) << 4)));
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sc[k]) : "r"(src + kRawCodes + (r0 + dr) * 16 + 4 * scale));
    }
    if (!free_slot(item)) return false;
    const int u0 = 2 * (col & 3);
    const uint32_t dst0 = c.sb + kOffRing + (item & 3) * kSlotBytes + (col >> 2) * kChunk;
    bool mended = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + ((32 * k) >> us);
      uint4 a, b;
      dequant4(v[k].x, sc[k], a.x, a.y);
      dequant4(v[k].y, sc[k], a.z, a.w);
      dequant4(v[k].z, sc[k], b.x, b.y);
      dequant4(v[k].w, sc[k], b.z, b.w);
      if (us == 3 && r >= mend) {
        a = r < end ? finite8(a, mended) : make_uint4(0, 0, 0, 0);
        b = r < end ? finite8(b, mended) : make_uint4(0, 0, 0, 0);
      }
      sts16(dst0 + r * 128 + ((u0 ^ (r & 7)) << 4), a);
      sts16(dst0 + r * 128 + (((u0 + 1) ^ (r & 7)) << 4), b);
    }
    if (us == 3 && mended) post_mended(c.sb);
    fence_proxy_async_smem();  // generic-proxy stores -> tensor-core reads
    __syncwarp();
    if (lane == 0) {
      arrive_lead(c.lead(kFull) + 8 * (item & 3));
      mbar_arrive(c.bar(kRawEmpty + raw));
    }
    if (++raw == kRawSlots) {
      raw = 0;
      raw_phase ^= 1;
    }
    item += 2;
    return true;
  };
  Segment s;
  while (walk.next(p, s)) {
    for (int u = s.t0; u <= s.t1; ++u) {
      if (u < s.t1) {
        const int row = page_row(p, s, 2 * u + rank);  // of the rope rows
#pragma unroll 1
        for (int k = 0; k < 4; ++k)
          if (!convert(std::integral_constant<int, 2>(), k, 0, 0)) return;
        // the rope rows are bf16: straight into the slot
        const uint32_t i = item - group;
        if (group == 0) {
          if (!free_slot(i)) return;
          if (lane == 0) {
            const uint32_t full = c.lead(kFull) + 8 * (i & 3);
            if (quarter == 0) {
              arrive_lead_tx(full, kSlotBytes);
              tma_pair(c.sb + kOffRing + (i & 3) * kSlotBytes, &maps.rope, 0, row, full);
            } else {
              arrive_lead(full);
            }
          }
          __syncwarp();
        }
        ++item;
      }
      if (u > s.t0) {
        const int groups = groups_of(s, u - 1);
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
          const int base = kTile * (u - 1) + 64 * g;
          if (!convert(std::integral_constant<int, 3>(), 2 * group + rank, s.ctx - base, s.act - base)) return;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ MMA issue and Q
__device__ __forceinline__ void load_q(const Params& p, const Ctx& c, const Maps& maps, const Segment& s) {
  const uint32_t full = c.lead(kQFull);
  const int row = s.b * p.rows + s.rb * kRowBlock + static_cast<int>(c.rank) * 64;
  arrive_lead_tx(full, kKeyItems * kChunk);
  for (int k = 0; k < 8; ++k) tma_pair(c.sb + kOffQ + k * kChunk, &maps.q_nope, 64 * k, row, full);
  tma_pair(c.sb + kOffQ + 8 * kChunk, &maps.q_rope, 0, row, full);
}

// The value of lane 0, which lets the compiler keep it in uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// One warp of each CTA; an elected lane of CTA 0's issues the pair's MMAs.  The
// warp stays converged, and what steers it (tile counts, outcomes of waits) is
// made uniform, so that descriptors and addresses live in uniform registers: a
// ring slot's four MMAs take 259 clocks to run and have to be issued in less.
template <int kSlots>
__device__ void mma_role(const Params& p, const Ctx& c, const Maps& maps, Walk walk) {
  constexpr uint32_t idesc_s = make_idesc_f16(128, 256, 1, 0, 0);  // A, B K-major
  constexpr uint32_t idesc_v = make_idesc_f16(128, 256, 1, 0, 1);  // B MN-major
  const bool lead = uniform(static_cast<int>(c.rank)) == 0;
  Segment s, nx;
  bool more = uniform(walk.next(p, s)) != 0, ok = true;
  if (more && elect_one()) load_q(p, c, maps, s);
  __syncwarp();
  int slot = 0, segs = 0, tile = 0;  // ring position, segments begun, tiles begun
  uint32_t phase = 0;
  // descriptors once; slots, chunks and k steps are additions to their address field
  const uint64_t desc_q = make_sdesc(c.sb + kOffQ, 16, 1024, kSwizzle128B);
  const uint64_t desc_p = make_sdesc(c.sb + kOffP, 16, 1024, kSwizzle128B);
  const uint64_t desc_k = make_sdesc(c.sb + kOffRing, 16, 1024, kSwizzle128B);
  const uint64_t desc_v = make_sdesc(c.sb + kOffRing, kChunk, 1024, kSwizzle128B);
  const int lane = threadIdx.x & 31;
  // Waits for the ring's next two slots (their barriers are tested side by side,
  // by even and odd lanes) or for one, and issues the four MMAs of each.  No
  // tcgen05 fence: what the wait orders is shared memory, written by TMA or
  // fenced by its writers.  After a wait that ran out nothing is issued or
  // committed: a commit would free a slot whose load is still in flight, and
  // its producer would arrive on a barrier that has no arrival left to take.
  auto take_slots = [&](bool two, uint32_t d0, uint32_t d1, uint64_t a0, uint64_t a1, uint64_t base, uint32_t b_step,
                        uint32_t idesc, bool first0, bool first1) {
    const int s0 = slot, s1 = slot + 1 == kSlots ? 0 : slot + 1;
    const uint32_t ph1 = phase ^ (s1 == 0 ? 1u : 0u);
    const bool odd = two && (lane & 1);
    const bool landed =
        mbar_wait<false>(c.bar(kFull) + 8 * (odd ? s1 : s0), odd ? ph1 : phase, c.abort, c.wait_ns);
    if (!__all_sync(0xffffffffu, landed)) return false;
    if (elect_one()) {
      const uint64_t b0 = base + static_cast<uint32_t>(s0 * (kSlotBytes >> 4));
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        umma2(d0, a0 + ks * (32 >> 4), b0 + ks * (b_step >> 4), idesc, (first0 && ks == 0) ? 0u : 1u);
      commit2(c.bar(kEmpty) + 8 * s0);
      if (two) {
        const uint64_t b1 = base + static_cast<uint32_t>(s1 * (kSlotBytes >> 4));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma2(d1, a1 + ks * (32 >> 4), b1 + ks * (b_step >> 4), idesc, (first1 && ks == 0) ? 0u : 1u);
        commit2(c.bar(kEmpty) + 8 * s1);
      }
    }
    __syncwarp();
    slot = two ? s1 + 1 : s0 + 1;
    phase = two ? ph1 : phase;
    if (slot == kSlots) {
      slot = 0;
      phase ^= 1;
    }
    return true;
  };
  auto commit = [&](int bar) {
    if (elect_one()) commit2(c.bar(bar));
    __syncwarp();
  };
  auto scores = [&](int t) {  // t: tiles begun before this one
    if (!warp_wait(c, kSFree + (t & 1), ((t >> 1) & 1) ^ 1)) return false;
    tc_fence_after();
    const uint32_t d = c.tmem + kTmemS + 128 * (t & 1);
#pragma unroll 1
    for (int k = 0; k < kKeyItems; k += 2) {
      const uint64_t a = desc_q + static_cast<uint32_t>(k * (kChunk >> 4));
      if (!take_slots(k + 1 < kKeyItems, d, d, a, a + (kChunk >> 4), desc_k, 32, idesc_s, k == 0, false)) return false;
    }
    commit(kSFull + (t & 1));
    return true;
  };
  auto values = [&](int t, int groups, bool first) {
    if (!warp_wait(c, kPReady, t & 1)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      const uint64_t a = desc_p + static_cast<uint32_t>(g * (kChunk >> 4));
      const bool begin = first && g == 0;
      if (!take_slots(true, c.tmem + kTmemO, c.tmem + kTmemO + 128, a, a, desc_v, 2048, idesc_v, begin, begin))
        return false;
    }
    commit(kPvDone);
    return true;
  };
  while (more && ok) {
    const int n = uniform(s.t1 - s.t0);
    if (lead) {
      ok = warp_wait(c, kQFull, segs & 1);
      for (int u = 0; u < n && ok; ++u) {
        ok = scores(tile + u);
        if (ok && u == n - 1) commit(kQFree);
        if (ok && u > 0) ok = values(tile + u - 1, uniform(groups_of(s, s.t0 + u - 1)), u == 1);
      }
      if (!ok) break;
    }
    // the next row block's Q as soon as this one's score MMAs are complete
    const bool again = uniform(walk.next(p, nx)) != 0;
    if (again) {
      ok = warp_wait(c, kQFree, segs & 1);
      if (!ok) break;
      if (elect_one()) load_q(p, c, maps, nx);
      __syncwarp();
    }
    if (lead) ok = values(tile + n - 1, uniform(groups_of(s, s.t1 - 1)), n == 1);
    tile += n;
    ++segs;
    s = nx;
    more = again;
  }
  // every MMA in flight lands, and its arrivals reach both CTAs, before they leave
  if (lead) commit(kFinal);
  volatile uint32_t never = 0;
  mbar_wait<false>(c.bar(kFinal), 0, &never, c.wait_ns > kDrainNs ? c.wait_ns : kDrainNs);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
// 64 bits of a mask row from bit `at` on (bits outside the row are 0).
__device__ __forceinline__ uint64_t mask_window(const uint64_t* row, int words, int64_t at) {
  const int64_t w = at >> 6;
  const int sh = static_cast<int>(at & 63);
  const uint64_t lo = w >= 0 && w < words ? __ldg(row + w) : 0ull;
  if (sh == 0) return lo;
  const uint64_t hi = w + 1 >= 0 && w + 1 < words ? __ldg(row + w + 1) : 0ull;
  return (lo >> sh) | (hi << (64 - sh));
}
__device__ __forceinline__ uint64_t low_bits(int64_t n) {
  return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1);
}
// 32-byte global store.
__device__ __forceinline__ void stg32(void* ptr, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(ptr), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// The NaN of 0 times infinity that mending the values took from a row: 128
// columns from `col` of drafted positions [lo, hi) that token `tok` sees, put
// into what the calling thread has stored: out, or its part of a partial state.
// Rare: the values of some draft were not finite.
__device__ __noinline__ void infinite_columns(const Params& p, int b, int ctx, int lo, int hi, const uint64_t* mrow,
                                              int tok, int col, uint16_t* out, float* part) {
  auto spoil = [&](int k) {
    if (out != nullptr) out[k] = 0x7FC0;
    else part[(k >> 2) * 512 + (k & 3)] = __uint_as_float(0x7FC00000u);
  };
  for (int pos = lo; pos < hi; ++pos) {
    const int j = pos - ctx, id = page_id(p, b, pos / kPage);
    if (!(mrow != nullptr ? (__ldg(mrow + (j >> 6)) >> (j & 63)) & 1 : j <= tok) || !good(p, id)) continue;
    const int64_t row = static_cast<int64_t>(id) * kPage + pos % kPage;
    if (p.kv_scales != nullptr) {
      const float scale = __ldg(p.kv_scales + row * 4 + col / 128);
      if (fabsf(scale) < 0x1p120f) continue;  // 128 codes times it stay below 2^127
      for (int k = 0; k < 128; ++k) {
        const float code = static_cast<float>(static_cast<int8_t>(__ldg(p.kv_nope + row * 512 + col + k)));
        if ((pack_bf16x2(code * scale, 0.f) & 0x7F80u) == 0x7F80u) spoil(k);
      }
    } else {
      const uint4* v = reinterpret_cast<const uint4*>(p.kv_nope + (row * 512 + col) * 2);
      for (int u = 0; u < 16; ++u) {
        const uint4 x = __ldg(v + u);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if ((w[k] & 0x7F80u) == 0x7F80u) spoil(8 * u + 2 * k);
          if ((w[k] & 0x7F800000u) == 0x7F800000u) spoil(8 * u + 2 * k + 1);
        }
      }
    }
  }
}

__device__ void softmax_role(const Params& p, const Ctx& c, Walk walk, int cid, int teams, int64_t total, int warp,
                             int lane) {
  const int q = warp & 3, sub = warp >> 2;  // TMEM lane quadrant, column half
  const int L = q * 32 + lane, row = L & 63, half = L >> 6;
  const int part = half * 2 + sub;  // which 64 keys of a tile this thread has
  const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
  const uint32_t tO = c.tmem + lanes + kTmemO + 128 * sub;
  // a positive scale leaves the order of scores alone: the maximum is taken of
  // the raw ones, and the scale goes into the exponent's multiply-add
  const bool raw = p.scale_log2 > 0.f;
  const float mul = raw ? p.scale_log2 : 1.f;
  float* exch = reinterpret_cast<float*>(c.smem + kOffExch);
  const int words = (p.S1 + 63) >> 6;
  const int maxbar = kMax + (q & 1);
  uint32_t uses = 0;  // of the exchange
  int tile = 0;       // tiles begun
  bool bad = false;
  // posts v and returns the four values of the row
  auto share = [&](float v, float (&all)[4]) {
    float* e = exch + (uses & 1) * 256;
    e[part * 64 + row] = v;
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(maxbar));
    if (!warp_wait(c, maxbar, uses & 1)) return false;
    ++uses;
#pragma unroll
    for (int k = 0; k < 4; ++k) all[k] = e[k * 64 + row];
    return true;
  };
  Segment s;
  while (walk.next(p, s)) {
    const int r = s.rb * kRowBlock + static_cast<int>(c.rank) * 64 + row;  // row of the sequence
    const int tok = min(r / p.n_q, p.S1 - 1);
    const bool live = r < p.rows && r / p.n_q < s.n;
    const uint64_t* mrow =
        p.tree_mask != nullptr ? p.tree_mask + (static_cast<int64_t>(s.b) * p.S1 + tok) * words : nullptr;
    float m = -INFINITY, l = 0.f;
    for (int t = s.t0; t < s.t1; ++t, ++tile) {
      const int buf = tile & 1;
      const int lb = 2 * t + half;
      const bool used = lb * kPage < s.act;
      const bool page = used && good(p, page_id(p, s.b, lb));
      bad = bad || (used && !page);
      uint64_t vis = page ? ~0ull : 0ull;
      if (kTile * (t + 1) > s.ctx) {
        const int64_t at = static_cast<int64_t>(kTile) * t + 64 * part - s.ctx;  // draft index of the first key
        uint64_t drafted = mrow != nullptr ? mask_window(mrow, words, at) : low_bits(tok + 1 - at);
        drafted &= low_bits(s.n - at) & ~low_bits(-at);
        vis &= live ? (low_bits(-at) | drafted) : 0ull;
      }
      if (!warp_wait(c, kSFull + buf, (tile >> 1) & 1)) return;
      tc_fence_after();
      float z[64];
      {
        uint32_t(&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(z);
        uint32_t(&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(z + 32);
        const uint32_t at = c.tmem + lanes + kTmemS + 128 * buf + 64 * sub;
        tmem_ld_32x32b_x32(at, lo);
        tmem_ld_32x32b_x32(at + 32, hi);
        tmem_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_lead(c.lead(kSFree + buf));
      if (!raw) {
#pragma unroll
        for (int k = 0; k < 64; ++k) z[k] *= p.scale_log2;
      }
      if (__any_sync(0xffffffffu, vis != ~0ull)) {
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (!((vis >> k) & 1)) z[k] = -INFINITY;
      }
      float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
      for (int k = 4; k < 64; ++k) mx[k & 3] = fmaxf(mx[k & 3], z[k]);
      float all[4];
      if (!share(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), all)) return;
      const float top = fmaxf(fmaxf(all[0], all[1]), fmaxf(all[2], all[3])) * mul;
      // the maximum moves only when a tile exceeds it by more than 2^8: P stays
      // below 2^8 and O is rarely rescaled
      const bool grow = top > m + 8.f;
      const float f = grow ? fast_exp2(m - top) : 1.f;
      if (grow) {
        l *= f;
        m = top;
      }
      const float mm = m == -INFINITY ? 0.f : m;
      uint32_t w[32];
      uint64_t sum[2] = {0, 0};
      const uint64_t mul_2 = pair(mul, mul), mm_2 = pair(-mm, -mm);
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        float2 e = unpair(fma2(pair(z[2 * k], z[2 * k + 1]), mul_2, mm_2));
        e.x = fast_exp2(e.x);
        e.y = fast_exp2(e.y);
        sum[k & 1] = add2(sum[k & 1], pair(e.x, e.y));
        // one bf16 term, off by 2^-8 of the weight at most: the second product and its operand
        // in shared memory are half of what a second term for the rest would make them
        w[k] = pack_bf16x2(e.x, e.y);
      }
      const float2 sums = unpair(add2(sum[0], sum[1]));
      l += sums.x + sums.y;
      // P and O are free once the tile before has been multiplied
      if (tile > 0 && !warp_wait(c, kPvDone, (tile - 1) & 1)) return;
      if (t > s.t0 && __any_sync(0xffffffffu, grow)) {
        tc_fence_after();
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO + 32 * ch, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          tmem_st_32x32b_x32(tO + 32 * ch, o);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      const uint32_t pr = c.sb + kOffP + part * kChunk + row * 128;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        sts16(pr + ((u ^ (row & 7)) << 4), make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_lead(c.lead(kPReady));
    }
    float all[4];
    if (!share(l, all)) return;
    l = (all[0] + all[1]) + (all[2] + all[3]);
    if (!live) {
      l = 0.f;
      m = -INFINITY;
    }
    if (!warp_wait(c, kPvDone, (tile - 1) & 1)) return;
    tc_fence_after();
    const bool whole = s.t0 == 0 && s.t1 == s.tiles;
    const int64_t grow = static_cast<int64_t>(s.b) * p.rows + r;
    if (whole) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint16_t* o = p.out + grow * 512 + sub * 256 + half * 128;
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tO + 32 * ch, v);
        tmem_wait_ld();
        if (r < p.rows) {
          uint4 y[4];
          uint32_t* yw = reinterpret_cast<uint32_t*>(y);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            yw[k] = l == 0.f ? 0u : pack_bf16x2(__uint_as_float(v[2 * k]) * inv, __uint_as_float(v[2 * k + 1]) * inv);
          if (p.out32) {
            stg32(o + 32 * ch, y[0], y[1]);
            stg32(o + 32 * ch + 16, y[2], y[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(o + 32 * ch)[k] = y[k];
          }
        }
      }
      if (*c.mended() && live && l != 0.f)
        infinite_columns(p, s.b, s.ctx, max(0, s.ctx), s.act, mrow, tok, sub * 256 + half * 128, o, nullptr);
      if (part == 0 && r < p.rows && p.lse != nullptr)
        p.lse[grow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
    } else {
      // partial state: slot 0 of the cluster when the row block began before this share, else slot 1
      const int at = s.t0 > 0 ? 0 : 1;
      float* dst = p.parts + (static_cast<int64_t>(cid * 2 + at) * 2 + c.rank) * kPartFloats;
#pragma unroll 1
      for (int ch = 0; ch < 4; ch += 2) {
        uint32_t v[64];
        tmem_ld_32x32b_x32(tO + 32 * ch, *reinterpret_cast<uint32_t(*)[32]>(v));
        tmem_ld_32x32b_x32(tO + 32 * ch + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k)
          reinterpret_cast<uint4*>(dst)[(sub * 32 + ch * 8 + k) * 128 + L] =
              make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      }
      if (*c.mended() && live)
        infinite_columns(p, s.b, s.ctx, max(max(0, s.ctx), kTile * s.t0), min(s.act, kTile * s.t1), mrow, tok,
                         sub * 256 + half * 128, nullptr, dst + (sub * 32 * 128 + L) * 4);
      if (part == 0) {
        // -inf says that the part is not the row's; the lowest maximum joins with weight 0 and
        // brings along the NaN of infinite values whose scores are all -inf
        dst[128 * 256 + row] = live ? fmaxf(m, -3.402823466e38f) : m;
        dst[128 * 256 + 64 + row] = l;
      }
      if (at == 1 && warp == 0 && lane == 0 && c.rank == 0) {
        // the teams that hold the rest: up to the one whose share has the last tile
        const int64_t last = s.first + s.tiles - 1;
        const int end = static_cast<int>(((last + 1) * teams + total - 1) / total - 1);
        p.records[cid] = make_int4(s.b * p.rows + s.rb * kRowBlock, min(kRowBlock, p.rows - s.rb * kRowBlock),
                                   end - cid / p.team, 0);
      }
    }
    tc_fence_before();  // the reads of O come before the next row block's MMAs (through kPReady)
  }
  if (bad) atomicOr(&g_tree_status, MLA_DEVICE_BAD_BLOCK);
}

template <bool kInt8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Conf<kInt8>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using K = Conf<kInt8>;
  extern __shared__ uint8_t raw[];
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  Ctx c;
  c.sb = (smem_u32(raw) + 1023u) & ~1023u;  // swizzled operands need 1024-byte alignment
  c.smem = raw + (c.sb - smem_u32(raw));
  c.rank = cluster_ctarank();
  c.wait_ns = p.wait_ns;
  c.abort = reinterpret_cast<volatile uint32_t*>(c.smem + kOffAbort);
  const int cid = blockIdx.x >> 1;
  if (tid == 0) {
    *c.abort = 0u;
    *c.mended() = 0u;
    if (c.rank == 0) p.records[cid] = make_int4(0, 0, 0, 0);  // nothing to merge, until this thread finds a cut
    for (int i = 0; i < kRawSlots; ++i) {
      mbar_init(c.bar(kRawFull + i), 1);
      mbar_init(c.bar(kRawEmpty + i), K::kProducers);
    }
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(c.bar(kFull + i), 2 * K::kFillers);
      mbar_init(c.bar(kEmpty + i), 1);
      mbar_init(c.bar(kLocal + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(c.bar(kSFull + i), 1);
      mbar_init(c.bar(kSFree + i), 2 * kSoftmaxWarps);
      mbar_init(c.bar(kMax + i), 4);
    }
    mbar_init(c.bar(kPReady), 2 * kSoftmaxWarps);
    mbar_init(c.bar(kPvDone), 1);
    mbar_init(c.bar(kQFull), 2);
    mbar_init(c.bar(kQFree), 1);
    mbar_init(c.bar(kFinal), 1);
    fence_mbarrier_init_cluster();
  }
  if (warp == K::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;"
                 :: "r"(c.sb + kOffTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  Walk walk;
  int64_t total;
  int teams;
  tc_fence_before();
  __syncthreads();  // barriers and the tensor memory address are in place
  cluster_arrive();
  const bool busy = start_walk<K::kThreads>(p, c, cid, walk, total, teams);
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // rows expanded by the launch before
  cluster_wait();
  tc_fence_after();
  c.tmem = uniform(static_cast<int>(*reinterpret_cast<volatile uint32_t*>(c.smem + kOffTmem)));

  if (busy) {
    if (warp < kSoftmaxWarps) {
      if constexpr (kInt8) regs_increase<K::kSoftmaxRegs>();
      softmax_role(p, c, walk, cid, teams, total, warp, lane);
    } else if (warp < K::kMmaWarp) {
      if constexpr (kInt8) {
        regs_decrease<K::kConvertRegs>();
        convert_role(p, c, maps, walk, warp - kProducerWarp0, lane);
      } else {
        producer_role(p, c, maps, walk, warp - kProducerWarp0, lane);
      }
    } else if (warp == K::kMmaWarp) {
      mma_role<K::kSlots>(p, c, maps, walk);
    } else {
      if constexpr (kInt8) raw_load_role(p, c, maps, walk, lane);
    }
  }
  if (p.tree_lens != nullptr) {  // rows of row blocks without a drafted token, which no cluster takes
    const int grid = static_cast<int>(gridDim.x), sharers = max(1, grid / p.B);
    for (int w = blockIdx.x; w < p.B * sharers; w += grid) {
      const int b = w % p.B, part = w / p.B;
      for (int r = load_seq(p, b).blocks * kRowBlock + part * (K::kThreads / 32) + (tid >> 5); r < p.rows;
           r += sharers * (K::kThreads / 32)) {
        const int64_t row = static_cast<int64_t>(b) * p.rows + r;
        for (int k = lane; k < 64; k += 32) reinterpret_cast<uint4*>(p.out + row * 512)[k] = make_uint4(0, 0, 0, 0);
        if (lane == 0 && p.lse != nullptr) p.lse[row] = -INFINITY;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*c.abort) {
    // a wait ran out: loads of this CTA may still be in flight to its shared
    // memory; they take microseconds
    if (tid == 0) atomicOr(&g_tree_status, MLA_DEVICE_TIMEOUT);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000) {
    }
  }
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  if (warp == K::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(c.tmem) : "memory");
}

// ------------------------------------------------------------------ INT8 rows to bf16
// Every used page of every sequence once, 16 codes of a thread at a time, into
// rows of the same number.  Bound by memory: 656 bytes in, 1024 out per row; 13
// sequences of 500 to 20000 positions, 67 thousand rows, in 14.6 us.  A block
// takes a quarter of a page, which evens the blocks out (halves 15.8, whole
// pages 24).
__global__ void __launch_bounds__(256, 8)
    tree_dequant_kernel(const int8_t* __restrict__ codes, const __grid_constant__ Params p, uint16_t* out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int col = threadIdx.x & 31, r0 = threadIdx.x >> 5;  // 16 codes of rows r0, r0 + 8, ...
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const Seq q = load_seq(p, b);
    if (q.blocks == 0) continue;
    const int pages = (min(q.act, p.W * kPage) + kPage - 1) / kPage;
    for (int i = blockIdx.x; i < 4 * pages; i += gridDim.x) {
      const int lb = i / 4, first = i % 4 * 32;  // of the page's rows
      const int id = page_id(p, b, lb);
      if (!good(p, id)) continue;
      const int rows = min(32, q.act - lb * kPage - first);
      const int64_t row0 = static_cast<int64_t>(id) * kPage + first;
      uint4 v[4];
      float sc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + 8 * k;
        v[k] = make_uint4(0, 0, 0, 0);
        sc[k] = 0.f;
        if (r < rows) {
          v[k] = __ldg(reinterpret_cast<const uint4*>(codes + (row0 + r) * 512) + col);
          sc[k] = __ldg(p.kv_scales + (row0 + r) * 4 + (col >> 3));
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + 8 * k;
        uint4 x, y;
        dequant4(v[k].x, sc[k], x.x, x.y);
        dequant4(v[k].y, sc[k], x.z, x.w);
        dequant4(v[k].z, sc[k], y.x, y.y);
        dequant4(v[k].w, sc[k], y.z, y.w);
        if (r < rows) stg32(out + (row0 + r) * 512 + col * 16, x, y);
      }
    }
  }
}

// ------------------------------------------------------------------ merge
// Joins the parts of a row block that was cut between teams.  Thread L of each of
// kGroups groups is lane L of the parts' units and takes kUnits of them (of four
// columns each); a group takes every kGroups-th part, kAhead parts at a time.
// `from`: the cluster that the row block starts in, `item`: which units.
template <int kGroups, int kUnits, int kAhead>
struct Merge {
  static constexpr int kItems = 2 * 64 / kUnits;  // of a row block
  static constexpr int kThreads = 128 * kGroups;
  float sm[kGroups > 1 ? kGroups : 1][4 * kUnits + 2][kGroups > 1 ? 128 : 1];

  __device__ void run(const Params& p, const int4& rec, int from, int item) {
    const int L = threadIdx.x & 127, group = threadIdx.x >> 7, row = L & 63, half = L >> 6;
    const int rank = item / (kItems / 2), unit = item % (kItems / 2) * kUnits;
    float m = -INFINITY, l = 0.f, o[4 * kUnits];
#pragma unroll
    for (int k = 0; k < 4 * kUnits; ++k) o[k] = 0.f;
    for (int k0 = group; k0 <= rec.z; k0 += kAhead * kGroups) {
      float mk[kAhead], lk[kAhead];
      float4 v[kAhead][kUnits];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * kGroups;
        const bool in = k <= rec.z;
        const int cl = from + (in ? k : 0) * p.team;
        const float* src = p.parts + (static_cast<int64_t>(cl * 2 + (in && k > 0 ? 0 : 1)) * 2 + rank) * kPartFloats;
        mk[u] = in ? __ldcg(src + 128 * 256 + row) : -INFINITY;
        lk[u] = in ? __ldcg(src + 128 * 256 + 64 + row) : 0.f;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) v[u][i] = __ldcg(reinterpret_cast<const float4*>(src) + (unit + i) * 128 + L);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (mk[u] == -INFINITY && lk[u] == 0.f) continue;  // a part in which the row sees nothing
        const float top = fmaxf(m, mk[u]);
        const float f = m == -INFINITY ? 0.f : exp2f(m - top), w = exp2f(mk[u] - top);
        m = top;
        l = l * f + w * lk[u];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          o[4 * i] = o[4 * i] * f + w * v[u][i].x;
          o[4 * i + 1] = o[4 * i + 1] * f + w * v[u][i].y;
          o[4 * i + 2] = o[4 * i + 2] * f + w * v[u][i].z;
          o[4 * i + 3] = o[4 * i + 3] * f + w * v[u][i].w;
        }
      }
    }
    const int r = rank * 64 + row;
    if constexpr (kGroups > 1) {
      __syncthreads();  // the last item's values have been read
      sm[group][4 * kUnits][L] = m;
      sm[group][4 * kUnits + 1][L] = l;
#pragma unroll
      for (int k = 0; k < 4 * kUnits; ++k) sm[group][k][L] = o[k];
      __syncthreads();
      if (group != 0) return;
      for (int g = 1; g < kGroups; ++g) {
        const float mg = sm[g][4 * kUnits][L], lg = sm[g][4 * kUnits + 1][L];
        if (mg == -INFINITY && lg == 0.f) continue;
        const float top = fmaxf(m, mg);
        const float f = m == -INFINITY ? 0.f : exp2f(m - top), w = exp2f(mg - top);
        m = top;
        l = l * f + w * lg;
#pragma unroll
        for (int k = 0; k < 4 * kUnits; ++k) o[k] = o[k] * f + w * sm[g][k][L];
      }
    }
    if (r >= rec.y) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t y[2 * kUnits];
#pragma unroll
    for (int k = 0; k < 2 * kUnits; ++k) y[k] = l == 0.f ? 0u : pack_bf16x2(o[2 * k] * inv, o[2 * k + 1] * inv);
    const int64_t g = rec.x + r;
    uint16_t* out = p.out + g * 512 + (unit >> 5) * 256 + half * 128 + (unit & 31) * 4;
    if constexpr (kUnits == 4) {
      const uint4 a = make_uint4(y[0], y[1], y[2], y[3]), b = make_uint4(y[4], y[5], y[6], y[7]);
      if (p.out32) {
        stg32(out, a, b);
      } else {
        reinterpret_cast<uint4*>(out)[0] = a;
        reinterpret_cast<uint4*>(out)[1] = b;
      }
    } else {
      static_assert(kUnits == 1 || kUnits == 4, "stores");
      *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[1]);
    }
    if (unit == 0 && half == 0 && p.lse != nullptr)
      p.lse[g] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  }
};

// The usual two or three parts (75 row blocks in 8 us), and up to some fifteen:
// block x looks at the record of cluster x, block y takes 16 columns of the 256
// of one CTA.
using MergeFew = Merge<1, 4, 2>;
__global__ void __launch_bounds__(MergeFew::kThreads) tree_merge_kernel(const __grid_constant__ Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel's stores are visible
  const int4 rec = p.records[blockIdx.x];
  if (rec.y == 0) return;
  MergeFew merge;
  merge.run(p, rec, blockIdx.x, blockIdx.y);
}

// A few long sequences with a part from almost every team: four groups share out
// the parts, the blocks the row blocks that there are, four columns at a time (one
// sequence of 131072 positions, attention and merge, 60 us; in the form above,
// with four groups, 68).
using MergeMany = Merge<4, 1, 4>;
__global__ void __launch_bounds__(MergeMany::kThreads, 2) tree_merge_many_kernel(const __grid_constant__ Params p) {
  __shared__ MergeMany merge;
  __shared__ int found[4], list[128];
  static_assert(kMaxClusters <= 128, "a thread for each record");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31;
  const bool cut = tid < p.team * p.teams && p.records[tid].y != 0;
  const unsigned cuts = __ballot_sync(0xffffffffu, cut);
  if (lane == 0 && tid < 128) found[tid >> 5] = __popc(cuts);
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (cut && w == tid >> 5) list[n + __popc(cuts & ((1u << lane) - 1))] = tid;
    n += found[w];
  }
  __syncthreads();
  for (int i = blockIdx.x; i < n * MergeMany::kItems; i += gridDim.x) {
    const int from = list[i / MergeMany::kItems];
    merge.run(p, p.records[from], from, i % MergeMany::kItems);
  }
}

// ------------------------------------------------------------------ host side
constexpr int kMaxDevices = 64;
struct Device {
  bool ready = false;
  int clusters[2] = {0, 0};
};
Device g_dev[kMaxDevices];
std::mutex g_lock;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// Clusters of a team, for sequences of up to `blocks` row blocks.  Large teams
// share each key's way through L2 and over the chip; whole teams and whole
// passes leave clusters idle.  Measured, us, with teams of 1 / 2 / 4 / 8 (72 of
// 76 clusters): 64 sequences x 8 row blocks x 8192 positions 1023 / 888 / 842 /
// 815; one of 64 row blocks x 131072: 1559 / 1566 / 1590 / 1509, and 1490 with
// teams of 12 to 64 although 16% of the clusters idle: such calls run at the
// power cap, where idle clusters let the others run faster, so idling counts
// 0.3.  Drafts of unequal size (1 to 17 row blocks, 13 sequences): 122 / 123 /
// 136 / 159; what a pass leaves idle there counts in full, on average over all
// sizes.  The host does not see the lengths, so equal drafts given with tree_lens
// get the smaller teams too, with tree_lens / without it: 64 x 8 row blocks x 8192
// 864 / 735 (short bursts), 16 x 4 x 4096 75.8 / 70.5, one of 64 x 131072 1575 / 1472.
inline int team_size(int blocks, int clusters, bool ragged) {
  int best = 1;
  double least = 1e30;
  for (int g = 1; g <= std::min(blocks, clusters); ++g) {
    double taken = 0, used = 0;
    for (int n = ragged ? 1 : blocks; n <= blocks; n += std::max(1, blocks / 64)) {
      taken += static_cast<double>((n + g - 1) / g) * g;
      used += n;
    }
    const double idle = taken / used * clusters / (clusters / g * g) - 1;
    const double reads = blocks == 1 || g > 6 ? 1 : (g == 1 ? 1.25 : (g == 2 ? 1.09 : (g <= 4 ? 1.04 : 1.02)));
    const double cost = reads * (1 + (ragged ? 1 : 0.3) * idle);
    if (cost <= least + 1e-9) {
      least = cost;
      best = g;
    }
  }
  return best;
}

// A sequence of several row blocks has its INT8 rows converted once, into the
// workspace, rather than by every cluster that reads them (each converts a key
// twice: as a key and as a value).  Converted by the clusters / expanded first,
// us: one row block, 64 sequences of 8192: 182 / 271; two, the same: 334 / 345,
// 64 of 100 to 8192: 107 / 112, 16 of 3000: 53 / 50; three, 64 of 8192: 494 /
// 431; up to 17, 13 of 500 to 20000: 152 / 117; 64, one of 32768: 649 / 337.
// Expanded rows keep their numbers, so they take 128 KB for each block of the
// pool, used or not; above 32,768 blocks the clusters convert.
constexpr int kExpandBlocks = 3;
constexpr size_t kExpandBytes = size_t(4) << 30;  // workspace spent on it at most

inline int row_blocks(const mla_dims& d) {
  return static_cast<int>((static_cast<int64_t>(d.S1) * d.n_q + kRowBlock - 1) / kRowBlock);
}
// Teams with a tile each in the longest stream that `passes` groups of row blocks can give.
inline int64_t most_teams(const mla_dims& d, int64_t passes) {
  return std::max<int64_t>(1, d.B * passes * ((static_cast<int64_t>(d.max_blocks_per_seq) + 1) / 2));
}

// Which merge runs: the one for many parts where a row block has more than these
// from equally long sequences.  One for few / for many parts, us, single tokens
// of B sequences, 72 teams:
//   B                     1          2          4          5          8          10
//   4096 positions    20.7/18.7  20.8/18.9  23.4/23.0  27.0/29.0  28.2/32.1  29.2/35.4
//   8192              23.6/20.7  26.8/20.9  29.6/29.2  27.0/28.9  35.0/39.0  39.0/44.6
//   32768             36.3/25.8  36.8/31.1  54.3/53.6  62.9/64.0  83.6/87.0  96.2/101.2
// and one sequence of 8 row blocks over 8192 (9 parts) 30.8/33.5.  With tables
// much wider than the lengths the same; 300 positions there 18.6/16.9 (B = 1).
constexpr int kManyParts = 16;

// The workspace: partial states, records, expanded rows.  It has room for the
// schedule of any device and any drafts (a team has at most as many clusters, a
// sequence at most as many passes as there are row blocks).
struct Workspace {
  bool expand;  // INT8: the rows are turned into bf16 first
  size_t records_at, rows_at, bytes;
};
inline Workspace workspace_of(const mla_dims& d) {
  const int blocks = row_blocks(d);
  // each factor bounded first: their product passes 64 bits for the largest dims
  const size_t room = static_cast<size_t>(
      std::min<int64_t>(kMaxClusters, std::min<int64_t>(kMaxClusters, most_teams(d, blocks)) * blocks));
  Workspace w;
  w.records_at = room * 4 * kPartFloats * sizeof(float);
  w.rows_at = (w.records_at + room * sizeof(int4) + 1023) & ~static_cast<size_t>(1023);
  const size_t rows = static_cast<size_t>(d.num_blocks) * kPage * 1024;
  w.expand = d.kv_dtype == MLA_KV_INT8 && blocks >= kExpandBlocks && rows <= kExpandBytes;
  w.bytes = w.rows_at + (w.expand ? rows : 0);
  return w;
}

struct Plan {
  int blocks, team, teams, passes, clusters;
};
inline Plan plan_of(const mla_dims& d, int clusters, bool ragged) {
  Plan s;
  s.blocks = row_blocks(d);
  s.team = team_size(s.blocks, clusters, ragged);
  s.passes = (s.blocks + s.team - 1) / s.team;
  s.teams = static_cast<int>(std::min<int64_t>(clusters / s.team, most_teams(d, s.passes)));
  s.clusters = s.team * s.teams;
  return s;
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

struct Range {
  const void* ptr;
  uint64_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.ptr || !b.ptr || !a.bytes || !b.bytes) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.ptr), y = reinterpret_cast<uintptr_t>(b.ptr);
  return x < y ? y - x < a.bytes : x - y < b.bytes;
}

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
  if (d.S1 > (1 << 20) || d.max_blocks_per_seq > (1 << 23))
    return tree_fail(MLA_ERR_SHAPE, "S1=%d above 2^20 or max_blocks_per_seq=%d above 2^23", d.S1, d.max_blocks_per_seq);
  if (static_cast<int64_t>(d.B) * d.S1 * d.n_q >= (1ll << 31) - 256)
    return tree_fail(MLA_ERR_SHAPE, "B * S1 * n_q must be below 2^31 - 256");
  return MLA_OK;
}

#define TREE_CUDA(call, what)                                                                     \
  do {                                                                                            \
    const cudaError_t err_ = (call);                                                              \
    if (err_ != cudaSuccess) return tree_fail(MLA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(err_)); \
  } while (0)

// A launch that may begin while the launch before it on the stream ends: the
// kernel waits (griddepcontrol.wait) before it touches what that one writes.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, bool early,
                         const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool kInt8>
mla_status prepare_kernel(mlatree::Device& dev) {
  using namespace mlatree;
  TREE_CUDA(cudaFuncSetAttribute(tree_attn_kernel<kInt8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes),
            "kernel set-up");
  cudaFuncAttributes fa;
  TREE_CUDA(cudaFuncGetAttributes(&fa, tree_attn_kernel<kInt8>), "kernel attributes");
  if (fa.numRegs < Conf<kInt8>::kRegs && kInt8)  // the registers that the warpgroups divide
    return tree_fail(MLA_ERR_CUDA, "the kernel was built with %d registers", fa.numRegs);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(Conf<kInt8>::kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  TREE_CUDA(cudaOccupancyMaxActiveClusters(&n, tree_attn_kernel<kInt8>, &cfg), "kernel occupancy");
  if (n < 1) return tree_fail(MLA_ERR_CUDA, "the kernel does not fit this device");
  dev.clusters[kInt8 ? 1 : 0] = std::min(n, kMaxClusters);
  return MLA_OK;
}

// Kernel attributes and the tensor-map encoder; the first call on a device.
mla_status init_device(mlatree::Device& dev) {
  using namespace mlatree;
  if (dev.ready) return MLA_OK;
  if (g_encode == nullptr) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    TREE_CUDA(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q),
              "looking up cuTensorMapEncodeTiled");
    if (fn == nullptr || q != cudaDriverEntryPointSuccess)
      return tree_fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  mla_status st = prepare_kernel<false>(dev);
  if (st == MLA_OK) st = prepare_kernel<true>(dev);
  dev.ready = st == MLA_OK;
  return st;
}

// [rows, cols] in boxes of box_cols x box_rows.
mla_status tmap(CUtensorMap* m, CUtensorMapDataType type, int size, const void* base, int64_t cols, int64_t rows,
                int box_cols, int box_rows, CUtensorMapSwizzle swizzle, const char* what) {
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(cols) * size};
  const cuuint32_t bx[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  const CUresult r = mlatree::g_encode(m, type, 2, const_cast<void*>(base), dim, stride, bx, es,
                                       CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return tree_fail(MLA_ERR_CUDA, "tensor map of %s: error %d", what, static_cast<int>(r));
  return MLA_OK;
}
// An MMA operand: bf16 in boxes of 64 columns, 128-byte swizzle.
mla_status tmap_bf16(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int box_rows, const char* what) {
  return tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, cols, rows, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B, what);
}

}  // namespace

extern "C" {

size_t mla_tree_workspace_bytes(const mla_dims* dims) {
  g_tree_error[0] = '\0';
  if (dims == nullptr || check_dims(*dims) != MLA_OK) return 0;
  return mlatree::workspace_of(*dims).bytes;
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
  const mlatree::Workspace ws = mlatree::workspace_of(d);
  if (workspace_bytes < ws.bytes)
    return tree_fail(MLA_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, ws.bytes);
  // clusters read and write in no order: nothing that a call reads may be an output
  const uint64_t toks = static_cast<uint64_t>(d.B) * d.S1, heads = toks * d.n_q, pool = 128ull * d.num_blocks;
  const Range in[] = {{q_nope, heads * 1024}, {q_rope, heads * 128}, {kv_nope, pool * (int8 ? 512 : 1024)},
                      {kv_rope, pool * 128}, {int8 ? kv_scales : nullptr, pool * 16},
                      {block_table, 4ull * d.B * d.max_blocks_per_seq}, {act_seqs, 4ull * d.B}, {tree_lens, 4ull * d.B},
                      {tree_mask, 8 * toks * ((d.S1 + 63) / 64)}};
  const Range outs[] = {{out, heads * 1024}, {lse, heads * 4}, {workspace, ws.bytes}};
  for (const Range& o : outs)
    for (const Range& i : in)
      if (overlap(o, i)) return tree_fail(MLA_ERR_UNSUPPORTED, "an output or the workspace overlaps an input");
  if (overlap(outs[0], outs[1]) || overlap(outs[0], outs[2]) || overlap(outs[1], outs[2]))
    return tree_fail(MLA_ERR_UNSUPPORTED, "out, lse and the workspace overlap");
  int dev = 0;
  TREE_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev < 0 || dev >= mlatree::kMaxDevices) return tree_fail(MLA_ERR_UNSUPPORTED, "device ordinal %d too large", dev);
  int clusters = 0;
  {
    std::lock_guard<std::mutex> guard(mlatree::g_lock);
    const mla_status ist = init_device(mlatree::g_dev[dev]);
    if (ist != MLA_OK) return ist;
    clusters = std::min(mlatree::g_dev[dev].clusters[0], mlatree::g_dev[dev].clusters[1]);
  }
  const mlatree::Plan plan = mlatree::plan_of(d, clusters, tree_lens != nullptr);
  mlatree::Params p;
  p.kv_nope = static_cast<const uint8_t*>(kv_nope);
  p.kv_scales = int8 ? kv_scales : nullptr;
  p.block_table = block_table;
  p.act_seqs = act_seqs;
  p.tree_lens = tree_lens;
  p.tree_mask = tree_mask;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.parts = static_cast<float*>(workspace);
  p.records = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + ws.records_at);
  p.B = d.B;
  p.S1 = d.S1;
  p.n_q = d.n_q;
  p.W = d.max_blocks_per_seq;
  p.num_blocks = d.num_blocks;
  p.rows = d.S1 * d.n_q;
  p.team = plan.team;
  p.teams = plan.teams;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  p.out32 = aligned(out, 32) ? 1 : 0;
  p.once = plan.blocks == 1 ? 1 : 0;
  p.wait_ns = mlasp::host_wait_limit_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* latent = kv_nope;
  if (ws.expand) {
    uint16_t* wide = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + ws.rows_at);
    const int per_seq = std::max(1, std::min(4 * d.max_blocks_per_seq, 152 * 32 / d.B));
    mlatree::tree_dequant_kernel<<<dim3(static_cast<unsigned>(per_seq), static_cast<unsigned>(std::min(d.B, 65535))), 256, 0, s>>>(
        static_cast<const int8_t*>(kv_nope), p, wide);
    TREE_CUDA(cudaGetLastError(), "INT8 expansion launch");
    latent = wide;
  }
  const bool codes = int8 && !ws.expand;  // the attention kernel reads codes
  const int64_t rows = static_cast<int64_t>(d.num_blocks) * 128, tokens = static_cast<int64_t>(d.B) * p.rows;
  mlatree::Maps maps;
  mla_status ms = tmap_bf16(&maps.q_nope, q_nope, 512, tokens, 64, "q_nope");
  if (ms == MLA_OK) ms = tmap_bf16(&maps.q_rope, q_rope, 64, tokens, 64, "q_rope");
  if (ms == MLA_OK) ms = tmap_bf16(&maps.rope, kv_rope, 64, rows, 128, "kv_rope");
  if (codes) {  // scales as they lie, codes swizzled like every other tile
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const CUtensorMapSwizzle flat = CU_TENSOR_MAP_SWIZZLE_NONE;
    if (ms == MLA_OK) ms = tmap(&maps.key, u8, 1, kv_nope, 512, rows, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B, "kv_nope");
    if (ms == MLA_OK) ms = tmap(&maps.val, u8, 1, kv_nope, 512, rows, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B, "kv_nope");
    // the scales of 64 rows as one row of the map: 1 KB at a time instead of 16 bytes
    if (ms == MLA_OK) ms = tmap(&maps.key_scale, f32, 4, kv_scales, 256, rows / 64, 256, 2, flat, "kv_scales");
    if (ms == MLA_OK) ms = tmap(&maps.val_scale, f32, 4, kv_scales, 256, rows / 64, 256, 1, flat, "kv_scales");
  } else {
    if (ms == MLA_OK) ms = tmap_bf16(&maps.key, latent, 512, rows, 128, "kv_nope");
    if (ms == MLA_OK) ms = tmap_bf16(&maps.val, latent, 512, rows, 64, "kv_nope");
    maps.key_scale = maps.val_scale = maps.rope;  // not used
  }
  if (ms != MLA_OK) return ms;
  const dim3 grid(static_cast<unsigned>(2 * plan.clusters));
  if (codes)
    TREE_CUDA(launch_after(mlatree::tree_attn_kernel<true>, grid, mlatree::Conf<true>::kThreads, mlatree::kSmemBytes, s,
                           false, maps, p),
              "kernel launch");
  else
    TREE_CUDA(launch_after(mlatree::tree_attn_kernel<false>, grid, mlatree::Conf<false>::kThreads, mlatree::kSmemBytes,
                           s, ws.expand, maps, p),
              "kernel launch");
  if (plan.teams > 1)
    TREE_CUDA(plan.teams > mlatree::kManyParts * static_cast<int64_t>(d.B) * plan.passes
                  ? launch_after(mlatree::tree_merge_many_kernel, dim3(2 * 152), mlatree::MergeMany::kThreads, 0, s, true, p)
                  : launch_after(mlatree::tree_merge_kernel, dim3(static_cast<unsigned>(plan.clusters), mlatree::MergeFew::kItems),
                                 mlatree::MergeFew::kThreads, 0, s, true, p),
              "merge launch");
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
