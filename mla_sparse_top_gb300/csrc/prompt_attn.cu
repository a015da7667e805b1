// Attention of prompts for GB300 (sm_103a); formulas in mla_heads.h.
//
// Rows are (token, head) pairs of one key head, token by token, 128 to a tile:
// floor(128 / G) tokens and their G heads.  A CTA takes two tiles side by side
// through the same 128-key tiles, so that the tensor cores work on one while
// the softmax of the other runs:
//   S_i = Q_i K^T      128 x 128 in tensor memory, both operands in shared memory
//   P_i                over S_i in tensor memory, two 16-bit weights to a column
//   O_i += P_i V       128 x d_v in tensor memory, P from there, V from shared memory
// in the order P_0 V(t), Q_0 K(t+1), P_1 V(t), Q_1 K(t+1), so that a softmax has
// the length of two products.  The 512 columns of tensor memory hold two of each;
// where d_v is at most 64, P has columns of its own, and Q K(t+1) comes before P V(t).
// A score product of one CTA reads both operands from shared memory, which takes
// 96 clocks of an MMA's 64; where there are rows enough, pairs of CTAs hold half of
// the keys and of the values' columns each and issue MMAs of 256 rows (in_pairs).
//
// Keys and values stream through a ring of 16 KB slots (128 keys x 64 values of a
// key, 64 keys x 128 or 128 keys x 64 of a value; a pair's have half of that); Q stays.
//
// Warps: 0-3 and 4-7 softmax and epilogue of tile 0 and 1, one row to a thread;
// 8 MMA issue; 9 TMA loads; 10 the schedule; 11 mends value rows that not every
// token of the item sees (rows behind the sequence become zero, others lose
// their NaN and infinities, which a weight of 0 would carry into the product).
//
// Schedule.  An item is (sequence, key head, two row tiles), from the last rows
// (which see most keys) to the first, heads in groups whose keys and values fit
// L2 side by side.  CTAs draw items from a counter.  Where there are too few for
// the GPU, the key tiles of an item are cut into parts, whose states go to the
// workspace and are joined by a launch of their own.  What is cut follows from the
// lengths alone, so results do not depend on timing.
//
// Bound by the chain of a row tile (score product, softmax of some 1750 clocks, value
// product, 2900 to 3000 clocks a key tile where the MMAs of both tiles take 2560) and,
// in long runs, by the power cap.  Measured (graph replay): 8192 tokens, 128 heads of 192
// and 128, causal, 1600 to 1720 us (1.60 to 1.72 PFLOP/s; tensor cores active 75% of the
// time); 32 heads of 128 on 8 key heads 344 (1.60 PFLOP/s), every key seen 660 (1.67).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "heads.h"
#include "heads_device.cuh"

namespace mlaheads {

__device__ unsigned int g_prompt_status = 0;

cudaError_t prompt_status(unsigned int* v, bool clear) { return read_status(g_prompt_status, v, clear); }

constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kPlanWarp = 10, kMendWarp = 11;
constexpr int kThreads = 384;
constexpr int kRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kRegs, "register budget");
constexpr int kTile = 128;
constexpr int kChunk = 16384;  // 128 rows of 64 columns
constexpr int kMaxSlots = 20;
constexpr int kTileSmem = 14 * kChunk;  // Q and ring together
constexpr int kItemSlots = 2;
constexpr int kDrawTiles = 1;  // key tiles of an item still to be loaded when the next is drawn
constexpr int kItemReaders = kSoftmaxWarps + 3;  // MMA, load and mend warps

// A CTA alone, or a pair of them that shares the keys and values of its rows.
template <bool kPair>
struct Shape {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTiles = 2 * kCtas;  // row tiles of an item
  static constexpr int kSlotBytes = kChunk / kCtas;
  __host__ __device__ static constexpr int slots(int kc) {
    const int n = (kTileSmem - 2 * kc * kChunk) / kSlotBytes;
    return n < kMaxSlots ? n : kMaxSlots;
  }
};

constexpr int kFull = 0;                     // [kMaxSlots] the slot's bytes have landed and are mended
constexpr int kEmpty = kFull + kMaxSlots;    // [kMaxSlots] the MMAs that read the slot are complete
constexpr int kLocal = kEmpty + kMaxSlots;   // [kMaxSlots] bytes have landed that are still to be mended
constexpr int kQFull = kLocal + kMaxSlots;   // [2]
constexpr int kQFree = kQFull + 2;           // [2] the item's last score MMAs are complete
constexpr int kSFull = kQFree + 2;           // [2] scores, and every MMA before them, are complete
constexpr int kPReady = kSFull + 2;          // [2] weights are written, O is rescaled
constexpr int kOFull = kPReady + 2;          // [2] the item's MMAs are complete
constexpr int kItemFull = kOFull + 2;        // [kItemSlots]
constexpr int kItemEmpty = kItemFull + kItemSlots;
constexpr int kDraw = kItemEmpty + kItemSlots;  // the item's loads are nearly all issued
constexpr int kSFree = kDraw + 1;             // [2] apart: scores are in registers
constexpr int kPFree = kSFree + 2;             // [2] apart: the MMAs that read the weights, and wrote O, are complete
constexpr int kFinal = kPFree + 2;
constexpr int kNumBars = kFinal + 1;

struct Item {
  int live;        // 0: no more items
  int b, hk, m;    // sequence, key head, group of row tiles
  int n, len, pos; // queries, keys within the table, position of query 0 (may be negative)
  int q0, key0;    // first query row, first packed key row
  int t0, ta, tb;  // key tiles [t0, ta) of a CTA's row tile 0, [t0, tb) of row tile 1
  int lo;          // keys from here on are not seen by every row
  int part;        // slot of a partial state, -1: the item is whole
  __device__ __forceinline__ int t1(int h) const { return h ? tb : ta; }
  // as four 16-byte words, field by field: through pointers it would live in local memory
  __device__ __forceinline__ void unpack(int4 w0, int4 w1, int4 w2, int4 w3) {
    live = w0.x; b = w0.y; hk = w0.z; m = w0.w;
    n = w1.x; len = w1.y; pos = w1.z; q0 = w1.w;
    key0 = w2.x; t0 = w2.y; ta = w2.z; tb = w2.w;
    lo = w3.x; part = w3.y;
  }
  __device__ __forceinline__ int4 word(int i) const {
    return i == 0 ? make_int4(live, b, hk, m) : i == 1 ? make_int4(n, len, pos, q0) : i == 2 ? make_int4(key0, t0, ta, tb) : make_int4(lo, part, 0, 0);
  }
};
constexpr int kItemBytes = 64;

constexpr int kOffItems = kTileSmem;
constexpr int kOffBars = kOffItems + kItemSlots * kItemBytes;
constexpr int kOffTmem = kOffBars + 8 * kNumBars;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffMended = kOffAbort + 4;
constexpr int kSmemBytes = kOffMended + 4 + 1024;  // 1024: the base is aligned by hand
static_assert(kSmemBytes <= 232448 && kOffBars % 8 == 0, "shared memory");

// Columns of tensor memory: two S of 128, two O, and where values have up to 64 columns, P
// apart from S, so that the next S of a row tile is made while the softmax of this one runs
// (16 heads of 64, 300 tokens 14.1 -> 13.4 us; 32 heads, four prompts of 4096 333 -> 326).
constexpr uint32_t kTmemS = 0;
template <bool kApart>
struct Tmem {
  static constexpr uint32_t kO = kApart ? 384 : 256, kOStep = kApart ? 64 : 128;
  static constexpr uint32_t kP = kApart ? 256 : kTmemS, kPStep = kApart ? 64 : 128;
};

// What the plan leaves for the other kernels, followed by three int32 arrays over the sequences.
struct Head {
  int items;    // parts of all items
  int next;     // drawn so far
  int states;   // partial states
  int failed;   // a wait ran out: not every part was written, nothing is joined
  int cap;      // key tiles of a part at most
  int pad[3];
};
// Of a partial state: the item that it is a part of.
struct Record {
  int row0, tokens;  // first query row, rows from there on that are written
  int hk;
  int cut, cuts;     // the part, of so many
  int pad[3];
};

struct Params {
  Problem x;
  Head* head;
  // of the sequences in the order in which they are taken up
  int* first;    // [B + 1] first part of an item
  int* part0;    // [B] first partial state
  int* order;    // [B] the sequence
  Record* records;  // [max_parts]
  float* parts;
  int part_floats, max_parts;
  int G, tpt;    // heads to a key head, tokens of a row tile
  int tiles, span;  // row tiles of an item, tokens of them
  int kc, vc;    // 64-column chunks of a key, of a value
  int slots;
  int sms;       // or pairs of them
  uint32_t idesc_s, idesc_v;
  int ks_qk;     // 16-wide steps of a key
  unsigned long long wait_ns;
};

struct Maps {
  CUtensorMap q, k, v;
};

struct Seq {
  int n, len, pos, q0, key0, pairs;
  bool bad_len, bad_table;
};
__device__ __forceinline__ Seq load_seq(const Params& p, int b) {
  const Problem& x = p.x;
  Seq s;
  s.bad_len = s.bad_table = false;
  s.key0 = 0;
  auto range = [&](const int32_t* cu, int most, int& first) {
    const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
    first = min(max(lo, 0), most);
    const int end = min(max(hi, 0), most);
    s.bad_len = s.bad_len || first != lo || end != hi || end < first;
    return max(0, end - first);
  };
  if (x.S1 > 0) {
    s.q0 = b * x.S1;
    s.n = x.q_lens != nullptr ? min(x.S1, max(0, __ldg(x.q_lens + b))) : x.S1;
  } else {
    s.n = range(x.cu_q, x.T, s.q0);
  }
  int len;
  if (x.num_blocks > 0) {
    len = max(0, __ldg(x.act_seqs + b));
    s.len = min(len, x.W * kPage);
    s.bad_table = s.len < len && s.n > 0;
  } else {
    len = range(x.cu_k != nullptr ? x.cu_k : x.cu_q, x.Tk, s.key0);
    s.len = len;
  }
  s.pos = len - s.n;
  // padded rows are items too: they are written
  const int tokens = x.S1 > 0 ? x.S1 : s.n;
  s.pairs = (tokens + p.span - 1) / p.span;
  return s;
}
// Keys that the first `tokens` queries see.
__device__ __forceinline__ int seen_by(const Params& p, const Seq& s, int tokens) {
  if (s.n == 0) return 0;
  return p.x.causal ? min(s.len, max(0, s.pos + min(tokens, s.n))) : s.len;
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }

// How the items of a key head of a sequence are cut: the pair of row tiles m into
// of(m) parts of at most `cap` tiles.  The later a pair, the more keys it sees, so
// parts are numbered from the last pair to the first: all that are cut come before
// those that are whole.
struct Cuts {
  int pairs, most, cap;  // pairs, parts of the last one
  int all;               // parts that every pair has
  int rows, pos;         // tokens of a pair, position of query 0
  // `last`: key tiles of the last pair
  __device__ __forceinline__ Cuts(const Params& p, int pairs_, int last, int pos_, int cap_) : pairs(pairs_), cap(cap_), rows(p.span), pos(pos_) {
    most = max(1, (last + cap - 1) / cap);
    all = p.x.causal && pairs > 1 ? min(most, static_cast<int>(static_cast<uint32_t>(max(pos, 0)) / (static_cast<uint32_t>(cap) * kTile)) + 1) : most;
  }
  // pairs that are cut into `c` parts or more: those that see more than c - 1 parts' keys
  __device__ __forceinline__ int at_least(int c) const {
    if (c <= all) return pairs;
    if (c > most) return 0;
    const uint32_t behind = static_cast<uint32_t>((c - 1) * cap * kTile) - static_cast<uint32_t>(pos);  // above 0, below 2^32
    return pairs - static_cast<int>(min(static_cast<uint32_t>(pairs), behind / static_cast<uint32_t>(rows)));
  }
  __device__ __forceinline__ int64_t parts() const {  // of a key head
    int64_t n = static_cast<int64_t>(all) * pairs;
#pragma unroll 1
    for (int c = all + 1; c <= most; ++c) n += at_least(c);
    return n;
  }
  // pair, part and parts of a key head's part k
  __device__ __forceinline__ void find(int k, int& m, int& cut, int& cuts) const {
    int behind = 0, c = most;  // pairs with more parts
#pragma unroll 1
    for (; c > all; --c) {
      const int here = at_least(c) - behind;
      if (k < here * c) break;
      k -= here * c;
      behind += here;
    }
    m = pairs - 1 - behind - k / c;
    cut = k % c;
    cuts = c;
  }
};
__device__ __forceinline__ Cuts cuts_of(const Params& p, const Seq& s, int cap) { return Cuts(p, s.pairs, tiles_of(seen_by(p, s, s.n)), s.pos, cap); }

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 512;
constexpr int kMinTiles = 4;    // key tiles of a part at least
constexpr int64_t kMostItems = (int64_t(1) << 31) - 384;  // and drawn ones behind them
constexpr int kRankSeqs = 256;  // sequences of which the longest come first
constexpr int kWarpSeqs = 32;   // sequences that a warp plans, one to a lane

// Sums over the threads before this one, and over the block.
template <int N>
__device__ __forceinline__ void plan_scan(int64_t (&v)[N], int64_t (&total)[N], int64_t (*part)[kPlanThreads / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int64_t x = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part[i][warp] = x;
    v[i] = x - v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    total[i] = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) v[i] += part[i][w];
      total[i] += part[i][w];
    }
  }
  __syncthreads();
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Parts of at most `cap` tiles.  The candidates are an SM's share of the work, a half, a third
// and a fifth of it (long items among short ones), and as many parts to an item as one to four
// rounds of the SMs have (items alike: chunks over long contexts); or nothing is cut.
constexpr int kCandidates = 8;
__device__ __forceinline__ int share_of(const Params& p, int64_t work) {
  int64_t rest;
  return static_cast<int>(min(divide(work + p.sms - 1, p.sms, rest), static_cast<int64_t>(1) << 24));
}
__device__ __forceinline__ int cap_of(const Params& p, int share, int most, int64_t items, int i) {
  if (i < 4) return max(kMinTiles, share / (i == 3 ? 5 : i + 1));
  const int each = max(1, (i - 3) * p.sms / static_cast<int>(max(static_cast<int64_t>(1), min(items, static_cast<int64_t>(1) << 24))));
  return max(kMinTiles, (most + each - 1) / each);
}
// When a plan is estimated to end, in key tiles: an item's end costs two, that of a part three
// more, and parts alike take whole rounds of the SMs; behind that the second launch joins the
// states.  Against an even share of the work plus half of the longest part, which leaves
// rounds out: 128 tokens over 100000 keys 231 -> 166 us, 512 over 30000 236 -> 209, three
// chunks of 257 to 300 over 5000 to 60000 252 -> 225, 8 of 64 over 8000 108 -> 86.
// Rounded step by step: the merge's plan and the attention's have to agree.
__device__ __forceinline__ float time_of(const Params& p, int64_t work, int64_t parts, int64_t states, int longest) {
  const int n = static_cast<int>(max(static_cast<int64_t>(1), min(parts, static_cast<int64_t>(1) << 30)));
  const int rounds = (n + p.sms - 1) / p.sms;
  const float all = __ll2float_rn(work + 2ll * n + 3 * states);
  const float even = __fdiv_rn(__fmul_rn(__int2float_rn(rounds), all), __int2float_rn(n));
  return __fadd_rn(fmaxf(even, __int2float_rn(longest + 2)), states > 0 ? __int2float_rn(2 + static_cast<int>(states / 64)) : 0.f);
}
// Whether a plan with cuts can end before `least`.
__device__ __forceinline__ bool cuts_may_pay(const Params& p, int64_t work, int64_t items, int most, float least) {
  return most > kMinTiles && p.max_parts > 0 && __fadd_rn(__fdiv_rn(__ll2float_rn(work + 2 * items), __int2float_rn(p.sms)), 2.f) < least;
}
// Key tiles of a sequence's items: the first and the last, between which they grow evenly.
__device__ __forceinline__ int64_t work_of(const Params& p, const Seq& s, int last) {
  return static_cast<int64_t>(s.pairs) * p.x.n_kv * (tiles_of(seen_by(p, s, p.span)) + last) / 2;
}
// Parts and partial states of a sequence.
__device__ __forceinline__ void count_parts(const Params& p, const Seq& s, int cap, int64_t (&v)[2]) {
  const Cuts cuts = cuts_of(p, s, cap);
  v[0] = cuts.parts() * p.x.n_kv;
  v[1] = v[0] - static_cast<int64_t>(cuts.pairs - cuts.at_least(2)) * p.x.n_kv;
}
__device__ __forceinline__ void report_seq(bool bad_len, bool bad_table) {
  if (bad_len || bad_table)
    atomicOr(&g_prompt_status, (bad_len ? MLA_DEVICE_BAD_LENGTH : 0u) | (bad_table ? MLA_DEVICE_BAD_BLOCK : 0u));
}

// The plan of few sequences: lane i has the i-th in the order in which they are taken up.
struct WarpPlan {
  int items, states, cap;
  int seq, first, part0;
  Seq s;
};
__device__ __forceinline__ WarpPlan plan_warp(const Params& p) {
  const int B = p.x.B, lane = threadIdx.x & 31;
  WarpPlan w;
  Seq s = {};
  int last = -1;
  int64_t work = 0;
  if (lane < B) {
    s = load_seq(p, lane);
    last = tiles_of(seen_by(p, s, s.n));
    work = work_of(p, s, last);
  }
  work = warp_sum(work);
  const int most = __reduce_max_sync(0xffffffffu, last);
  w.cap = max(most, 1);
  const int64_t items = warp_sum(static_cast<int64_t>(s.pairs) * p.x.n_kv);
  float least = time_of(p, work, items, 0, most);
  if (cuts_may_pay(p, work, items, most, least)) {  // four lanes to a candidate
    const int cap = cap_of(p, share_of(p, work), most, items, lane >> 2);
    int states = 0, extra = 0;  // parts that cuts make more
#pragma unroll 1
    for (int i = lane & 3; i < ((B + 3) & ~3); i += 4) {
      const int n = __shfl_sync(0xffffffffu, s.pairs, i), end = __shfl_sync(0xffffffffu, last, i), pos = __shfl_sync(0xffffffffu, s.pos, i);
      if (i < B) {
        const Cuts cuts(p, n, end, pos, min(cap, most));
        const int64_t more = (cuts.parts() - n) * p.x.n_kv;
        extra += static_cast<int>(min(more, static_cast<int64_t>(1) << 20));
        states += static_cast<int>(min(more + static_cast<int64_t>(cuts.at_least(2)) * p.x.n_kv, static_cast<int64_t>(1) << 20));
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      states += __shfl_xor_sync(0xffffffffu, states, o);
      extra += __shfl_xor_sync(0xffffffffu, extra, o);
    }
    const float time = cap < most && states <= p.max_parts ? time_of(p, work, items + extra, states, cap) : INFINITY;
#pragma unroll 1
    for (int i = 0; i < 32; i += 32 / kCandidates) {
      const float other = __shfl_sync(0xffffffffu, time, i);
      const int its = __shfl_sync(0xffffffffu, cap, i);
      if (other < least) {
        least = other;
        w.cap = its;
      }
    }
  }
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < B; ++i) {
    const int other = __shfl_sync(0xffffffffu, last, i);
    rank += other > last || (other == last && i < lane) ? 1 : 0;
  }
  w.seq = 0;
#pragma unroll 1
  for (int i = 0; i < B; ++i)
    if (__shfl_sync(0xffffffffu, rank, i) == lane) w.seq = i;
  auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, w.seq); };
  w.s.n = of(s.n);
  w.s.len = of(s.len);
  w.s.pos = of(s.pos);
  w.s.q0 = of(s.q0);
  w.s.key0 = of(s.key0);
  w.s.pairs = of(s.pairs);
  w.s.bad_len = of(s.bad_len ? 1 : 0) != 0;
  w.s.bad_table = of(s.bad_table ? 1 : 0) != 0;
  int64_t counts[2] = {0, 0};
  if (lane < B) count_parts(p, w.s, w.cap, counts);
  // a sequence has fewer than 2^26 items, but where offsets run back and forth, which is reported
  constexpr int kMost = (1 << 26) - 1;
  const int v[2] = {static_cast<int>(min(counts[0], static_cast<int64_t>(kMost))), static_cast<int>(counts[1])};
  int upto[2] = {v[0], v[1]};
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int y = __shfl_up_sync(0xffffffffu, upto[j], o);
      if (lane >= o) upto[j] += y;
    }
  }
  w.first = lane < B ? upto[0] - v[0] : 0x7FFFFFFF;
  w.part0 = upto[1] - v[1];
  const int parts = __shfl_sync(0xffffffffu, upto[0], 31);
  w.items = parts < kMost ? parts : 0;
  w.states = parts < kMost ? __shfl_sync(0xffffffffu, upto[1], 31) : 0;
  return w;
}

// Counts the work, decides what is cut, puts the sequences with the longest items
// first, which leaves short ones to even out the end, and numbers everything.  Few
// sequences are a warp's work, which every CTA of the attention does again for itself
// rather than wait for this launch and read what it wrote (5 + 5 us of a call);
// more are a block's, which goes round three times only.
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const __grid_constant__ Params p) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ int64_t part[2][kWarps];
  __shared__ int64_t works[kWarps], counts[kWarps];
  __shared__ float times[kCandidates];
  __shared__ int mosts[kWarps], lengths[kRankSeqs], order[kRankSeqs];
  const int B = p.x.B, Hkv = p.x.n_kv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = (B + kPlanThreads - 1) / kPlanThreads;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (B <= kWarpSeqs) {  // one warp was launched
    if (lane == 0) p.head->next = p.head->failed = 0;
    const WarpPlan w = plan_warp(p);
    if (lane < B) report_seq(w.s.bad_len, w.s.bad_table);
    if (lane == 0) p.head->states = w.states;
    return;
  }
  int64_t work = 0, items = 0;  // key tiles of all items
  int most = 0;                 // of an item
  bool bad_len = false, bad_table = false;
  for (int c = 0; c < chunks; ++c) {
    const int b = c * kPlanThreads + tid;
    if (b >= B) break;
    const Seq s = load_seq(p, b);
    bad_len = bad_len || s.bad_len;
    bad_table = bad_table || s.bad_table;
    const int last = tiles_of(seen_by(p, s, s.n));
    work += work_of(p, s, last);
    items += static_cast<int64_t>(s.pairs) * Hkv;
    most = max(most, last);
    if (B <= kRankSeqs) lengths[b] = last;
  }
  report_seq(bad_len, bad_table);
  work = warp_sum(work);
  items = warp_sum(items);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    works[warp] = work;
    counts[warp] = items;
    mosts[warp] = most;
  }
  __syncthreads();
  work = items = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    work += works[w];
    items += counts[w];
    most = max(most, mosts[w]);
  }
  const int share = share_of(p, work);
  if (warp < kCandidates) {
    const int cap = cap_of(p, share, most, items, warp);
    int64_t states = 0, parts = 0;
    if (cap < most && p.max_parts > 0) {
      for (int b = lane; b < B; b += 32) {
        int64_t v[2];
        count_parts(p, load_seq(p, b), cap, v);
        parts += v[0];
        states += v[1];
      }
    }
    states = warp_sum(states);
    parts = warp_sum(parts);
    if (lane == 0) times[warp] = cap < most && p.max_parts > 0 && states <= p.max_parts ? time_of(p, work, parts, states, cap) : INFINITY;
  } else if (warp == kCandidates) {  // ranks
    for (int b = lane; b < B && B <= kRankSeqs; b += 32) {
      int rank = 0;
      for (int i = 0; i < B; ++i) rank += lengths[i] > lengths[b] || (lengths[i] == lengths[b] && i < b) ? 1 : 0;
      order[rank] = b;
    }
  }
  __syncthreads();
  int cap = max(most, 1);
  float least = time_of(p, work, items, 0, most);
#pragma unroll
  for (int i = 0; i < kCandidates; ++i) {
    if (times[i] < least) {
      least = times[i];
      cap = cap_of(p, share, most, items, i);
    }
  }
  int64_t carry[2] = {0, 0};  // parts, partial states
  for (int c = 0; c < chunks; ++c) {
    const int i = c * kPlanThreads + tid;
    int64_t v[2] = {0, 0}, sum[2];
    if (i < B) {
      const int b = B <= kRankSeqs ? order[i] : i;
      count_parts(p, load_seq(p, b), cap, v);
      p.order[i] = b;
    }
    plan_scan(v, sum, part);
    if (i < B) {
      p.first[i] = static_cast<int>(carry[0] + v[0]);
      p.part0[i] = static_cast<int>(carry[1] + v[1]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) carry[j] += sum[j];
  }
  if (tid == 0) {
    const bool few = carry[0] < kMostItems;
    p.first[B] = static_cast<int>(carry[0]);
    p.head->items = few ? static_cast<int>(carry[0]) : 0;
    p.head->states = few ? static_cast<int>(carry[1]) : 0;
    p.head->next = p.head->failed = 0;
    p.head->cap = cap;
  }
}

// The sequence whose range of `first` holds i; the whole warp searches.
__device__ __forceinline__ int find_seq(const int* first, int B, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, count = B;
  while (count > 1) {
    const int step = (count + 31) / 32;
    const int at = lo + lane * step;
    const bool below = lane * step < count && __ldcg(first + at) <= i;
    const int k = __popc(__ballot_sync(0xffffffffu, below)) - 1;
    lo += k * step;
    count = min(step, count - k * step);
  }
  return lo;
}

// ------------------------------------------------------------------ roles
struct Ctx {
  uint32_t sb;
  uint8_t* smem;
  uint32_t tmem, rank;  // of the CTA in its pair
  uint64_t wait_ns;
  volatile uint32_t* abort;
  __device__ uint32_t bar(int i) const { return sb + kOffBars + 8 * i; }
  __device__ volatile uint32_t* mended() const { return reinterpret_cast<volatile uint32_t*>(smem + kOffMended); }
};
// Arrivals on a barrier of the pair's first CTA (or the only one).  Release at CTA scope:
// what they hand over is tensor memory or shared memory of the arriving CTA, already
// ordered for the tensor core (tcgen05.wait, fence.proxy.async).
template <bool kPair>
__device__ __forceinline__ uint32_t lead(uint32_t bar) {
  return kPair ? mapa_shared(bar, 0) : bar;
}
template <bool kPair>
__device__ __forceinline__ void arrive(uint32_t bar) {
  if constexpr (kPair) asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
  else mbar_arrive(bar);
}
template <bool kPair>
__device__ __forceinline__ void arrive_tx(uint32_t bar, uint32_t bytes) {
  if constexpr (kPair)
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cluster.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
  else mbar_arrive_expect_tx(bar, bytes);
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
// Loads whose bytes count on a barrier of either CTA of the pair.
template <bool kPair>
__device__ __forceinline__ void load_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
  if constexpr (kPair)
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
  else tma_3d(dst, map, x, y, z, bar);
}
template <bool kPair>
__device__ __forceinline__ void load_4d(uint32_t dst, const void* map, int x, int y, int z, int w, uint32_t bar) {
  if constexpr (kPair)
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar) : "memory");
  else tma_4d(dst, map, x, y, z, w, bar);
}
template <bool kPair>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (kPair)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
  else umma_ss(d, a, b, idesc, acc);
}
template <bool kPair>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (kPair)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
  else umma_ts(d, a, b, idesc, acc);
}
// Arrive on the barrier at this offset, of both CTAs, when the MMAs issued so far are complete.
template <bool kPair>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (kPair)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
  else umma_commit(bar);
}

struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// A reader's walk over the items that the plan warp posts.
template <bool kPair>
struct Items {
  uint32_t count = 0;
  __device__ __forceinline__ bool next(const Ctx& c, Item& it) {
    const int s = count % kItemSlots;
    if (!__all_sync(0xffffffffu, mbar_wait<kPair>(c.bar(kItemFull + s), (count / kItemSlots) & 1, c.abort, c.wait_ns))) return false;
    const int4* src = reinterpret_cast<const int4*>(c.smem + kOffItems) + 4 * s;
    it.unpack(src[0], src[1], src[2], src[3]);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      if constexpr (kPair) arrive_cluster(lead<true>(c.bar(kItemEmpty + s)));
      else mbar_arrive(c.bar(kItemEmpty + s));
    }
    ++count;
    return uniform(it.live) != 0;
  }
};

__device__ __forceinline__ int page_of(const Params& p, int b, int t) {
  const int id = __ldg(p.x.block_table + static_cast<int64_t>(b) * p.x.W + t);
  return id >= 0 && id < p.x.num_blocks ? id : -1;
}

template <bool kPair>
__device__ void plan_role(const Params& p, const Ctx& c, const WarpPlan& w) {
  const int lane = threadIdx.x & 31, B = p.x.B;
  uint32_t count = 0;
  constexpr int kCtas = Shape<kPair>::kCtas;
  int i = blockIdx.x / kCtas, drawn = 0;
  // a lane keeps a sequence, where there are no more than 32: no item waits for its description then
  const bool kept = B <= kWarpSeqs;
  int total, states, cap, first, part0, seq;
  Seq mine;
  auto load = [&](int at) {
    seq = __ldcg(p.order + at);
    first = __ldcg(p.first + at);
    part0 = __ldcg(p.part0 + at);
    mine = load_seq(p, seq);
  };
  if (kept) {
    total = w.items;
    states = w.states;
    cap = w.cap;
    first = w.first;
    part0 = w.part0;
    seq = w.seq;
    mine = w.s;
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
    total = __ldcg(&p.head->items);
    states = __ldcg(&p.head->states);
    cap = __ldcg(&p.head->cap);
  }
  while (true) {
    Item it = {};
    it.live = i < total ? 1 : 0;
    if (it.live) {
      int from = 0;  // the lane that has the sequence
      if (kept) from = __popc(__ballot_sync(0xffffffffu, first <= i)) - 1;
      else load(find_seq(p.first, B, i));
      auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, from); };
      Seq s;
      s.n = of(mine.n);
      s.len = of(mine.len);
      s.pos = of(mine.pos);
      s.q0 = of(mine.q0);
      s.key0 = of(mine.key0);
      s.pairs = of(mine.pairs);
      s.bad_len = s.bad_table = false;
      const int b = of(seq), Hkv = p.x.n_kv;
      int k = i - of(first), m, hk, cut = 0, cuts = 1;
      bool whole = states == 0;
      if (!whole) {
        const Cuts how = cuts_of(p, s, cap);
        whole = how.at_least(2) == 0;
        if (!whole) {
          how.find(k / Hkv, m, cut, cuts);
          hk = k % Hkv;
        }
      }
      if (whole) {
        // heads whose keys and values fill about a third of L2 go side by side
        const int64_t bytes = static_cast<int64_t>(max(1, s.len)) * (p.x.d_qk + p.x.d_v) * 2;
        int g = 0, heads = Hkv, r = k;
        if (bytes * Hkv > (40 << 20)) {
          const int group = bytes > (40 << 20) ? 1 : min(Hkv, (40 << 20) / static_cast<int>(bytes));
          const int per_group = s.pairs * group;  // no more than there are items
          g = k / per_group;
          r = k - g * per_group;
          g *= group;
          heads = min(group, Hkv - g);
        }
        const int row = r / heads;
        m = s.pairs - 1 - row;
        hk = g + r - row * heads;
      }
      it.b = b;
      it.hk = hk;
      it.m = m;
      it.n = s.n;
      it.len = s.len;
      it.pos = s.pos;
      it.q0 = s.q0;
      it.key0 = s.key0;
      const int tok = m * p.span, half = p.span / 2;
      int tiles[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) tiles[h] = tok + h * half < s.n ? tiles_of(seen_by(p, s, tok + (h + 1) * half)) : 0;
      const int most = max(tiles[0], tiles[1]);
      const int each = most / cuts, more = most - each * cuts;  // the first `more` parts have a tile more
      it.t0 = cut * each + min(cut, more);
      const int end = it.t0 + each + (cut < more ? 1 : 0);
      it.ta = max(it.t0, min(tiles[0], end));
      it.tb = max(it.t0, min(tiles[1], end));
      it.lo = seen_by(p, s, tok + 1);
      it.part = cuts > 1 ? of(part0) + k : -1;
      if (it.part >= 0 && lane == 0) p.records[it.part] = {s.q0 + tok, (p.x.S1 > 0 ? p.x.S1 : s.n) - tok, hk, cut, cuts, {}};
    }
    const int s = count % kItemSlots;
    if (!__all_sync(0xffffffffu, mbar_wait<kPair>(c.bar(kItemEmpty + s), ((count / kItemSlots) & 1) ^ 1, c.abort, c.wait_ns))) return;
    if (lane == 0) {
      int4* to = reinterpret_cast<int4*>(c.smem + kOffItems) + 4 * s;
#pragma unroll
      for (int k = 0; k < 4; ++k) to[k] = it.word(k);
      mbar_arrive(c.bar(kItemFull + s));
      if constexpr (kPair) {
        const uint32_t at = mapa_shared(c.sb + kOffItems + s * kItemBytes, 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int4 w = it.word(k);
          asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(at + 16 * k), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
        }
        arrive_cluster(mapa_shared(c.bar(kItemFull + s), 1));
      }
    }
    __syncwarp();
    if (!it.live) return;
    // CTAs draw as late as will do, so that the one with least left to do is the next to draw:
    // 9 prompts of 3 to 1680 tokens 62 us when they drew two items ahead, now 52
    if (!warp_wait(c, kDraw, count & 1)) return;
    if (count++ == 0) asm volatile("griddepcontrol.wait;" ::: "memory");  // the counter begins at 0
    if (lane == 0) drawn = static_cast<int>(gridDim.x) / kCtas + atomicAdd(&p.head->next, 1);
    i = uniform(drawn);
  }
}

template <bool kPair>
__device__ void load_role(const Params& p, const Ctx& c, const Maps& maps) {
  constexpr int kSlotBytes = Shape<kPair>::kSlotBytes;
  const int lane = threadIdx.x & 31, rank = static_cast<int>(c.rank);
  const uint32_t ring = c.sb + 2 * p.kc * kChunk;
  const int value_slots = kPair ? 2 : p.vc;  // of a tile
  const bool paged = p.x.num_blocks > 0;
  Items<kPair> items;
  Item it;
  Ring r;
  uint32_t used[2] = {0, 0};  // times that a row tile's Q was loaded
  while (items.next(c, it)) {
    const int end = max(it.ta, it.tb);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (it.t1(h) <= it.t0) continue;
      if (!warp_wait(c, kQFree + h, (used[h] & 1) ^ 1)) return;
      ++used[h];
      if (lane == 0) {
        const uint32_t bar = lead<kPair>(c.bar(kQFull + h));
        const int tile = kPair ? 2 * h + rank : h;
        arrive_tx<kPair>(bar, p.kc * 128 * p.G * p.tpt);
        for (int k = 0; k < p.kc; ++k)
          load_3d<kPair>(c.sb + (h * p.kc + k) * kChunk, &maps.q, 64 * k, it.hk * p.G, it.q0 + it.m * p.span + tile * p.tpt, bar);
      }
      __syncwarp();
    }
    const bool tells = rank == 0 && lane == 0;
    if (tells && it.t0 >= end) mbar_arrive(c.bar(kDraw));
    int page = paged && it.t0 < end ? page_of(p, it.b, it.t0) : 0;
    for (int t = it.t0; t < end; ++t) {
      if (tells && t == max(it.t0, end - kDrawTiles)) mbar_arrive(c.bar(kDraw));
      const int ahead = paged && t + 1 < end ? page_of(p, it.b, t + 1) : 0;
      const int row = paged ? 0 : it.key0 + kTile * t;
      const int block = paged ? (page < 0 ? p.x.num_blocks : page) : 0;  // beyond the pool: zeros
      for (int k = 0; k < p.kc; ++k) {
        if (!warp_wait(c, kEmpty + r.slot, r.phase ^ 1)) return;
        if (lane == 0) {
          // of a pair, each CTA has half of the keys
          const uint32_t bar = lead<kPair>(c.bar(kFull + r.slot));
          arrive_tx<kPair>(bar, kSlotBytes);
          load_4d<kPair>(ring + r.slot * kSlotBytes, &maps.k, 64 * k, row + 64 * rank, it.hk, block, bar);
        }
        __syncwarp();
        r.step(p.slots);
      }
      const int bars = kTile * (t + 1) > it.lo ? kLocal : kFull;
      for (int k = 0; k < value_slots; ++k) {
        if (!warp_wait(c, kEmpty + r.slot, r.phase ^ 1)) return;
        if (lane == 0) {
          const uint32_t dst = ring + r.slot * kSlotBytes;
          if (kPair && bars == kFull) {  // and half of the values' columns
            const uint32_t bar = lead<kPair>(c.bar(kFull + r.slot));
            arrive_tx<kPair>(bar, kSlotBytes);
            load_4d<kPair>(dst, &maps.v, 64 * rank, row + 64 * k, it.hk, block, bar);
          } else {
            const uint32_t bar = c.bar(bars + r.slot);
            mbar_arrive_expect_tx(bar, kSlotBytes);
            tma_4d(dst, &maps.v, 64 * rank, row + 64 * k, it.hk, block, bar);
            if (!kPair && p.vc == 2) tma_4d(dst + kSlotBytes / 2, &maps.v, 64, row + 64 * k, it.hk, block, bar);
          }
        }
        __syncwarp();
        r.step(p.slots);
      }
      page = ahead;
    }
  }
}

// Tells the softmax warps, of both CTAs of a pair, before the barrier that hands the values on.
template <bool kPair>
__device__ __noinline__ void post_mended(const Ctx& c) {
  if constexpr (kPair) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      asm volatile("st.shared::cluster.u32 [%0], 1;" :: "r"(mapa_shared(c.sb + kOffMended, r)) : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");  // returns when the other CTA's shared memory has the word
  } else {
    *c.mended() = 1u;
  }
}

template <typename E, bool kPair>
__device__ void mend_role(const Params& p, const Ctx& c) {
  constexpr int kSlotBytes = Shape<kPair>::kSlotBytes;
  const int lane = threadIdx.x & 31;
  const uint32_t ring = c.sb + 2 * p.kc * kChunk;
  const int value_slots = kPair ? 2 : p.vc;
  Items<kPair> items;
  Item it;
  Ring r;
  uint32_t seen = 0;  // a bit per slot: parity of its local barrier
  const int rows = kPair || p.vc == 2 ? 64 : 128, units = !kPair && p.vc == 2 ? 16 : 8;  // keys of a slot, 16-byte units of a key
  const int unit = lane & (units - 1);
  while (items.next(c, it)) {
    const int end = max(it.ta, it.tb);
    for (int t = it.t0; t < end; ++t) {
      for (int k = 0; k < p.kc; ++k) r.step(p.slots);
      for (int k = 0; k < value_slots; ++k, r.step(p.slots)) {
        if (kTile * (t + 1) <= it.lo) continue;
        if (!warp_wait(c, kLocal + r.slot, (seen >> r.slot) & 1)) return;
        seen ^= 1u << r.slot;
        const int base = kTile * t + 64 * k;
        const int first = max(0, min(it.lo - base, rows)), live = max(0, min(it.len - base, rows));
        const uint32_t slot = ring + r.slot * kSlotBytes + (unit >> 3) * (kSlotBytes / 2);
        auto at = [&](int row) { return slot + row * 128 + (((unit & 7) ^ (row & 7)) << 4); };
        auto load = [&](int row) {
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at(row)));
          return v;
        };
        auto store = [&](int row, uint4 v) {
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at(row)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
        };
        bool good = true;
        const int step = 32 / units;
        for (int row = first + lane / units; row < live; row += 4 * step) {
          uint4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = row + u * step < live ? load(row + u * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int u = 0; u < 4; ++u) good = good && finite4<E>(v[u]);
        }
        bool wrote = live < rows;
        for (int row = max(first, live) + lane / units; row < rows; row += step) store(row, make_uint4(0, 0, 0, 0));
        if (__any_sync(0xffffffffu, !good)) {
          wrote = true;
          post_mended<kPair>(c);
          for (int row = first + lane / units; row < live; row += step) {
            const uint4 v = load(row);
            store(row, make_uint4(finite2<E>(v.x), finite2<E>(v.y), finite2<E>(v.z), finite2<E>(v.w)));
          }
        }
        if (wrote) fence_proxy_async_smem();  // generic-proxy stores -> tensor-core reads
        __syncwarp();
        if (lane == 0) arrive<kPair>(lead<kPair>(c.bar(kFull + r.slot)));
      }
    }
  }
}

// The warp stays converged around an elected issuer, and what steers it is made
// uniform, so that descriptors live in uniform registers: an MMA takes 64 clocks,
// and with loops over runtime counts its issue took 115.
template <bool kPair, int kKc, int kVc>
__device__ void mma_role(const Params& p, const Ctx& c) {
  constexpr int kSlotBytes = Shape<kPair>::kSlotBytes, kSlots = Shape<kPair>::slots(kKc);
  constexpr int kVSteps = kVc == 2 ? 4 : 8;
  constexpr uint32_t kSlot = kSlotBytes >> 4, kQ = kChunk >> 4;  // in a descriptor's address field
  const uint64_t desc_q = make_sdesc(c.sb, 16, 1024, kSwizzle128B);
  const uint64_t desc_k = make_sdesc(c.sb + 2 * kKc * kChunk, 16, 1024, kSwizzle128B);
  const uint64_t desc_v = make_sdesc(c.sb + 2 * kKc * kChunk, kChunk / 2, 1024, kSwizzle128B);
  const uint32_t idesc_s = uniform(static_cast<int>(p.idesc_s)), idesc_v = uniform(static_cast<int>(p.idesc_v));
  const int last_steps = uniform(p.ks_qk) - 4 * (kKc - 1);  // of the last chunk of a key
  Items<kPair> items;
  Item it;
  int slot = 0;  // the next that no MMA has used
  uint32_t phase = 0;
  uint32_t q_uses[2] = {0, 0}, p_uses[2] = {0, 0}, s_uses[2] = {0, 0};
  auto after = [&](int s, int n) { return s + n >= kSlots ? s + n - kSlots : s + n; };
  auto take = [&](int n) {  // waits for the next n slots
#pragma unroll
    for (int k = 0; k < n; ++k) {
      if (!warp_wait(c, kFull + slot, phase)) return false;
      phase ^= slot + 1 == kSlots ? 1u : 0u;
      slot = after(slot, 1);
    }
    return true;
  };
  // S_h = Q_h K^T of the keys in `at` and the slots behind it
  auto scores = [&](int h, int at, bool free_keys, bool last) {
    if (elect_one()) {
      const uint32_t d = c.tmem + kTmemS + 128 * h;
#pragma unroll
      for (int k = 0; k < kKc; ++k) {
        const uint64_t a = desc_q + (h * kKc + k) * kQ;
        const uint64_t b = desc_k + static_cast<uint32_t>(after(at, k)) * kSlot;
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (k + 1 < kKc || s < last_steps) mma_ss<kPair>(d, a + 2 * s, b + 2 * s, idesc_s, (k | s) != 0 ? 1u : 0u);
      }
      commit<kPair>(c.bar(kSFull + h));
      if (free_keys) {
#pragma unroll
        for (int k = 0; k < kKc; ++k) commit<kPair>(c.bar(kEmpty) + 8 * after(at, k));
      }
      if (last) commit<kPair>(c.bar(kQFree + h));
    }
    __syncwarp();
  };
  // O_h += P_h V
  constexpr bool kApart = kVc == 1;
  using Cols = Tmem<kApart>;
  auto values = [&](int h, int at, bool first, bool free_values, bool last) {
    if (elect_one()) {
      const uint32_t d = c.tmem + Cols::kO + Cols::kOStep * h, a = c.tmem + Cols::kP + Cols::kPStep * h;
#pragma unroll
      for (int k = 0; k < kVc; ++k) {
        const uint64_t b = desc_v + static_cast<uint32_t>(after(at, k)) * kSlot;
#pragma unroll
        for (int s = 0; s < kVSteps; ++s)
          mma_ts<kPair>(d, a + 8 * (k * kVSteps + s), b + 128 * s, idesc_v, (k | s) == 0 && first ? 0u : 1u);
      }
      if (free_values) {
#pragma unroll
        for (int k = 0; k < kVc; ++k) commit<kPair>(c.bar(kEmpty) + 8 * after(at, k));
      }
      if (kApart) commit<kPair>(c.bar(kPFree + h));
      if (last) commit<kPair>(c.bar(kOFull + h));
    }
    __syncwarp();
  };
  bool ok = !kPair || uniform(static_cast<int>(c.rank)) == 0;  // the first CTA issues for both
  const bool issuer = ok;
  while (ok && items.next(c, it)) {
    const int t0 = uniform(it.t0), ta = uniform(it.ta), tb = uniform(it.tb), end = max(ta, tb);
    if (t0 >= end) continue;
    int key = slot;
    ok = take(kKc);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t1 = h == 0 ? ta : tb;
      if (!ok || t0 >= t1) continue;
      ok = warp_wait(c, kQFull + h, q_uses[h]++ & 1);
      if (ok) scores(h, key, h == (t0 < tb ? 1 : 0), t0 + 1 == t1);
    }
    for (int t = t0; t < end && ok; ++t) {
      const int value = slot;
      ok = take(kVc);
      key = slot;
      if (ok && t + 1 < end) ok = take(kKc);
      if constexpr (kApart) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t1 = h == 0 ? ta : tb;
          if (!ok || t + 1 >= t1) continue;
          ok = warp_wait(c, kSFree + h, s_uses[h]++ & 1);
          if (!ok) continue;
          tc_fence_after();
          scores(h, key, h == (t + 1 < tb ? 1 : 0), t + 2 == t1);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t1 = h == 0 ? ta : tb;
        if (!ok || t >= t1) continue;
        ok = warp_wait(c, kPReady + h, p_uses[h]++ & 1);
        if (!ok) continue;
        tc_fence_after();
        // the last row tile that reads a key or value tile gives its slots up
        values(h, value, t == t0, h == (t < tb ? 1 : 0), t + 1 == t1);
        if (!kApart && t + 1 < t1) scores(h, key, h == (t + 1 < tb ? 1 : 0), t + 2 == t1);
      }
    }
  }
  // every MMA in flight lands before the CTA leaves
  if (issuer && elect_one()) commit<kPair>(c.bar(kFinal));
  __syncwarp();
  volatile uint32_t never = 0;
  mbar_wait<false>(c.bar(kFinal), 0, &never, c.wait_ns > 500000000ull ? c.wait_ns : 500000000ull);
  __syncwarp();
}

template <bool kPair, bool kApart>
__device__ __forceinline__ void mma_role(const Params& p, const Ctx& c) {
  constexpr int kVc = kApart ? 1 : 2;
  if (p.kc == 1) return mma_role<kPair, 1, kVc>(p, c);
  if (p.kc == 2) return mma_role<kPair, 2, kVc>(p, c);
  return mma_role<kPair, 3, kVc>(p, c);
}

// The NaN of values that are not finite, which mending took from a row: keys [lo,
// hi) of the sequence, put into what the calling thread has stored, its row of out
// or of a partial state.  Rare: such values lay where not every row sees them.
template <typename E>
__device__ __noinline__ void infinite_columns(const Params& p, int b, int hk, int key0, int lo, int hi, E* out, float* part) {
  constexpr uint32_t kExp = __is_same(E, __half) ? 0x7C00u : 0x7F80u;
  for (int key = lo; key < hi; ++key) {
    int64_t at = hk * p.x.v.head_stride;
    if (p.x.num_blocks > 0) {
      const int page = page_of(p, b, key / kPage);
      if (page < 0) continue;
      at += page * p.x.v.block_stride + (key % kPage) * p.x.v.row_stride;
    } else {
      at += static_cast<int64_t>(key0 + key) * p.x.v.row_stride;
    }
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x.v.data) + at);
    for (int u = 0; u < p.x.d_v / 8; ++u) {
      const uint4 x = __ldg(v + u);
      if (finite4<E>(x)) continue;
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      for (int k = 0; k < 8; ++k) {
        if (((w[k >> 1] >> (k & 1) * 16) & kExp) != kExp) continue;
        const int d = 8 * u + k;
        if (out != nullptr) reinterpret_cast<uint16_t*>(out)[d] = 0x7FFF;
        else part[(d >> 2) * 512 + (d & 3)] = __uint_as_float(0x7FC00000u);
      }
    }
  }
}

// Among each two lanes: units 2i and 2i + 1 (four words each) of the two rows, so
// that the even lane has both rows' units 2i and the odd one their units 2i + 1.
__device__ __forceinline__ void turn_units(uint32_t (&y)[32], int lane) {
  const bool odd = (lane & 1) != 0;
#pragma unroll
  for (int u = 0; u < 8; u += 2) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t &lo = y[4 * u + w], &hi = y[4 * u + 4 + w];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
      if (odd) lo = got;
      else hi = got;
    }
  }
}

template <typename E, bool kPair, bool kApart>
__device__ void softmax_role(const Params& p, const Ctx& c, int warp, int lane) {
  const int h = warp >> 2, row = (warp & 3) * 32 + lane;  // row tile, row of it
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  using Cols = Tmem<kApart>;
  const uint32_t tS = c.tmem + lanes + kTmemS + 128 * h, tO = c.tmem + lanes + Cols::kO + Cols::kOStep * h;
  const uint32_t tP = c.tmem + lanes + Cols::kP + Cols::kPStep * h;
  // a positive scale leaves the order of scores alone: the maximum is taken of
  // the raw ones, and the scale goes into the exponent's multiply-add
  const float scale = p.x.scale_log2;
  const bool raw = scale > 0.f;
  const float mul = raw ? scale : 1.f;
  const int tok_in = row / p.G, head_in = row - tok_in * p.G;
  const bool paged = p.x.num_blocks > 0;
  uint32_t uses = 0, outs = 0, products = 0;
  bool bad = false;
  Items<kPair> items;
  Item it;
  while (items.next(c, it)) {
    const int tile = kPair ? 2 * h + static_cast<int>(c.rank) : h;  // of the item
    const int tok = it.m * p.span + tile * p.tpt + tok_in;
    const bool live = tok_in < p.tpt && tok < it.n;
    const bool padded = tok_in < p.tpt && p.x.S1 > 0 && tok < p.x.S1;  // written, live or not
    const int vis = p.x.causal ? min(it.len, max(0, it.pos + tok + 1)) : it.len;  // keys that this row sees
    float m = -INFINITY, l = 0.f;
    for (int t = it.t0; t < it.t1(h); ++t) {
      const bool page = !paged || page_of(p, it.b, t) >= 0;
      bad = bad || !page;
      const int here = page ? vis - kTile * t : 0;
      if (!warp_wait(c, kSFull + h, uses++ & 1)) return;
      tc_fence_after();
      auto load = [&](float (&z)[128]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld_32x32b_x32(tS + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(z + 32 * k));
        tmem_wait_ld();
      };
      auto mask = [&](float (&z)[128]) {
        if (!raw) {
#pragma unroll
          for (int k = 0; k < 128; ++k) z[k] *= scale;
        }
        if (__any_sync(0xffffffffu, here < kTile)) {
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k >= here) z[k] = -INFINITY;
        }
      };
      auto maximum = [&](const float (&z)[128]) {
        float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
        for (int k = 4; k < 128; k += 8) {
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = fmaxf(fmaxf(mx[j], z[k + j]), k + 4 + j < 128 ? z[k + 4 + j] : -INFINITY);
        }
        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
      };
      auto rescale = [&](float f) {  // O
#pragma unroll 1
        for (int k = 0; k < p.x.d_v; k += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO + k, o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tmem_st_32x32b_x32(tO + k, o);
        }
      };
      uint32_t w[64];
      // one pair's weights, and their part of the sum; 16 bits: half a step, as one rounding of the output costs
      auto weigh = [&](const float (&z)[128], int k, uint64_t mul_2, uint64_t mm_2, uint64_t& sum) {
        float2 e = unpair(fma2(pair(z[2 * k], z[2 * k + 1]), mul_2, mm_2));
        e.x = fast_exp2(e.x);
        e.y = fast_exp2(e.y);
        sum = add2(sum, pair(e.x, e.y));
        w[k] = pack16<E>(e.x, e.y);
      };
      const uint64_t mul_2 = pair(mul, mul);
      uint64_t sum[2];
      // The maximum moves only when a tile exceeds it by more than 2^8: weights stay below
      // 2^8 (lifted, 2^15) and O is rarely rescaled.
      if constexpr (kPair) {
        // So weights are made of the maximum so far while the tile's is found beside them, and in the
        // rare case again from the scores, which stay in tensor memory until then: 8192 tokens, 32 heads
        // on 8 of 128 372 -> 342 us.  A CTA alone is bound by shared memory or, with small heads, by the
        // softmax warps together, whose phases then mix worse: prompts of 4096, heads of 64, 329 -> 359.
        bool first = t == it.t0, again;
        do {
          float z[128];
          load(z);
          mask(z);
          if (first) m = maximum(z) - kLift<E>;
          first = false;
          const float mm = m == -INFINITY ? 0.f : m;
          const uint64_t mm_2 = pair(-mm, -mm);
          sum[0] = sum[1] = 0;
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 64; ++k) {
            mx[k & 3] = fmaxf(fmaxf(mx[k & 3], z[2 * k]), z[2 * k + 1]);
            weigh(z, k, mul_2, mm_2, sum[k & 1]);
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mul;
          const bool grow = top > m + (8.f + kLift<E>);
          again = __any_sync(0xffffffffu, grow);
          if (again) {  // the MMAs before these scores are complete, the one before on O among them
            const float to = top - kLift<E>, f = grow ? fast_exp2(m - to) : 1.f;
            l *= f;
            if (grow) m = to;
            if (t > it.t0) rescale(f);
          }
        } while (again);
        tmem_st_32x32b_x32(tP, *reinterpret_cast<uint32_t(*)[32]>(w));
      } else {
        float z[128];
        load(z);
        if (kApart && t + 1 < it.t1(h)) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(c.bar(kSFree + h));
        }
        mask(z);
        const float top = maximum(z);
        const bool grow = top > m + (8.f + kLift<E>);
        const float to = top - kLift<E>, f = grow ? fast_exp2(m - to) : 1.f;
        if (grow) {
          l *= f;
          m = to;
        }
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t mm_2 = pair(-mm, -mm);
        sum[0] = sum[1] = 0;
#pragma unroll
        for (int k = 0; k < 64; ++k) {
          weigh(z, k, mul_2, mm_2, sum[k & 1]);
          if (k == 31) {
            if (kApart && t > it.t0) {  // the product before this one is through with the weights, and with O
              if (!warp_wait(c, kPFree + h, products++ & 1)) return;
              tc_fence_after();
            }
            tmem_st_32x32b_x32(tP, *reinterpret_cast<uint32_t(*)[32]>(w));
          }
        }
        // the MMAs before these scores are complete, the one before on O among them (apart: see above)
        if (t > it.t0 && __any_sync(0xffffffffu, grow)) rescale(f);
      }
      const float2 sums = unpair(add2(sum[0], sum[1]));
      l += sums.x + sums.y;
      tmem_st_32x32b_x32(tP + 32, *reinterpret_cast<uint32_t(*)[32]>(w + 32));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive<kPair>(lead<kPair>(c.bar(kPReady + h)));
    }
    const bool any = it.t1(h) > it.t0;
    if (any) {
      if (!warp_wait(c, kOFull + h, outs++ & 1)) return;
      tc_fence_after();
      ++products;  // the last one's, whose barrier nobody waits for
    }
    if (!any || !live) {
      l = 0.f;
      m = -INFINITY;
    }
    const bool nothing = l == 0.f;
    if (it.part < 0) {
      const float inv = nothing ? 0.f : 1.f / l;
      const int64_t at = static_cast<int64_t>(it.q0 + tok) * p.x.n_q + it.hk * p.G + head_in;
      E* out = static_cast<E*>(p.x.out) + at * p.x.d_v;
      const bool put = live || padded;
      const int at_row = put ? static_cast<int>(at) : -1;  // T * n_q is below 2^31
#pragma unroll 1
      for (int k = 0; k < p.x.d_v; k += 64) {
        uint32_t y[32];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[32];
          if (any) {
            tmem_ld_32x32b_x32(tO + k + 32 * half, v);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            y[16 * half + j] = nothing ? 0u : pack16<E>(__uint_as_float(v[2 * j]) * inv, __uint_as_float(v[2 * j + 1]) * inv);
        }
        // Two lanes swap 16-byte units of their rows, so that a store writes whole 32-byte sectors:
        // rows written by their own threads, halves of sectors, took 6000 clocks an item, these
        // 4300 and whole 128-byte lines (eight lanes, three times the shuffles) no less.  The rest
        // is the way to memory: all SMs end items at about the same time.
        turn_units(y, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int to = __shfl_sync(0xffffffffu, at_row, (lane & 30) + (j & 1)), col = k + 8 * ((lane & 1) + (j & 6));
          if (to >= 0 && col < p.x.d_v)
            *reinterpret_cast<uint4*>(static_cast<E*>(p.x.out) + static_cast<int64_t>(to) * p.x.d_v + col) =
                make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        }
      }
      __syncwarp();  // infinite columns go over what other lanes have written
      if (*c.mended() && live && !nothing) infinite_columns<E>(p, it.b, it.hk, it.key0, it.lo, vis, out, nullptr);
      if (put && p.x.lse != nullptr) p.x.lse[at] = nothing ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
    } else {
      float* dst = p.parts + static_cast<int64_t>(it.part) * p.part_floats + tile * (p.part_floats / Shape<kPair>::kTiles);
      if (any) {
#pragma unroll 1
        for (int k = 0; k < p.x.d_v; k += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tO + k, v);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (k + 4 * u < p.x.d_v)
              reinterpret_cast<uint4*>(dst)[((k >> 2) + u) * 128 + row] = make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
        }
        if (*c.mended() && live)
          infinite_columns<E>(p, it.b, it.hk, it.key0, max(it.lo, kTile * it.t0), min(vis, kTile * it.t1(h)), nullptr, dst + row * 4);
      }
      // -inf says that the part is not the row's; the lowest maximum joins with weight 0 and
      // brings along the NaN of infinite values whose scores are all -inf
      dst[128 * p.x.d_v + row] = any && live ? fmaxf(m, -3.402823466e38f) : -INFINITY;
      dst[128 * p.x.d_v + 128 + row] = l;
    }
    tc_fence_before();  // the reads of O come before the next item's MMAs (through kPReady)
  }
  if (bad) atomicOr(&g_prompt_status, MLA_DEVICE_BAD_BLOCK);
}

template <typename E, bool kPair, bool kApart>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ uint8_t raw[];
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  Ctx c;
  c.sb = (smem_u32(raw) + 1023u) & ~1023u;  // swizzled operands need 1024-byte alignment
  c.smem = raw + (c.sb - smem_u32(raw));
  c.rank = kPair ? cluster_ctarank() : 0;
  c.wait_ns = p.wait_ns;
  c.abort = reinterpret_cast<volatile uint32_t*>(c.smem + kOffAbort);
  constexpr int kCtas = Shape<kPair>::kCtas;
  if (tid < kNumBars) {  // arrivals of each phase
    const int i = tid;
    const int count = i < kEmpty ? kCtas                                     // kFull
                      : i >= kQFull && i < kQFree ? kCtas
                      : i >= kPReady && i < kOFull ? 4 * kCtas
                      : i >= kSFree && i < kPFree ? 4
                      : i >= kItemEmpty && i < kDraw ? (kPair ? 2 * kItemReaders - 1 : kItemReaders)  // a pair has one MMA warp
                                                     : 1;
    mbar_init(c.bar(i), count);
    if (tid == 0) *c.abort = *c.mended() = 0u;
    fence_mbarrier_init_cluster();
  }
  if (warp == kLoadWarp && lane < 3) {
    const CUtensorMap* map = lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v;
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  if (warp == kMmaWarp) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(c.sb + kOffTmem) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(c.sb + kOffTmem, 512);
      tmem_relinquish();
    }
  }
  // while tensor memory is allocated; nothing begins before the first item
  WarpPlan plan = {};
  if (warp == kPlanWarp && c.rank == 0 && p.x.B <= kWarpSeqs) plan = plan_warp(p);
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) {  // the other CTA's barriers are in place
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  c.tmem = uniform(static_cast<int>(*reinterpret_cast<volatile uint32_t*>(c.smem + kOffTmem)));
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp < kSoftmaxWarps) {
    regs_increase<kSoftmaxRegs>();
    softmax_role<E, kPair, kApart>(p, c, warp, lane);
  } else {
    regs_decrease<kOtherRegs>();
    if (warp == kMmaWarp) {
      mma_role<kPair, kApart>(p, c);
    } else if (warp == kLoadWarp) {
      load_role<kPair>(p, c, maps);
    } else if (warp == kPlanWarp) {
      if (c.rank == 0) plan_role<kPair>(p, c, plan);
    } else if (warp == kMendWarp) {
      mend_role<E, kPair>(p, c);
    }
  }

  // the launch behind this one reads what the plan has written: it must not end before the plan
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (*c.abort) {
    // a wait ran out: loads may still be in flight to shared memory; they take microseconds
    if (tid == 0) {
      atomicOr(&g_prompt_status, MLA_DEVICE_TIMEOUT);
      // for the join alone: what the plan wrote may still be read by CTAs that come later
      p.head->failed = 1;
    }
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000) {
    }
  }
  if constexpr (kPair) {  // nothing of this CTA is needed by the other any more
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  if (warp == kMmaWarp) {
    if constexpr (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(c.tmem) : "memory");
    else tmem_dealloc(c.tmem, 512);
  }
}

// ------------------------------------------------------------------ merge
// Joins the parts of the items that were cut: a block takes the 128 rows of a row
// tile and a quarter of the columns, a thread one row and four columns at a time.  The
// parts of an item share its row tiles, and what they are a part of stands in records,
// so that nothing is searched for.
constexpr int kMergeThreads = 256, kMergeSlices = 4, kAhead = 2;  // parts in flight
constexpr int kMergeQuads = kMaxDv / 4 / kMergeSlices / 2;          // four columns each, of a thread
template <typename E>
__global__ void __launch_bounds__(kMergeThreads) prompt_merge_kernel(const __grid_constant__ Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 head = __ldcg(reinterpret_cast<const int4*>(p.head));  // items, next, states, failed
  const int states = head.w != 0 ? 0 : head.z;
  const int row = threadIdx.x & 127, side = threadIdx.x >> 7, quads = p.x.d_v / 4;
  const int per_slice = (quads + kMergeSlices - 1) / kMergeSlices;  // at most 2 * kMergeQuads
  const int64_t step = static_cast<int64_t>(p.part_floats) * p.x.n_kv;      // an item's parts: heads lie between them
  for (int unit = blockIdx.x; unit < states * kMergeSlices; unit += gridDim.x) {
    // quarter u % 4 of the row tiles that fall to this part, one after the other among the item's parts
    const int index = unit / kMergeSlices, slice = unit % kMergeSlices;
    const int4 rec = __ldcg(reinterpret_cast<const int4*>(p.records + index));  // row0, tokens, hk, cut
    const int cuts = __ldcg(&p.records[index].cuts), cut = rec.w;
    for (int tile = cut; tile < p.tiles; tile += cuts) {
      const int tok_in = row / p.G, tok = tile * p.tpt + tok_in;
      const bool put = tok_in < p.tpt && tok < rec.y;
      const float* src = p.parts + index * static_cast<int64_t>(p.part_floats) - cut * step + tile * (p.part_floats / p.tiles);
      const int quad0 = slice * per_slice + side, quad1 = min(quads, (slice + 1) * per_slice);
      float top = -INFINITY, l = 0.f, o[kMergeQuads][4] = {};
      for (int c0 = 0; c0 < cuts; c0 += kAhead) {
        float mk[kAhead], lk[kAhead];
        float4 x[kAhead][kMergeQuads];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float* part = src + min(c0 + u, cuts - 1) * step;
          mk[u] = __ldcg(part + 128 * p.x.d_v + row);
          lk[u] = __ldcg(part + 128 * p.x.d_v + 128 + row);
#pragma unroll
          for (int q = 0; q < kMergeQuads; ++q)
            x[u][q] = quad0 + 2 * q < quad1 ? __ldcg(reinterpret_cast<const float4*>(part) + (quad0 + 2 * q) * 128 + row) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (c0 + u >= cuts || mk[u] == -INFINITY) continue;  // a part in which the row sees nothing
          const float next = fmaxf(top, mk[u]), f = top == -INFINITY ? 0.f : exp2f(top - next), w = exp2f(mk[u] - next);
          top = next;
          l = l * f + lk[u] * w;
#pragma unroll
          for (int q = 0; q < kMergeQuads; ++q) {
            o[q][0] = o[q][0] * f + x[u][q].x * w;
            o[q][1] = o[q][1] * f + x[u][q].y * w;
            o[q][2] = o[q][2] * f + x[u][q].z * w;
            o[q][3] = o[q][3] * f + x[u][q].w * w;
          }
        }
      }
      const bool nothing = l == 0.f;
      const float inv = nothing ? 0.f : 1.f / l;
      const int64_t at = static_cast<int64_t>(rec.x + tok) * p.x.n_q + rec.z * p.G + (row - tok_in * p.G);
#pragma unroll
      for (int q = 0; q < kMergeQuads; ++q) {
        uint2 y = make_uint2(pack16<E>(o[q][0] * inv, o[q][1] * inv), pack16<E>(o[q][2] * inv, o[q][3] * inv));
        if (nothing) y = make_uint2(0u, 0u);
        if (put && quad0 + 2 * q < quad1) *reinterpret_cast<uint2*>(static_cast<E*>(p.x.out) + at * p.x.d_v + (quad0 + 2 * q) * 4) = y;
      }
      if (put && slice == 0 && side == 0 && p.x.lse != nullptr)
        p.x.lse[at] = nothing ? -INFINITY : (top + log2f(l)) * 0.69314718055994530942f;
    }
  }
}

// ------------------------------------------------------------------ host side
namespace {

constexpr int kMaxDevices = 64;
struct Device {
  bool ready = false;
  int sms = 0, pairs = 0;
};
Device g_dev[kMaxDevices];
std::mutex g_lock;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

constexpr int kMaxParts = 640;  // partial states in the workspace at most
constexpr int kSmPairs = 76;    // of a GB300; a constant, since the workspace's size is asked for without a device

// Whether pairs of CTAs run: they hold half of the keys and values each, which eases
// shared memory, the bound of a CTA alone, but take 512 rows at a time, so they need
// rows for two rounds.  Alone and in pairs: one prompt of 8192, 128 heads of 192 and 128,
// 1888 and 1600 to 1670 us; 32 heads of 128 on 8 key heads 382 and 344, of 4096 127 and
// 123; 64 heads on 8, 2048 tokens, 74 and 72; 16 prompts of 512 (2048 rows to a key head)
// 72 and 73.  Chunks over long contexts, which are cut, gain 3 to 7%, but the host sees the
// table's width, not their lengths, and 8 chunks of 300 over 2000 take 98 instead of 75.
bool in_pairs(const Problem& p) {
  const int64_t rows = static_cast<int64_t>(p.T) * (p.n_q / p.n_kv);  // of a key head
  return p.d_v > 64 && rows >= 4096 * static_cast<int64_t>(p.B) && rows * p.n_kv >= 2 * 512 * kSmPairs;
}
int item_tiles(const Problem& p) { return in_pairs(p) ? 4 : 2; }

// Partial states that a call can need: none where no item has more key tiles than a part has at least.
int parts_of(const Problem& p) {
  const int64_t keys = p.num_blocks > 0 ? static_cast<int64_t>(p.W) * kPage : p.Tk;
  if (keys <= kMinTiles * kTile) return 0;
  const int64_t span = item_tiles(p) * (kTile / (p.n_q / p.n_kv)), tiles = (keys + kTile - 1) / kTile;
  const int64_t pairs = p.S1 > 0 ? p.B * ((p.S1 + span - 1) / span) : p.T / span + p.B;
  // each factor bounded first: their product passes 64 bits for the largest dims
  const int64_t items = std::min<int64_t>(kMaxParts, std::min<int64_t>(kMaxParts, pairs) * p.n_kv);
  return static_cast<int>(std::min<int64_t>(kMaxParts, items * std::min<int64_t>(kMaxParts, (tiles + kMinTiles - 1) / kMinTiles)));
}
int part_floats(const Problem& p) { return item_tiles(p) * (128 * p.d_v + 256); }
size_t lists_bytes(const Problem& p) { return (sizeof(Head) + (3 * static_cast<size_t>(p.B) + 1) * sizeof(int) + 255) & ~size_t(255); }
size_t records_bytes(const Problem& p) { return (parts_of(p) * sizeof(Record) + 255) & ~size_t(255); }

cudaLaunchConfig_t config_of(unsigned ctas, bool pair, cudaStream_t s, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pair ? 2 : 1;
  return cfg;
}

template <typename E, bool kPair, bool kApart>
mla_status prepare_kernel(Device& d) {
  HEADS_CUDA(cudaFuncSetAttribute(prompt_attn_kernel<E, kPair, kApart>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes), "kernel set-up");
  cudaFuncAttributes fa;
  HEADS_CUDA(cudaFuncGetAttributes(&fa, prompt_attn_kernel<E, kPair, kApart>), "kernel attributes");
  if constexpr (kPair) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config_of(2, true, nullptr, attr);
    attr[0] = attr[1];
    cfg.numAttrs = 1;
    int n = 0;
    HEADS_CUDA(cudaOccupancyMaxActiveClusters(&n, prompt_attn_kernel<E, kPair, kApart>, &cfg), "kernel occupancy");
    if (n < 1) return fail(MLA_ERR_CUDA, "the kernel does not fit this device");
    d.pairs = n;
  }
  if (fa.numRegs < kRegs) return fail(MLA_ERR_CUDA, "the kernel was built with %d registers", fa.numRegs);  // what the warpgroups divide
  return MLA_OK;
}

template <typename E>
mla_status prepare_kernels(Device& d) {
  mla_status st = prepare_kernel<E, false, false>(d);
  if (st == MLA_OK) st = prepare_kernel<E, false, true>(d);
  if (st == MLA_OK) st = prepare_kernel<E, true, false>(d);
  return st;
}

// Kernel attributes and the tensor-map encoder; the first call on a device.
mla_status init_device(int* sms, int* pairs) {
  int dev = 0;
  HEADS_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(MLA_ERR_UNSUPPORTED, "device ordinal %d too large", dev);
  std::lock_guard<std::mutex> guard(g_lock);
  Device& d = g_dev[dev];
  if (!d.ready) {
    mla_status st = tensor_map_encoder(&g_encode);
    if (st != MLA_OK) return st;
    HEADS_CUDA(cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev), "device attributes");
    st = prepare_kernels<__nv_bfloat16>(d);
    if (st == MLA_OK) st = prepare_kernels<__half>(d);
    if (st != MLA_OK) return st;
    d.ready = true;
  }
  *sms = d.sms;
  *pairs = d.pairs;
  return MLA_OK;
}

template <typename E>
mla_status launch_attention(bool pair, unsigned workers, const Maps& maps, const Params& p, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config_of(pair ? 2 * workers : workers, pair, s, attr);
  HEADS_CUDA(pair ? cudaLaunchKernelEx(&cfg, prompt_attn_kernel<E, true, false>, maps, p)
             : p.vc == 1 ? cudaLaunchKernelEx(&cfg, prompt_attn_kernel<E, false, true>, maps, p)
                         : cudaLaunchKernelEx(&cfg, prompt_attn_kernel<E, false, false>, maps, p),
             "kernel launch");
  return MLA_OK;
}

}  // namespace

size_t tiles_workspace(const Problem& p) { return lists_bytes(p) + records_bytes(p) + static_cast<size_t>(parts_of(p)) * part_floats(p) * sizeof(float); }

mla_status launch_tiles(const Problem& x, cudaStream_t s) {
  int sms = 0, cta_pairs = 0;
  const mla_status st = init_device(&sms, &cta_pairs);
  if (st != MLA_OK) return st;
  const bool pair = in_pairs(x);
  Params p;
  p.x = x;
  uint8_t* ws = static_cast<uint8_t*>(x.workspace);
  p.head = reinterpret_cast<Head*>(ws);
  p.first = reinterpret_cast<int*>(ws + sizeof(Head));
  p.part0 = p.first + x.B + 1;
  p.order = p.part0 + x.B;
  p.records = reinterpret_cast<Record*>(ws + lists_bytes(x));
  p.parts = reinterpret_cast<float*>(ws + lists_bytes(x) + records_bytes(x));
  p.part_floats = part_floats(x);
  p.max_parts = parts_of(x);
  p.G = x.n_q / x.n_kv;
  p.tpt = kTile / p.G;
  p.tiles = item_tiles(x);
  p.span = p.tiles * p.tpt;
  p.kc = (x.d_qk + 63) / 64;
  p.vc = x.d_v > 64 ? 2 : 1;
  p.slots = pair ? Shape<true>::slots(p.kc) : Shape<false>::slots(p.kc);
  p.sms = pair ? cta_pairs : sms;
  const uint32_t bf16 = x.dtype == MLA_ROPE_BF16 ? 1 : 0;
  const uint32_t M = pair ? 256 : 128;
  p.idesc_s = make_idesc_f16(M, 128, bf16, 0, 0);                                                       // A, B K-major
  p.idesc_v = make_idesc_f16(M, pair ? 128 : static_cast<uint32_t>((x.d_v + 15) & ~15), bf16, 0, 1);  // B MN-major
  p.ks_qk = (x.d_qk + 15) / 16;
  p.wait_ns = host_wait_limit_ns();
  Maps maps;
  {
    const int64_t size[3] = {x.d_qk, x.n_q, x.T}, stride[2] = {x.q.head_stride, x.q.token_stride};
    const int box[3] = {64, p.G, p.tpt};
    const mla_status ms = tmap(g_encode, &maps.q, x.dtype, x.q.data, 3, size, stride, box, "q");
    if (ms != MLA_OK) return ms;
  }
  for (int i = 0; i < 2; ++i) {
    const mla_kv_cache& c = i == 0 ? x.k : x.v;
    const bool none = x.num_blocks == 0 && x.Tk == 0;  // no key is ever loaded
    const int64_t size[4] = {i == 0 ? x.d_qk : x.d_v, x.num_blocks > 0 ? kPage : std::max(1, x.Tk), x.n_kv, std::max(1, x.num_blocks)};
    const int64_t stride[3] = {c.row_stride, c.head_stride, c.block_stride};
    const int box[4] = {64, pair || (i == 1 && p.vc == 2) ? 64 : 128, 1, 1};
    CUtensorMap* map = i == 0 ? &maps.k : &maps.v;
    const mla_status ms = none ? MLA_OK : tmap(g_encode, map, x.dtype, c.data, 4, size, stride, box, i == 0 ? "k" : "v");
    if (ms != MLA_OK) return ms;
    if (none) *map = maps.q;
  }
  const bool bf = x.dtype == MLA_ROPE_BF16;
  prompt_plan_kernel<<<1, x.B <= kWarpSeqs ? 32 : kPlanThreads, 0, s>>>(p);
  HEADS_CUDA(cudaGetLastError(), "plan launch");
  const int64_t groups = x.S1 > 0 ? static_cast<int64_t>(x.B) * ((x.S1 + p.span - 1) / p.span) : x.T / p.span + x.B;
  const int64_t most = std::min<int64_t>(p.sms, groups) * x.n_kv + p.max_parts;
  const unsigned workers = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(p.sms, most)));
  const mla_status ls = bf ? launch_attention<__nv_bfloat16>(pair, workers, maps, p, s) : launch_attention<__half>(pair, workers, maps, p, s);
  if (ls != MLA_OK) return ls;
  if (p.max_parts > 0)
    HEADS_CUDA(bf ? launch_after(prompt_merge_kernel<__nv_bfloat16>, dim3(static_cast<unsigned>(4 * sms)), kMergeThreads, 0, s, p)
                  : launch_after(prompt_merge_kernel<__half>, dim3(static_cast<unsigned>(4 * sms)), kMergeThreads, 0, s, p),
               "merge launch");
  return MLA_OK;
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
  if (static_cast<int64_t>(d.T) * d.n_q >= (1ll << 31) - 1024 || d.B > (1 << 24))
    return fail(MLA_ERR_SHAPE, "T * n_q must be below 2^31 - 1024, B at most 2^24");
  if (d.Tk >= INT32_MAX - 256) return fail(MLA_ERR_SHAPE, "Tk=%d must be below 2^31 - 257", d.Tk);
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
