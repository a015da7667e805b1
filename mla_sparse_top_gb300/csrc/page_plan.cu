// Page plan for GB300 (sm_103a): block tables, slot maps, positions and tree
// masks of one step from the request lengths (formulas in mla_pages.h).
//
// One launch, no scratch and no atomics on results: what a block needs from
// the sequences before its own is two sums (pages taken, tokens added), and
// every block adds them up itself.  B lengths are a few KB that stay in L2, so
// this costs less than a second launch or a chain of blocks waiting for one
// another, and the result does not depend on the order of the blocks.
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "../../include/mla_pages.h"

namespace mlapg {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPage = 128;
constexpr int kTileTokens = 1024;  // packed: tokens of one block

__device__ unsigned int g_page_status = 0;

struct Params {
  mla_page_io io;
  int B, S1, T, W, num_blocks, num_free, seqs_per_block;
};

struct Seq {
  int64_t ctx;  // cached positions
  int64_t add;  // new tokens
  int have;     // table entries the cached positions use
  int need;     // pages to take
};

__device__ __forceinline__ int pages_of(int64_t positions, int W) {
  return static_cast<int>(min(static_cast<int64_t>(W), (positions + kPage - 1) / kPage));
}

__device__ __forceinline__ Seq load_seq(const Params& p, int b) {
  Seq s;
  s.ctx = max(0, __ldg(p.io.ctx_lens + b));
  s.add = p.io.new_lens != nullptr ? max(0, __ldg(p.io.new_lens + b)) : p.S1;
  if (p.S1 > 0) s.add = min(s.add, static_cast<int64_t>(p.S1));
  s.have = pages_of(s.ctx, p.W);
  s.need = pages_of(s.ctx + s.add, p.W) - s.have;
  return s;
}

// Sums of the block's (pages, tokens) pairs over the threads before this one;
// `total` is the whole block's.  The block calls it together.
__device__ __forceinline__ longlong2 block_scan(longlong2 v, longlong2* part, longlong2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  longlong2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) {
      x.x += a;
      x.y += b;
    }
  }
  __syncthreads();  // the last use of `part` is over
  if (lane == 31) part[warp] = x;
  __syncthreads();
  longlong2 before = make_longlong2(0, 0);
  total = make_longlong2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const longlong2 y = part[w];
    if (w < warp) {
      before.x += y.x;
      before.y += y.y;
    }
    total.x += y.x;
    total.y += y.y;
  }
  return make_longlong2(before.x + x.x - v.x, before.y + x.y - v.y);
}

// Page `lb` of a sequence: the table's own entry for the cached positions, the
// free list's for the new ones (so no block waits for another's table writes).
__device__ __forceinline__ int page_id(const Params& p, int b, int64_t lb, int have, int64_t first_free) {
  if (lb >= p.W) return -1;
  if (lb < have) return p.io.block_table[static_cast<int64_t>(b) * p.W + lb];
  const int64_t k = first_free + lb - have;
  return k < p.num_free ? __ldg(p.io.free_blocks + k) : -1;
}

__device__ __forceinline__ int64_t row_of(const Params& p, int b, int64_t slot, int have, int64_t first_free,
                                          unsigned& flags) {
  const int64_t lb = slot / kPage;
  const int id = page_id(p, b, lb, have, first_free);
  if (id >= 0 && id < p.num_blocks) return static_cast<int64_t>(id) * kPage + slot % kPage;
  flags |= lb >= p.W || (lb >= have && first_free + lb - have >= p.num_free) ? MLA_DEVICE_NO_PAGE : MLA_DEVICE_BAD_BLOCK;
  return -1;
}

__device__ __forceinline__ int sat32(int64_t v) { return static_cast<int>(min(v, static_cast<int64_t>(0x7fffffff))); }

// Table entry k of one sequence's new pages.
__device__ __forceinline__ void write_page(const Params& p, int b, int have, int k, int64_t first_free, unsigned& flags) {
  const int id = page_id(p, b, have + k, have, first_free);
  p.io.block_table[static_cast<int64_t>(b) * p.W + have + k] = id;
  if (id < 0 && first_free + k >= p.num_free) flags |= MLA_DEVICE_NO_PAGE;
}
// A step that adds a few tokens takes a page or none: the sequence's own thread
// writes up to kOwnPages, so all sequences of a block do at once; the pages of
// prompts beyond those are a warp's work.
constexpr int kOwnPages = 2;
__device__ __forceinline__ void write_own_pages(const Params& p, int b, const Seq& s, int64_t first_free,
                                                unsigned& flags) {
  for (int k = 0; k < min(s.need, kOwnPages); ++k) write_page(p, b, s.have, k, first_free, flags);
}
__device__ __forceinline__ void write_more_pages(const Params& p, int b, int have, int need, int64_t first_free,
                                                 unsigned& flags) {
  for (int k = kOwnPages + (threadIdx.x & 31); k < need; k += 32) write_page(p, b, have, k, first_free, flags);
}

// Outputs of each sequence: thread's sequence b with its sums.
__device__ __forceinline__ void write_seq(const Params& p, int b, const Seq& s, longlong2 before) {
  p.io.act_seqs[b] = sat32(s.ctx + s.add);
  if (p.io.cu_seqs != nullptr) {
    if (b == 0) p.io.cu_seqs[0] = 0;
    p.io.cu_seqs[b + 1] = sat32(before.y + s.add);
  }
  if (b == p.B - 1 && p.io.num_taken != nullptr)
    *p.io.num_taken = static_cast<int>(min(static_cast<int64_t>(before.x + s.need), static_cast<int64_t>(p.num_free)));
}

struct Shared {
  longlong2 part[kWarps];
  int64_t ctx[kThreads], first_free[kThreads], start[kThreads];
  int have[kThreads], need[kThreads];
  int add[kThreads];
};

__device__ __forceinline__ void keep(Shared& sh, int at, const Seq& s, longlong2 before) {
  sh.ctx[at] = s.ctx;
  sh.first_free[at] = before.x;
  sh.start[at] = before.y;
  sh.have[at] = s.have;
  sh.need[at] = s.need;
  sh.add[at] = sat32(s.add);
}

// Mask and depth of drafted token i: its parents have smaller indices, so the
// walk up goes through the mask's words from the highest down.  Without parents
// every earlier token is an ancestor.
__device__ __forceinline__ int walk_up(const Params& p, int b, int i, uint64_t* mask) {
  const int words = (p.S1 + 63) / 64;
  if (p.io.parents == nullptr) {
    for (int k = 0; k < words; ++k)
      mask[k] = k < (i >> 6) ? ~0ull : (k == (i >> 6) ? ~0ull >> (63 - (i & 63)) : 0ull);
    return i;
  }
  const int32_t* par = p.io.parents + static_cast<int64_t>(b) * p.S1;
  int w = words - 1, depth = -1;
  uint64_t bits = 0;
  for (int c = i; c >= 0;) {
    if (mask != nullptr)
      while (w > (c >> 6)) {
        mask[w--] = bits;
        bits = 0;
      }
    bits |= 1ull << (c & 63);
    ++depth;
    const int up = __ldg(par + c);
    c = up < c ? up : -1;
  }
  if (mask != nullptr)
    for (; w >= 0; --w) {
      mask[w] = bits;
      bits = 0;
    }
  return depth;
}

// Padded layout: a block owns seqs_per_block sequences (at most one per thread).
__global__ void __launch_bounds__(kThreads) plan_padded_kernel(const Params p) {
  __shared__ Shared sh;
  const int b0 = blockIdx.x * p.seqs_per_block, nb = min(p.seqs_per_block, p.B - b0);
  const int tid = threadIdx.x;
  longlong2 prior = make_longlong2(0, 0), total;
#pragma unroll 4
  for (int b = tid; b < b0; b += kThreads) {
    const Seq s = load_seq(p, b);
    prior.x += s.need;
    prior.y += s.add;
  }
  Seq s = {};
  if (tid < nb) s = load_seq(p, b0 + tid);
  block_scan(prior, sh.part, prior);  // prior: the sums over all sequences before the block's
  longlong2 before = block_scan(make_longlong2(s.need, s.add), sh.part, total);
  before.x += prior.x;
  before.y += prior.y;
  unsigned flags = 0;
  if (tid < nb) {
    keep(sh, tid, s, before);
    write_seq(p, b0 + tid, s, before);
    write_own_pages(p, b0 + tid, s, before.x, flags);
  }
  __syncthreads();
  for (int q = tid >> 5; q < nb; q += kWarps)
    write_more_pages(p, b0 + q, sh.have[q], sh.need[q], sh.first_free[q], flags);
  const int words = (p.S1 + 63) / 64;
  for (int r = tid; r < nb * p.S1; r += kThreads) {
    const int q = r / p.S1, i = r - q * p.S1, b = b0 + q;
    const int64_t t = static_cast<int64_t>(b0) * p.S1 + r;
    const bool live = i < sh.add[q];
    uint64_t* mask = p.io.tree_mask != nullptr ? p.io.tree_mask + t * words : nullptr;
    int depth = i;
    if (!live) {
      if (mask != nullptr)
        for (int w = 0; w < words; ++w) mask[w] = 0;
    } else if (p.io.parents != nullptr || mask != nullptr) {
      depth = walk_up(p, b, i, mask);
    }
    p.io.cache_index[t] = live ? row_of(p, b, sh.ctx[q] + i, sh.have[q], sh.first_free[q], flags) : -1;
    if (p.io.positions != nullptr) p.io.positions[t] = live ? sat32(sh.ctx[q] + depth) : 0;
    if (p.io.seq_ids != nullptr) p.io.seq_ids[t] = live ? b : -1;
  }
  if (flags) atomicOr(&g_page_status, flags);
}

// Packed layout: a block owns kTileTokens rows.  It runs over the sequences in
// chunks of one per thread, up to the chunk that ends its tile, and at least up
// to chunk blockIdx.x; block c writes the per-sequence outputs of chunk c, and
// all the blocks that come past a chunk share out its pages.
__global__ void __launch_bounds__(kThreads) plan_packed_kernel(const Params p) {
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  const int chunks = (p.B + kThreads - 1) / kThreads;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTileTokens;
  const int64_t t1 = min(t0 + kTileTokens, static_cast<int64_t>(p.T));
  longlong2 carry = make_longlong2(0, 0);
  unsigned flags = 0;
  for (int c = 0; c < chunks && (carry.y < t1 || c <= static_cast<int>(blockIdx.x)); ++c) {
    const int b = c * kThreads + tid;
    Seq s = {};
    if (b < p.B) s = load_seq(p, b);
    longlong2 total;
    longlong2 before = block_scan(make_longlong2(s.need, s.add), sh.part, total);
    before.x += carry.x;
    before.y += carry.y;
    keep(sh, tid, s, before);
    const int n = min(kThreads, p.B - c * kThreads);
    if (c == static_cast<int>(blockIdx.x)) {
      if (b < p.B) write_seq(p, b, s, before);
      if (c == chunks - 1 && carry.y + total.y > p.T) flags |= MLA_DEVICE_NO_PAGE;
    }
    __syncthreads();
    if (c <= static_cast<int>(blockIdx.x)) {  // blocks c .. gridDim.x - 1 come past chunk c
      const int sharers = static_cast<int>(gridDim.x) - c;
      for (int q = (static_cast<int>(blockIdx.x) - c) * kWarps + (tid >> 5); q < n; q += sharers * kWarps)
        for (int k = tid & 31; k < sh.need[q]; k += 32)
          write_page(p, c * kThreads + q, sh.have[q], k, sh.first_free[q], flags);
    }
    // this tile's rows that belong to the chunk's sequences
    const int64_t lo = max(t0, static_cast<int64_t>(carry.y)), hi = min(t1, static_cast<int64_t>(carry.y + total.y));
    for (int64_t t = t0 + tid; t < hi; t += kThreads) {
      if (t < lo) continue;
      int a = 0, e = n - 1;  // the last sequence that starts at or before t
      while (a < e) {
        const int m = (a + e + 1) >> 1;
        if (sh.start[m] <= t) a = m;
        else e = m - 1;
      }
      const int64_t slot = sh.ctx[a] + (t - sh.start[a]);
      const int q = c * kThreads + a;
      p.io.cache_index[t] = row_of(p, q, slot, sh.have[a], sh.first_free[a], flags);
      if (p.io.positions != nullptr) p.io.positions[t] = sat32(slot);
      if (p.io.seq_ids != nullptr) p.io.seq_ids[t] = q;
    }
    carry.x += total.x;
    carry.y += total.y;
    __syncthreads();  // `sh` is rewritten by the next chunk
  }
  for (int64_t t = t0 + tid; t < t1; t += kThreads) {  // rows behind the last token
    if (t < carry.y) continue;
    p.io.cache_index[t] = -1;
    if (p.io.positions != nullptr) p.io.positions[t] = 0;
    if (p.io.seq_ids != nullptr) p.io.seq_ids[t] = -1;
  }
  if (flags) atomicOr(&g_page_status, flags);
}

}  // namespace mlapg

namespace {

thread_local char g_page_error[256] = "";

mla_status page_fail(mla_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mla_status page_fail(mla_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_page_error, sizeof g_page_error, fmt, ap);
  va_end(ap);
  return s;
}

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

struct Range {
  const void* ptr;
  int64_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.ptr || !b.ptr || !a.bytes || !b.bytes) return false;  // an empty list is nowhere
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.ptr), y = reinterpret_cast<uintptr_t>(b.ptr);
  return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

}  // namespace

extern "C" {

mla_status mla_page_plan(const mla_page_dims* dims, const mla_page_io* io, void* stream) {
  g_page_error[0] = '\0';
  if (dims == nullptr || io == nullptr) return page_fail(MLA_ERR_NULL, "dims or io is NULL");
  const mla_page_dims d = *dims;
  if (d.B < 0 || d.S1 < 0 || d.T < 0 || d.num_free < 0 || d.num_blocks < 1 || d.max_blocks_per_seq < 1)
    return page_fail(MLA_ERR_SHAPE, "B, S1, T, num_free must be >= 0, num_blocks and max_blocks_per_seq >= 1");
  if (d.num_blocks >= (1 << 24)) return page_fail(MLA_ERR_SHAPE, "num_blocks=%d must be < 2^24", d.num_blocks);
  if (d.block_size != mlapg::kPage)
    return page_fail(MLA_ERR_UNSUPPORTED, "block_size=%d: only 128 is implemented", d.block_size);
  if (d.S1 > 0 && static_cast<int64_t>(d.B) * d.S1 != d.T)
    return page_fail(MLA_ERR_SHAPE, "padded rows: T=%d is not B * S1 = %d * %d", d.T, d.B, d.S1);
  if (d.S1 == 0 && (io->parents != nullptr || io->tree_mask != nullptr))
    return page_fail(MLA_ERR_UNSUPPORTED, "parents and tree_mask need padded rows (S1 >= 1)");
  if (d.B == 0 && d.T == 0) return MLA_OK;  // nothing is read or written
  if (d.B == 0) return page_fail(MLA_ERR_SHAPE, "packed rows without a sequence (B=0, T=%d)", d.T);
  if (!io->ctx_lens || !io->block_table || !io->act_seqs || (d.T > 0 && !io->cache_index) ||
      (d.num_free > 0 && !io->free_blocks) || (d.S1 == 0 && !io->new_lens))
    return page_fail(MLA_ERR_NULL, "a required pointer is NULL (packed rows need new_lens)");
  const void* words[] = {io->ctx_lens, io->new_lens, io->free_blocks, io->parents, io->block_table,
                         io->act_seqs, io->positions, io->seq_ids,    io->cu_seqs, io->num_taken};
  for (const void* w : words)
    if (!aligned(w, 4)) return page_fail(MLA_ERR_ALIGN, "int32 tensors must be 4-byte aligned");
  if (!aligned(io->cache_index, 8) || !aligned(io->tree_mask, 8))
    return page_fail(MLA_ERR_ALIGN, "cache_index and tree_mask must be 8-byte aligned");
  // every block adds up the lengths of the sequences before its own: nothing it reads may be an output
  const int64_t B = d.B, T = d.T, words64 = (static_cast<int64_t>(d.S1) + 63) / 64;
  const Range in[] = {{io->ctx_lens, 4 * B}, {io->new_lens, 4 * B}, {io->free_blocks, 4ll * d.num_free},
                      {io->parents, 4 * T}};
  const Range out[] = {{io->block_table, 4 * B * d.max_blocks_per_seq}, {io->act_seqs, 4 * B}, {io->cache_index, 8 * T},
                       {io->positions, 4 * T}, {io->seq_ids, 4 * T}, {io->cu_seqs, 4 * (B + 1)},
                       {io->tree_mask, 8 * T * words64}, {io->num_taken, 4}};
  for (const Range& o : out)
    for (const Range& i : in)
      if (overlap(i, o)) return page_fail(MLA_ERR_UNSUPPORTED, "an output overlaps an input");
  for (const Range& o : out)
    for (const Range* q = out; q != &o; ++q)
      if (overlap(*q, o)) return page_fail(MLA_ERR_UNSUPPORTED, "two outputs overlap");
  mlapg::Params p;
  p.io = *io;
  p.B = d.B;
  p.S1 = d.S1;
  p.T = d.T;
  p.W = d.max_blocks_per_seq;
  p.num_blocks = d.num_blocks;
  p.num_free = d.num_free;
  p.seqs_per_block = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d.S1 > 0) {
    // about one row per thread, at most one sequence per thread
    p.seqs_per_block = std::max(1, mlapg::kThreads / d.S1);
    const unsigned grid = static_cast<unsigned>((d.B + p.seqs_per_block - 1) / p.seqs_per_block);
    mlapg::plan_padded_kernel<<<grid, mlapg::kThreads, 0, s>>>(p);
  } else {
    const int tiles = static_cast<int>((static_cast<int64_t>(d.T) + mlapg::kTileTokens - 1) / mlapg::kTileTokens);
    const int chunks = (d.B + mlapg::kThreads - 1) / mlapg::kThreads;
    mlapg::plan_packed_kernel<<<static_cast<unsigned>(std::max(tiles, chunks)), mlapg::kThreads, 0, s>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return page_fail(MLA_ERR_CUDA, "page plan launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

const char* mla_page_last_error(void) { return g_page_error; }

mla_status mla_page_device_status(void* stream, uint32_t* flags, int32_t clear) {
  g_page_error[0] = '\0';
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return page_fail(MLA_ERR_CUDA, "cudaStreamSynchronize: %s", cudaGetErrorString(e));
  unsigned int v = 0;
  e = cudaMemcpyFromSymbol(&v, mlapg::g_page_status, sizeof v);
  if (e != cudaSuccess) return page_fail(MLA_ERR_CUDA, "reading the status word: %s", cudaGetErrorString(e));
  if (clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(mlapg::g_page_status, &zero, sizeof zero);
    if (e != cudaSuccess) return page_fail(MLA_ERR_CUDA, "clearing the status word: %s", cudaGetErrorString(e));
  }
  if (flags) *flags = v;
  if (v != 0) return page_fail(MLA_ERR_DEVICE_STATUS, "page plan device status 0x%x", v);
  return MLA_OK;
}

}  // extern "C"
