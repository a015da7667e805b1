// Host checks that calls with strided tensors share: do two of them touch a
// common byte, and is an output's layout free of places that coincide.
#pragma once
#include <stdint.h>

#include <initializer_list>

namespace mlasp {

inline bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// What a call reads or writes: a run of bytes at each of n[0] x n[1] x n[2] places.
struct Area {
  uintptr_t at;
  int64_t n[3], stride[3], bytes;  // strides in bytes
};
inline Area run(const void* ptr, int64_t bytes) {
  return {reinterpret_cast<uintptr_t>(ptr), {1, 1, 1}, {0, 0, 0}, bytes};
}

// Whether the areas have a byte in common.  Views of one tensor interleave, so
// areas whose stretches overlap are also told apart by their strides: runs of a
// and b bytes that repeat at multiples of g miss one another when the distance
// of their starts, modulo g, is at least a, and b short of g.  Tried for every
// choice of the levels that repeat, the others making up the run; what none of
// them tells apart counts as overlapping.
inline bool overlap(const Area& a, const Area& b) {
  typedef __int128 Wide;  // 2^40 places times a stride of 2^42
  if (a.at == 0 || b.at == 0) return false;
  const Wide delta = static_cast<Wide>(b.at) - static_cast<Wide>(a.at);
  auto stride = [](const Area& x, int i) { return x.n[i] > 1 ? static_cast<Wide>(x.stride[i]) : 0; };
  auto length = [&](const Area& x, int repeats) {
    Wide l = x.bytes;
    for (int i = 0; i < 3; ++i)
      if (!((repeats >> i) & 1)) l += static_cast<Wide>(x.n[i] - 1) * stride(x, i);
    return l;
  };
  if (delta >= length(a, 0) || -delta >= length(b, 0)) return false;
  for (int repeats = 1; repeats < 8; ++repeats) {
    Wide g = 0;
    for (int i = 0; i < 3; ++i) {
      if (!((repeats >> i) & 1)) continue;
      for (Wide y : {stride(a, i), stride(b, i)}) {
        while (y != 0) {
          const Wide r = g % y;
          g = y;
          y = r;
        }
      }
    }
    if (g == 0) continue;  // nothing repeats: the stretches have been compared
    const Wide r = (delta % g + g) % g;
    if (r >= length(a, repeats) && g - r >= length(b, repeats)) return false;
  }
  return true;
}

// Whether no two places of an output coincide: sorted by stride, each level steps over all of the ones inside it.
inline bool distinct(const Area& a) {
  typedef __int128 Wide;
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (a.stride[order[j]] > a.stride[order[j + 1]]) {
        const int t = order[j];
        order[j] = order[j + 1];
        order[j + 1] = t;
      }
  Wide inner = a.bytes;
  for (int i : order) {
    if (a.n[i] <= 1) continue;
    if (a.stride[i] < inner) return false;
    inner += static_cast<Wide>(a.n[i] - 1) * a.stride[i];
  }
  return true;
}

}  // namespace mlasp
