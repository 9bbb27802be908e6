// What the two kernels of prompt attention share: a call's work, its order over tiles, the
// permutation of LDS rows.
#pragma once

#include <algorithm>

#include "attention.hpp"
#include "kernels.hpp"

namespace dspark {

namespace {

struct Work {
  PromptArgs a;
  int G;
  float c;               // scale * log2 e
};

template <int HD>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (HD == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  return ((r & 3) << 2) | ((r >> 2) & 3);
}

__device__ __forceinline__ void sequence(const PromptArgs& a, int b, int& start, int& n) {
  start = clampi(a.cu_seqlens[b], 0, a.T);
  n = clampi(a.cu_seqlens[b + 1], start, a.T) - start;
}

// The sequence and row tile of item u; every wave finds them for itself.  A causal tile
// costs as much as its index says, and the dearest go first: item u is the u-th of all
// tiles by falling index (of up to 64 sequences; a longer batch has tiles enough to even
// out in the order of its sequences, a sequence's last first).
__device__ bool find_tile(const Work& w, int u, int rows, int& start, int& n, int& tile) {
  const PromptArgs& a = w.a;
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](int len) { return (int)(((int64_t)len * w.G + rows - 1) / rows); };
  if (a.B == 1) {
    sequence(a, 0, start, n);
    start = uniform(start);
    n = uniform(n);
    tile = uniform(tiles_of(n)) - 1 - u;
    return tile >= 0;
  }
  if (a.causal && a.B <= 64) {
    int s = 0, len = 0;
    if (lane < a.B) sequence(a, lane, s, len);
    const int mine = tiles_of(len);
    // the level: the largest index that leaves more than u tiles at or above it (all counts
    // are below 2^24: exact in float)
    auto at_least = [&](int level) { return uniform((int)group_sum((float)max(mine - level, 0), 64)); };
    int lo = 0, hi = uniform((int)wave_max_u32((uint32_t)mine));
    if (at_least(0) <= u) return false;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (at_least(mid) > u) lo = mid;
      else hi = mid;
    }
    uint64_t have = __ballot(mine > lo);     // one tile of this index each
    for (int skip = u - at_least(lo + 1); skip > 0; --skip) have &= have - 1;
    const int q = __builtin_ctzll(have);
    start = __builtin_amdgcn_readlane(s, q);
    n = __builtin_amdgcn_readlane(len, q);
    tile = lo;
    return true;
  }
  int before = 0;
  for (int base = 0; base < a.B; base += 64) {
    int s = 0, len = 0, cnt = 0;
    if (base + lane < a.B) {
      sequence(a, base + lane, s, len);
      cnt = tiles_of(len);
    }
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(inc, o);
      if (lane >= o) inc += v;
    }
    const uint64_t hit = __ballot(before + inc > u);
    if (hit) {
      const int q = __builtin_ctzll(hit);
      start = __builtin_amdgcn_readlane(s, q);
      n = __builtin_amdgcn_readlane(len, q);
      tile = before + __builtin_amdgcn_readlane(inc, q) - 1 - u;
      return true;
    }
    before += __builtin_amdgcn_readlane(inc, 63);
  }
  return false;
}

__device__ __forceinline__ float halves_sum(float v) {
  uint32_t lo, hi;
  halves_pair(__float_as_uint(v), lo, hi);
  return __uint_as_float(lo) + __uint_as_float(hi);
}

// The running maximum is raised only when a row's scores exceed it by kRaise (weights up to
// 2^kRaise, more where the maximum itself is rounded by more than that, which neither float
// nor bf16 minds): the accumulators are rescaled on a row's first tile and hardly ever after.
constexpr float kRaise = 8.0f;

Work work_of(const PromptArgs& a) {
  Work w;
  w.a = a;
  w.G = a.nh / a.nkv;
  w.c = a.scale * kLog2e;
  return w;
}

}  // namespace

}  // namespace dspark
