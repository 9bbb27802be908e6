// Attention of a few query tokens per request over its pages of the key-value cache.
//
//   out[r] = sum_s exp2(x_rs - m_r) v_s / sum_s exp2(x_rs - m_r),   x_rs = q_r . k_s * scale * log2 e
//
// over the keys s row r sees, in one pass with a running maximum m_r and sum.  The nh / nkv
// query heads that share a kv head, times the request's query tokens, are the rows of one
// product, so a key or value is read from memory once per kv head (row blocks of 16 RT).
//
// Scores are formed transposed, S^T = K Q^T, with v_mfma_f32_16x16x32_bf16 over tiles of 32
// keys: lane (g, c) = (lane / 16, lane % 16) then holds row c and the keys 16 s + 4 g + i
// (s = 0, 1; i = 0..3).  The second product O^T = V^T P^T may take its 32 keys in any order
// as long as both operands agree, so those eight scores, rounded to bf16, are its B operand
// as they stand.
//
// Up to 16 rows (paged_rows): memory-bound, one product hardly fills a matrix instruction.
// Each of a workgroup's four or eight waves takes tiles of its own straight into registers; V's
// operand (eight keys of one dim per lane) comes from loads of 8 consecutive dims of eight
// keys (16 lanes cover a row, 16 bytes each), transposed by byte permutes, product t then
// covering the dims 8 c + t.  The waves are joined through LDS at the end.  256 requests of
// one token over 2048 keys, 32/8 heads of 128: 380 us, 5.7 TB/s.
// More rows (paged_shared): below.
//
// Work items (request, range of its keys) times (row block, kv head) come from the lengths
// on the device: ranges are cut equal and listed by falling length (paged_plan), each
// workgroup takes one.  A request of one range is written straight to the output; the
// others leave a maximum, a sum and an unnormalised row each, joined by paged_join in the
// order of the ranges.
//
// Which keys a row sees (kSeen) is one of three rules:
//   kBlock   those up to its own place (causal), or all
//   kRecent  of those, the last `window` up to its own place and the first `sinks`
//   kTree    the context before the block, and the block's keys that its mask names
// In a tile that some row does not see whole, a row's rule is a word of 32 bits, one a key.
// Between the sinks and the first window of a request lie keys that no row sees: they are
// left out of the request's *span*, in which ranges and tiles are counted.  The span's keys
// below sink_keys are the cache's own, those behind it lie `skip` further.
#pragma once

#include <algorithm>

#include "attention.hpp"
#include "kernels.hpp"

namespace dspark {

namespace {

// The running maximum is raised only when a row's scores exceed it by kRaise (weights up
// to 2^kRaise, more where the maximum itself is rounded by more than that, which neither float
// nor bf16 minds): the accumulators are rescaled on a row's first tile and hardly ever after.
constexpr float kRaise = 8.0f;

constexpr int KT = 32;         // keys per tile
constexpr int kStep = 4 * KT;  // ranges are whole numbers of these
constexpr int kCus = 256;      // compute units of the card
constexpr int kJoinGroups = 2048;   // workgroups of the joining pass aimed at

enum Seen { kBlock, kRecent, kTree };

// a range of one request's span: the work of a workgroup for every (row block, kv head)
struct __attribute__((aligned(16))) Item {
  int b, k0, k1;       // request, k0 .. k1 - 1 of its span
  int pid;             // partial to leave, or -1: the request's only range
  int q0, n, kv;       // the request's first query token, their number, its keys
  int skip;            // keys left out of the span
};

struct Work {
  PagedArgs a;
  int G, RB, unit;     // heads per kv head, row blocks, nkv * RB
  int target_log2;     // items aimed at, a power of two
  int min_chunk;       // keys of a range, at least
  int cut;             // requests may be cut: some can be longer than one range may be
  int pid_cap;         // ranges the workspace has room for
  float c;             // scale * log2 e
  float* part_o;       // [pid_cap, unit, 16 RT, hd]
  floatx4* part_ml;    // [pid_cap, unit, 16 RT]: maximum, sum of rounded weights, of unrounded ones
  int2* req;           // [B]: first partial and number of ranges of a split request (one: not split)
  Item* plan;          // the items, dearest first, or null: one request, or none is ever cut
  int* count;          // how many of them
};

// n counts all of the request's query tokens; the first max_q of them are computed
__device__ __forceinline__ void request(const PagedArgs& a, int b, int& q0, int& n, int& kv) {
  q0 = clampi(a.cu_q[b], 0, a.T);
  n = clampi(a.cu_q[b + 1], q0, a.T) - q0;
  kv = clampi(a.kv_len[b], 0, a.width << a.page_shift);
}

// The keys of a request that some row sees, and how many before them are left out.  The window of
// its first row is the lowest; it begins with a whole group of keys that lie together (16, or
// a smaller page), so that a page behind the window, which the caller may have given back, is
// never looked for.
template <int kSeen>
__device__ __forceinline__ int span_of(const PagedArgs& a, int n, int kv, int& skip) {
  skip = 0;
  if constexpr (kSeen == kRecent) {
    // (not below 0: the difference of the two is then within 32 bits, whatever the lengths)
    const int low = max(kv - n - a.window + 1, 0) & -min(1 << a.page_shift, 16);
    skip = max(low - a.sink_keys, 0);
  }
  return kv - skip;
}

// Ranges of all requests are at most `chunk` keys; a longer request is cut into equal ones.
__device__ __forceinline__ int chunk_of(const Work& w, int64_t total) {
  const int64_t per = (total * w.unit + (1 << w.target_log2) - 1) >> w.target_log2;
  const int64_t up = (per + kStep - 1) / kStep * kStep;
  return (int)(up < w.min_chunk ? w.min_chunk : up > (1 << 30) ? (1 << 30) : up);
}
__device__ __forceinline__ int range_len(int kv, int ranges) {
  return ((kv + ranges - 1) / ranges + kStep - 1) / kStep * kStep;
}

// the u-th item of the call
template <int kSeen>
__device__ __forceinline__ bool find_item(const Work& w, int u, Item& it) {
  const PagedArgs& a = w.a;
  if (w.plan) {
    if (u >= *w.count) return false;
    it = w.plan[u];
  } else if (a.B == 1 && w.cut) {
    request(a, 0, it.q0, it.n, it.kv);
    const int span = span_of<kSeen>(a, it.n, it.kv, it.skip), chunk = chunk_of(w, span);
    const int len = range_len(span, max(1, (span + chunk - 1) / chunk));
    const int ranges = len > 0 ? (span + len - 1) / len : 1;
    if (u >= ranges || it.n == 0) return false;
    it.b = 0;
    it.k0 = u * len;
    it.k1 = min(span, it.k0 + len);
    it.pid = ranges > 1 ? u : -1;
    if (u == 0 && threadIdx.x == 0) w.req[0] = make_int2(0, ranges);
  } else {
    request(a, u, it.q0, it.n, it.kv);
    if (it.n == 0) return false;
    it.b = u;
    it.k0 = 0;
    it.k1 = span_of<kSeen>(a, it.n, it.kv, it.skip);
    it.pid = -1;
  }
  it.b = uniform(it.b);
  it.k0 = uniform(it.k0);
  it.k1 = uniform(it.k1);
  it.pid = uniform(it.pid);
  it.q0 = uniform(it.q0);
  it.n = uniform(it.n);
  it.kv = uniform(it.kv);
  it.skip = uniform(it.skip);
  return true;
}

// The plan of a call with several requests: one workgroup cuts the requests into ranges
// and lists them by falling length (to a 256th of the longest), so that the dearest start
// first.  The order among equals is that of the atomics and decides nothing but time: a
// range's place among the partials comes from the requests alone.
constexpr int kPlanThreads = 1024, kPlanEach = 4;   // 256 threads are enough for 1024 requests

template <int kSeen>
__global__ __launch_bounds__(kPlanThreads) void paged_plan(Work w) {
  const PagedArgs& a = w.a;
  __shared__ int64_t sums[kPlanThreads / 64];
  __shared__ int offs[kPlanThreads / 64], bins[256], cursor[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x;
  int q0[kPlanEach], n[kPlanEach], kv[kPlanEach], span[kPlanEach], skip[kPlanEach], ranges[kPlanEach], len[kPlanEach];
  int64_t total = 0;
#pragma unroll
  for (int e = 0; e < kPlanEach; ++e) {
    const int b = e * threads + tid;
    q0[e] = n[e] = kv[e] = 0;
    if (b < a.B) request(a, b, q0[e], n[e], kv[e]);
    span[e] = span_of<kSeen>(a, n[e], kv[e], skip[e]);
    if (n[e] > 0) total += span[e];
  }
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  if (lane == 0) sums[wave] = total;
  if (tid < 256) bins[tid] = 0;
  __syncthreads();
  total = 0;
  for (int v = 0; v < threads / 64; ++v) total += sums[v];
  const int chunk = chunk_of(w, total);
  const float per_bin = 255.0f / (float)chunk;
  auto bin = [&](int keys) { return 255 - min(255, (int)((float)keys * per_bin)); };
  int split = 0;                                  // ranges of this thread's split requests
#pragma unroll
  for (int e = 0; e < kPlanEach; ++e) {
    ranges[e] = 0;
    if (n[e] > 0) {
      len[e] = range_len(span[e], max(1, (span[e] + chunk - 1) / chunk));
      ranges[e] = len[e] > 0 ? (span[e] + len[e] - 1) / len[e] : 1;
      if (ranges[e] > 1) {
        split += ranges[e];
        atomicAdd(&bins[bin(len[e])], ranges[e] - 1);
      }
      atomicAdd(&bins[bin(span[e] - (ranges[e] - 1) * len[e])], 1);
    }
  }
  int before = split;                             // inclusive scan over the workgroup
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(before, o);
    if (lane >= o) before += v;
  }
  if (lane == 63) offs[wave] = before;
  __syncthreads();
  for (int v = 0; v < wave; ++v) before += offs[v];
  if (wave == 0) {                                // where each length's items begin
    int c[4], sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += c[e] = bins[4 * lane + e];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(inc, o);
      if (lane >= o) inc += v;
    }
    int at = inc - sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cursor[4 * lane + e] = at;
      at += c[e];
    }
    if (lane == 63) *w.count = inc;
  }
  __syncthreads();
  int pid = before - split;
#pragma unroll
  for (int e = 0; e < kPlanEach; ++e) {
    if (n[e] == 0) continue;
    const int b = e * threads + tid, full = ranges[e] - 1;
    w.req[b] = make_int2(pid, ranges[e]);
    if (full > 0) {
      const int at = atomicAdd(&cursor[bin(len[e])], full);
      for (int r = 0; r < full; ++r)
        w.plan[at + r] = Item{b, r * len[e], (r + 1) * len[e], pid + r, q0[e], n[e], kv[e], skip[e]};
    }
    const int at = atomicAdd(&cursor[bin(span[e] - full * len[e])], 1);
    w.plan[at] = Item{b, full * len[e], span[e], full > 0 ? pid + full : -1, q0[e], n[e], kv[e], skip[e]};
    if (full > 0) pid += ranges[e];
  }
}

// What a row sees of the keys.  `lim`: keys below it (kTree: the context's end, behind which
// the row's mask counts); kRecent: `low` and up, or below the sinks.
struct Row {
  int lim, low;
  const uint32_t* mask;
};

// query token j of the item
template <int kSeen>
__device__ __forceinline__ Row row_of(const PagedArgs& a, const Item& it, int j, bool ok) {
  Row r{it.kv, 0, nullptr};
  const int place = it.kv - it.n + j;
  if constexpr (kSeen == kTree) {
    r.lim = it.kv - it.n;
    r.mask = a.mask + (size_t)(it.q0 + (ok ? j : 0)) * 4;
  } else {
    if (ok && a.causal) r.lim = place + 1;
    if constexpr (kSeen == kRecent) r.low = place - a.window + 1;
  }
  return r;
}

// bit i: the row sees the key key0 + i (key0 uniform), if it exists
template <int kSeen>
__device__ __forceinline__ uint32_t seen_of(const PagedArgs& a, const Row& r, int key0) {
  uint32_t bits = bits_below(r.lim - key0);
  if constexpr (kSeen == kRecent) bits &= ~bits_below(r.low - key0) | bits_below(a.sinks - key0);
  if constexpr (kSeen == kTree) {
    const int node = key0 - r.lim;                // of bit 0; below 0 the context
    if (node > -32 && node < 128) {
      const int w = node >> 5;                    // (-1 where the tile begins in the context)
      const uint32_t lo = w >= 0 ? r.mask[w] : 0u, hi = w < 3 ? r.mask[w + 1] : 0u;
      bits |= (uint32_t)((((uint64_t)hi << 32) | lo) >> (node & 31));
    }
  }
  return bits;
}

// Every row of query tokens j0 .. j1 sees the keys below `lim` that are not below `low`, and
// those below the sinks: tiles of such keys alone need no mask.
struct All {
  int lim, low;
};
template <int kSeen>
__device__ __forceinline__ All all_of(const PagedArgs& a, const Item& it, int j0, int j1) {
  const int place = it.kv - it.n;
  All r{it.kv, 0};
  if constexpr (kSeen == kTree) r.lim = place;
  else if (a.causal) r.lim = place + 1 + j0;
  if constexpr (kSeen == kRecent) r.low = place + j1 - a.window + 1;
  return r;
}
template <int kSeen>
__device__ __forceinline__ bool seen_whole(const PagedArgs& a, const All& r, int key0) {
  return key0 + KT <= r.lim && (kSeen != kRecent || key0 >= r.low || key0 + KT <= a.sinks);
}

// the key of the cache at place x of the span (a multiple of KT, or any within a tile that begins at one)
template <int kSeen>
__device__ __forceinline__ int key_at(const PagedArgs& a, const Item& it, int x) {
  return kSeen == kRecent && x >= a.sink_keys ? x + it.skip : x;
}

// max / sum over the four lane groups that share a row
__device__ __forceinline__ float groups_max(float v) {
  uint32_t a, b;
  rows_pair(__float_as_uint(v), a, b);
  v = fmaxf(__uint_as_float(a), __uint_as_float(b));
  halves_pair(__float_as_uint(v), a, b);
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float groups_sum(float v) {
  uint32_t a, b;
  rows_pair(__float_as_uint(v), a, b);
  v = __uint_as_float(a) + __uint_as_float(b);
  halves_pair(__float_as_uint(v), a, b);
  return __uint_as_float(a) + __uint_as_float(b);
}

// eight weights rounded to bf16, and added to the sum of the rounded and (kLse) of the unrounded
template <bool kLse>
__device__ __forceinline__ bf16x8 pack_weights(const float (&x)[8], float& l, float& lx) {
  uint32_t p[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) p[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
  l += add_bf16x2(p[1], add_bf16x2(p[0], 0.0f)) + add_bf16x2(p[3], add_bf16x2(p[2], 0.0f));
  if (kLse) lx += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  return __builtin_bit_cast(bf16x8, make_uint4(p[0], p[1], p[2], p[3]));
}

template <int HD>
struct Dims {
  static constexpr int VD = HD >= 128 ? 8 : 4;    // dims a lane loads of a value row, per group of 16 VD
  static constexpr int VU = HD / (16 * VD);       // such groups
  static constexpr int VW = VD / 2;               // their 32-bit words
};

// kSlots: pages smaller than 16, so the slot of every key is looked up by a lane of its
// own; otherwise 16 aligned keys lie in one page and the wave looks up two
template <int HD, int NW, bool kSlots, bool kLse, int kSeen>
__global__ __launch_bounds__(64 * NW) void paged_rows(Work w) {
  using D = Dims<HD>;
  constexpr int ODIM = 16 * D::VD;                // dims of one group
  const PagedArgs& a = w.a;
  __shared__ float obuf[NW][16][ODIM + 4];
  __shared__ float mbuf[NW][16], lbuf[NW][16], xbuf[NW][16];

  const int u = blockIdx.x / w.unit, kvh = blockIdx.x % w.unit;
  Item it;
  if (!find_item<kSeen>(w, u, it)) return;
  if (it.pid >= w.pid_cap) return;                // (the workspace holds every range)
  const int nq = min(it.n, a.max_q);

  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);

  // queries: the B operand of S^T, row c, dims 32 kk + 8 g ..
  const int qj = c / w.G;
  const bool ok = qj < nq;
  const Row row = row_of<kSeen>(a, it, qj, ok);
  const All all = all_of<kSeen>(a, it, 0, nq - 1);
  bf16x8 qf[HD / 32];
  {
    const uint16_t* src = a.q + (size_t)(it.q0 + (ok ? qj : 0)) * a.q_stride + (size_t)(ok ? kvh * w.G + c % w.G : 0) * HD;
#pragma unroll
    for (int kk = 0; kk < HD / 32; ++kk) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 32 * kk + 8 * g);
      qf[kk] = __builtin_bit_cast(bf16x8, ok ? v : make_uint4(0, 0, 0, 0));
    }
  }

  floatx4 o[D::VU][D::VD];
#pragma unroll
  for (int x = 0; x < D::VU; ++x)
#pragma unroll
    for (int t = 0; t < D::VD; ++t) o[x][t] = floatx4{0.f, 0.f, 0.f, 0.f};
  // m: running maximum, in units of the row's factor rc; mb: m, or 0 while the row has seen
  // nothing; lx: l of unrounded weights
  float m = -INFINITY, mb = 0.0f, l = 0.0f, lx = 0.0f, rc = w.c;

  const int32_t* table = a.page_table + (size_t)it.b * a.width;
  const int rstride = a.nkv * HD;                 // elements between slots
  const int pmask = (1 << a.page_shift) - 1;

  // where a tile lies, looked up a tile ahead (behind the last: some page of the request)
  int where[2];                                   // the pages of its halves; kSlots: of key lane % 32
  auto find = [&](int x) {
    const int key0 = key_at<kSeen>(a, it, x);
    if constexpr (kSlots) {
      where[0] = table[min(key0 + (lane & 31), it.kv - 1) >> a.page_shift];
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) where[s] = table[min(key0 + 16 * s, it.kv - 1) >> a.page_shift];
    }
  };
  if (it.k0 + KT * wave < it.k1) find(it.k0 + KT * wave);
  for (int x = it.k0 + KT * wave; x < it.k1; x += KT * NW) {
    const int key0 = key_at<kSeen>(a, it, x);
    // the tile's keys and values; a key that does not exist reads an existing row
    uint32_t held;                                // bit i: key key0 + i exists
    uint32_t kf[2][HD / 32][4], vf[D::VU][8][D::VW];
    auto key_row = [&](int s, const uint16_t* src) {
#pragma unroll
      for (int kk = 0; kk < HD / 32; ++kk)
        *reinterpret_cast<uint4*>(kf[s][kk]) = *reinterpret_cast<const uint4*>(src + 32 * kk + 8 * g);
    };
    auto value_row = [&](int j, const uint16_t* src) {
#pragma unroll
      for (int x = 0; x < D::VU; ++x)
        if constexpr (D::VD == 8)
          *reinterpret_cast<uint4*>(vf[x][j]) = *reinterpret_cast<const uint4*>(src + ODIM * x + 8 * c);
        else
          *reinterpret_cast<uint2*>(vf[x][j]) = *reinterpret_cast<const uint2*>(src + ODIM * x + 4 * c);
    };
    if constexpr (kSlots) {
      const int key = min(key0 + (lane & 31), it.kv - 1), page = where[0];
      const bool there = page >= 0 && page < a.num_pages;
      const int slot = (there ? page << a.page_shift : 0) + (key & pmask);
      held = (uint32_t)__ballot(there && key0 + (lane & 31) < it.kv);
#pragma unroll
      for (int s = 0; s < 2; ++s) key_row(s, a.k_cache + ((size_t)__shfl(slot, 16 * s + c) * rstride + kvh * HD));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        value_row(j, a.v_cache + ((size_t)__shfl(slot, 16 * (j >> 2) + 4 * g + (j & 3)) * rstride + kvh * HD));
    } else {
      held = 0;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int ks = key0 + 16 * s;
        int page = uniform(where[s]);
        int cnt = clampi(it.kv - ks, 0, 16);      // keys of this half
        if (page < 0 || page >= a.num_pages) page = cnt = 0;
        held |= ((1u << cnt) - 1u) << (16 * s);
        const size_t at = (((size_t)page << a.page_shift) + (ks & pmask)) * rstride + kvh * HD;
        const int last = max(cnt - 1, 0);
        key_row(s, a.k_cache + at + min(c, last) * rstride);
#pragma unroll
        for (int j = 0; j < 4; ++j) value_row(4 * s + j, a.v_cache + at + min(4 * g + j, last) * rstride);
      }
    }
    find(x + KT * NW);
    held = (uint32_t)uniform((int)held);
    const bool partial = uniform(held != 0xFFFFFFFFu || !seen_whole<kSeen>(a, all, key0)) != 0;

    // scores, and from them the weights: registers only
    floatx4 sc[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      sc[s] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < HD / 32; ++kk)
        sc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, *reinterpret_cast<uint4*>(kf[s][kk])), qf[kk], sc[s], 0, 0, 0);
    }
    uint32_t top = 0;                             // the largest exponent of a value, in the high half
    uint32_t sees = 0;                            // bit i: the row sees key key0 + i (set where it matters)
    if (partial) {
      sees = held & seen_of<kSeen>(a, row, key0);
      const uint32_t mine = sees >> (4 * g);
#pragma unroll
      for (int e = 0; e < 8; ++e) sc[e >> 2][e & 3] = where_bit(mine, 16 * (e >> 2) + (e & 3), sc[e >> 2][e & 3]);
#pragma unroll
      for (int y = 0; y < D::VU; ++y)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int d = 0; d < D::VW; ++d) {
            const uint32_t e = vf[y][j][d] & 0x7F807F80u;
            top = max(top, max(e, e << 16));
          }
    }
    float hi = sc[0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) hi = fmaxf(hi, sc[e >> 2][e & 3]);
    hi = groups_max(hi);
    const bool up = hi * rc > m + kRaise;
    if (uniform(__any(up))) {
      if (up) rc = row_factor(hi, w.c);
      const float mn = up ? hi * rc : m;
      const float al = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      mb = mn == -INFINITY ? 0.0f : mn;
      l *= al;
      lx *= al;
#pragma unroll
      for (int y = 0; y < D::VU; ++y)
#pragma unroll
        for (int t = 0; t < D::VD; ++t) o[y][t] *= al;
    }
    float wt[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) wt[e] = __builtin_amdgcn_exp2f(fmaf(sc[e >> 2][e & 3], rc, -mb));
    // the weights' rounding to bf16, the second product's operand type
    const bf16x8 p = pack_weights<kLse>(wt, l, lx);

    // in a tile some row does not see whole, a value that is not finite must not meet
    // that row's zero weight
    const int odd = uniform(__any(top >= 0x7F800000u));
#pragma unroll
    for (int y = 0; y < D::VU; ++y) {
#pragma unroll
      for (int t = 0; t < D::VD; ++t) {
        uint32_t vt[4];
#pragma unroll
        for (int d = 0; d < 4; ++d)
          vt[d] = __builtin_amdgcn_perm(vf[y][2 * d + 1][t >> 1], vf[y][2 * d][t >> 1], t & 1 ? 0x07060302u : 0x05040100u);
        if (!odd) {
          o[y][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, make_uint4(vt[0], vt[1], vt[2], vt[3])), p, o[y][t], 0, 0, 0);
        } else {
          // key by key, added only to the rows that see it
#pragma unroll 1
          for (int k = 0; k < KT; ++k) {
            if (!((held >> k) & 1u)) continue;
            const int j = (k & 3) | ((k >> 4) << 2);
            const uint32_t keep = g == ((k >> 2) & 3) ? (j & 1 ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
            const bf16x8 va = __builtin_bit_cast(
                bf16x8, make_uint4(j / 2 == 0 ? vt[0] & keep : 0u, j / 2 == 1 ? vt[1] & keep : 0u,
                                   j / 2 == 2 ? vt[2] & keep : 0u, j / 2 == 3 ? vt[3] & keep : 0u));
            const floatx4 add = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, p, (floatx4{0.f, 0.f, 0.f, 0.f}), 0, 0, 0);
            if ((sees >> k) & 1u) o[y][t] += add;
          }
        }
      }
    }
  }

  // join the waves, one dim group at a time
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  l = groups_sum(l);
  if (kLse) lx = groups_sum(lx);
#pragma unroll
  for (int y = 0; y < D::VU; ++y) {
    if (y) __syncthreads();
    if (g == 0 && y == 0) {
      mbuf[wave][c] = m;
      lbuf[wave][c] = l;
      if (kLse) xbuf[wave][c] = lx;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < D::VD; t += 4)
        *reinterpret_cast<floatx4*>(&obuf[wave][c][D::VD * (4 * g + i) + t]) =
            floatx4{o[y][t][i], o[y][t + 1][i], o[y][t + 2][i], o[y][t + 3][i]};
    __syncthreads();
    if (tr >= 16) continue;                       // (256 threads join)
    float mm = -INFINITY, ll = 0.0f, xx = 0.0f, f[NW], acc[D::VD];
#pragma unroll
    for (int v = 0; v < NW; ++v) mm = fmaxf(mm, mbuf[v][tr]);
    const float ms = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      f[v] = __builtin_amdgcn_exp2f(mbuf[v][tr] - ms);
      ll += lbuf[v][tr] * f[v];
      if (kLse) xx += xbuf[v][tr] * f[v];
    }
#pragma unroll
    for (int t = 0; t < D::VD; ++t) {
      acc[t] = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) acc[t] += obuf[v][tr][D::VD * tc + t] * f[v];
    }
    const int j = tr / w.G, h = kvh * w.G + tr % w.G;
    if (j >= nq) continue;
    if (it.pid < 0) {
      const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
      const size_t at = (size_t)(it.q0 + j) * a.nh + h;
      uint32_t pk[D::VW];
#pragma unroll
      for (int t = 0; t < D::VW; ++t) pk[t] = ll == 0.0f ? 0u : pack_bf16x2(acc[2 * t] * inv, acc[2 * t + 1] * inv);
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + at * HD + ODIM * y + D::VD * tc);
#pragma unroll
      for (int t = 0; t < D::VW; ++t) dst[t] = pk[t];
      if (kLse && y == 0 && tc == 0) a.lse[at] = row_lse(mm, xx, w.c);
    } else {
      const size_t at = ((size_t)it.pid * w.unit + kvh) * 16 + tr;
      float* dst = w.part_o + at * HD + ODIM * y + D::VD * tc;
#pragma unroll
      for (int t = 0; t < D::VD; t += 4)
        *reinterpret_cast<floatx4*>(dst + t) = floatx4{acc[t], acc[t + 1], acc[t + 2], acc[t + 3]};
      if (y == 0 && tc == 0) w.part_ml[at] = floatx4{mm, ll, xx, 0.0f};
    }
  }
}

// ------------------------------------------------------------------ many rows
// The same work for more than 16 rows: a wave takes 16 rows, and all waves of the
// workgroup share the keys, which pass through three LDS buffers of 32 (one worked
// on, the others filling straight from memory).  Rows lie there in 16-byte pieces permuted (piece p of
// row r at p ^ swizzle(r)) so that the K reads (16 rows, one piece) and the transposing V
// reads (rows 0..7 or rows 0..3 and 8..11, two pieces) touch every bank once.  The slots of kWindow keys (small
// pages) or groups of 16 keys are looked up ahead into LDS by the whole workgroup.  Few
// registers and 52 KB of LDS leave room for three workgroups on a compute unit, which
// cover each other's waits.  Bound by memory: 256 requests of 1..17 tokens over up to 4096
// keys, 32/8 heads of 128, pages of 64: 430 us, 5.3 TB/s; 64 blocks of 16 tokens over
// 100..4000 keys found slot by slot: 145 us, 3.9 TB/s, where the ranges end unevenly.
constexpr int kWindow = 1024;
constexpr int kStages = 3;     // LDS buffers

template <int HD>
__device__ __forceinline__ int swizzle(int r) {
  const int far = (r >> 3) & 1, mid = ((r >> 2) & 1) ^ far;
  if constexpr (HD == 64) return (mid << 2) | (r & 2) | far;
  return (mid << 3) | ((r & 3) << 1) | far;
}

template <int HD>
constexpr int shared_lds() {
  return kStages * 2 * KT * HD * 2 + kWindow * 4;
}

template <int HD, int RT, bool kSlots, bool kLse, int kSeen>
__global__ __launch_bounds__(64 * RT, HD > 128 ? RT / 4 : RT == 8 ? 4 : 3) void paged_shared(Work w) {
  constexpr int ROWB = HD * 2, TILEB = KT * ROWB, PIECES = HD / 8;
  constexpr int LOADS = 2 * TILEB / 1024;         // 1 KB loads of one tile, K then V
  constexpr int LPW = LOADS / RT;                 // of a wave
  constexpr int LR = 64 / PIECES;                 // rows of one load
  extern __shared__ __attribute__((aligned(16))) char smem[];
  int32_t* slots = reinterpret_cast<int32_t*>(smem + kStages * 2 * TILEB);
  const PagedArgs& a = w.a;
  const int u = blockIdx.x / w.unit, rest = blockIdx.x % w.unit;
  const int kvh = rest % a.nkv, rb = rest / a.nkv;
  Item it;
  if (!find_item<kSeen>(w, u, it)) return;
  const int nq = min(it.n, a.max_q), row0 = rb * 16 * RT;
  if (nq * w.G <= row0) return;                                 // (no row of this block exists)
  if (it.pid >= w.pid_cap) return;                // (the workspace holds every range)

  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const bool idle = uniform(row0 + 16 * wave >= nq * w.G) != 0;  // a wave without rows only loads
  const int r0 = row0 + 16 * wave, j = (r0 + c) / w.G, h = kvh * w.G + (r0 + c) % w.G;
  const bool ok = j < nq;
  const Row row = row_of<kSeen>(a, it, j, ok);
  const All all = all_of<kSeen>(a, it, r0 / w.G, min(nq - 1, (r0 + 15) / w.G));
  bf16x8 qf[HD / 32];
  {
    const uint16_t* src = a.q + (size_t)(it.q0 + (ok ? j : 0)) * a.q_stride + (size_t)(ok ? h : 0) * HD;
#pragma unroll
    for (int kk = 0; kk < HD / 32; ++kk) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 32 * kk + 8 * g);
      qf[kk] = __builtin_bit_cast(bf16x8, ok ? v : make_uint4(0, 0, 0, 0));
    }
  }
  floatx4 o[HD / 16];                             // dims 16 d + 4 g + i of row c
#pragma unroll
  for (int d = 0; d < HD / 16; ++d) o[d] = floatx4{0.f, 0.f, 0.f, 0.f};
  // m: running maximum, in units of the row's factor rc; mb: m, or 0 while the row has seen
  // nothing; lx: l of unrounded weights
  float m = -INFINITY, mb = 0.0f, l = 0.0f, lx = 0.0f, rc = w.c;

  const int k0 = it.k0, k1 = it.k1;
  const int32_t* table = a.page_table + (size_t)it.b * a.width;
  const int64_t rbytes = (int64_t)a.nkv * ROWB;   // bytes between slots
  const int pmask = (1 << a.page_shift) - 1;
  const char* kbase = reinterpret_cast<const char*>(a.k_cache + kvh * HD);
  const char* vbase = reinterpret_cast<const char*>(a.v_cache + kvh * HD);
  const int lrow = lane / PIECES, lslot = lane % PIECES;
  const uint32_t lds0 = lds_address(smem);

  int gaps = 0;                                   // a key of the window has no slot
  // this wave's loads of a tile: load f = q RT + wave (of K, then of V) takes LR rows
  const char* from[LPW];                          // K or V
  uint32_t to[LPW], off[LPW];                     // LDS offset in the tile; byte offset behind the 16 keys' first slot
  int half[LPW], tile_row[LPW];                   // which 16 keys; this lane's row of the tile
#pragma unroll
  for (int q = 0; q < LPW; ++q) {
    const int f = uniform(q * RT + wave), fk = f % (LOADS / 2), r = fk * LR + lrow;
    from[q] = f < LOADS / 2 ? kbase : vbase;
    to[q] = f * 1024;
    half[q] = fk * LR >> 4;
    tile_row[q] = r;
    off[q] = (uint32_t)(lslot ^ swizzle<HD>(r)) << 4;
    if (!kSlots) off[q] += (uint32_t)(r & 15) * (uint32_t)rbytes;
  }
  // Where a tile lies is read from LDS a tile ahead; a key that does not exist reads an
  // existing row.
  int slot[kSlots ? LPW : 2];                     // of this lane's rows; of the two first keys
  // (x: the tile's place in the span, win0 and win1 too)
  auto find = [&](int x, int win0, int win1) {
    if constexpr (kSlots) {
#pragma unroll
      for (int q = 0; q < LPW; ++q) slot[q] = slots[min(x + tile_row[q], win1 - 1) - win0];
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) slot[s] = slots[(min(x + 16 * s, win1 - 1) - win0) >> 4];
    }
  };
  auto issue = [&](int x, int stage) {
    const uint32_t lds = lds0 + stage * 2 * TILEB;
    if constexpr (kSlots) {
#pragma unroll
      for (int q = 0; q < LPW; ++q) load_to_lds16(from[q] + (int64_t)max(slot[q], 0) * rbytes + off[q], uniform(lds + to[q]));
    } else {
      int64_t at[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) at[s] = (int64_t)max(uniform(slot[s]), 0) * rbytes;
      const int key0 = key_at<kSeen>(a, it, x);
      const bool tail = uniform(gaps || key0 + KT > it.kv) != 0;
#pragma unroll
      for (int q = 0; q < LPW; ++q) {
        uint32_t o = off[q];
        if (tail) {
          const int first = half[q] ? uniform(slot[1]) : uniform(slot[0]), r = tile_row[q] & 15;
          o -= (uint32_t)max(r - (first < 0 ? 0 : clampi(it.kv - 1 - key0 - 16 * half[q], 0, 15)), 0) * (uint32_t)rbytes;
        }
        load_to_lds16(from[q] + (half[q] ? at[1] : at[0]), o, uniform(lds + to[q]));
      }
    }
  };

  int koff = c * ROWB + ((g ^ swizzle<HD>(c)) << 4);   // K operand (s, kk): piece 4 kk + g of row 16 s + c
  int voff[2];                                    // V operand d: keys 16 e + 4 g .. + 3, dim 16 d + c
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 16 * e + 4 * g + (c >> 2), dim = 4 * (c & 3);
    voff[e] = r * ROWB + (((dim >> 3) ^ swizzle<HD>(r)) << 4) + ((dim & 4) << 1);
  }
  union VFrag {
    shortx4 s[2];
    uint32_t w[4];
    bf16x8 v;
  };
  auto value_frag = [&](const char* vb, int d) {
    VFrag f;
#pragma unroll
    for (int e = 0; e < 2; ++e) f.s[e] = lds_read_tr(vb + (voff[e] ^ (d << 5)));
    return f;
  };

  // bit i: key x + i of the span exists
  auto held_of = [&](int x, int win0) {
    const int last = it.kv - it.skip - 1, e = min(x + (lane & 31), last) - win0;   // (of the span)
    const bool there = slots[kSlots ? e : e >> 4] >= 0 && x + (lane & 31) <= last;
    return (uint32_t)uniform((int)(uint32_t)__ballot(there));
  };
  auto scores = [&](const char* kb, floatx4 (&sc)[2]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      sc[s] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < HD / 32; ++kk) {
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(kb + ((koff ^ (kk << 6)) + 16 * s * ROWB));
        sc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[kk], sc[s], 0, 0, 0);
      }
    }
  };
  // sees: bit i: the row sees key i of the tile
  auto mask = [&](floatx4 (&sc)[2], uint32_t sees) {
    sees >>= 4 * g;
#pragma unroll
    for (int e = 0; e < 8; ++e) sc[e >> 2][e & 3] = where_bit(sees, 16 * (e >> 2) + (e & 3), sc[e >> 2][e & 3]);
  };
  // weights, rounded to bf16 (the second product's operand type), added to two sums
  auto weights = [&](const floatx4 (&sc)[2], float& sum, float& sumx) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(sc[e >> 2][e & 3], rc, -mb));
    return pack_weights<kLse>(x, sum, sumx);
  };
  auto finite = [&](const char* vb) {             // every value of the tile
    uint32_t top = 0;                             // the largest exponent, in the high half
#pragma unroll 1
    for (int q = 0; q < TILEB / 1024; ++q) {
      const uint4 v = *reinterpret_cast<const uint4*>(vb + q * 1024 + lane * 16);
      const uint32_t x[4] = {v.x & 0x7F807F80u, v.y & 0x7F807F80u, v.z & 0x7F807F80u, v.w & 0x7F807F80u};
#pragma unroll
      for (int k = 0; k < 4; ++k) top = max(top, max(x[k], x[k] << 16));
    }
    return !uniform(__any(top >= 0x7F800000u));
  };

  // In a tile that some row does not see whole, a value that is not finite must not meet
  // that row's zero weight: such a tile's values are left out here and added afterwards.
  int left_out = 0;
  auto work_on = [&](const char* kb, int x, int win0) {
    const int key0 = key_at<kSeen>(a, it, x);
    const char* vb = kb + TILEB;
    asm volatile("" : "+v"(koff), "+v"(voff[0]), "+v"(voff[1]));   // (flipped offsets are cheaper than registers)
    floatx4 sc[2];
    scores(kb, sc);
    int whole = 1;
    if (uniform(gaps || !seen_whole<kSeen>(a, all, key0))) {
      mask(sc, held_of(x, win0) & seen_of<kSeen>(a, row, key0));
      whole = uniform(finite(vb));
      left_out |= !whole;
    }
    float hi = sc[0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) hi = fmaxf(hi, sc[e >> 2][e & 3]);
    hi = groups_max(hi);
    const bool up = hi * rc > m + kRaise;
    if (uniform(__any(up))) {
      if (up) rc = row_factor(hi, w.c);
      const float mn = up ? hi * rc : m;
      const float al = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      mb = mn == -INFINITY ? 0.0f : mn;
      l *= al;
      lx *= al;
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) o[d] *= al;
    }
    const bf16x8 p = weights(sc, l, lx);
    if (uniform(whole)) {
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(value_frag(vb, d).v, p, o[d], 0, 0, 0);
    }
  };
  // a tile that was left out, key by key, added only to the rows that see it
  auto add_left_out = [&](const char* kb, int x, int win0) {
    const int key0 = key_at<kSeen>(a, it, x);
    const char* vb = kb + TILEB;
    if (!uniform(gaps || !seen_whole<kSeen>(a, all, key0)) || finite(vb)) return;
    const uint32_t held = held_of(x, win0), sees = held & seen_of<kSeen>(a, row, key0);
    floatx4 sc[2];
    float counted = 0.0f;                         // (its weights are in the sums already)
    scores(kb, sc);
    mask(sc, sees);
    const bf16x8 p = weights(sc, counted, counted);
#pragma unroll 1
    for (int k = 0; k < KT; ++k) {
      if (!((held >> k) & 1u)) continue;
      const int jj = (k & 3) | ((k >> 4) << 2);
      const uint32_t keep = g == ((k >> 2) & 3) ? (jj & 1 ? 0xFFFF0000u : 0x0000FFFFu) : 0u;
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) {
        const VFrag f = value_frag(vb, d);
        const bf16x8 va = __builtin_bit_cast(
            bf16x8, make_uint4(jj / 2 == 0 ? f.w[0] & keep : 0u, jj / 2 == 1 ? f.w[1] & keep : 0u,
                               jj / 2 == 2 ? f.w[2] & keep : 0u, jj / 2 == 3 ? f.w[3] & keep : 0u));
        const floatx4 add = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, p, (floatx4{0.f, 0.f, 0.f, 0.f}), 0, 0, 0);
        if ((sees >> k) & 1u) o[d] += add;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  constexpr int wkeys = kSlots ? kWindow : kWindow * 16;
  auto look_up = [&](int win0, int win1) {        // the slots of a window's keys
    __syncthreads();
    const int entries = kSlots ? win1 - win0 : (win1 - win0 + 15) >> 4;
    int missing = 0;
    for (int e = threadIdx.x; e < entries; e += 64 * RT) {
      const int key = key_at<kSeen>(a, it, win0 + (kSlots ? e : e << 4));
      const int page = table[key >> a.page_shift];
      const int slot = page >= 0 && page < a.num_pages ? (page << a.page_shift) + (key & pmask) : -1;
      slots[e] = slot;
      // (a window's first tile and the sinks' last may hold keys that no row sees: masked as such)
      missing |= slot < 0 && (kSeen != kRecent || key < a.sinks || key + (kSlots ? 0 : 15) > it.kv - it.n - a.window);
    }
    gaps = uniform(__syncthreads_or(missing));
  };
  // every tile of the range, loaded kStages - 1 tiles ahead
  auto walk = [&](auto on_tile) {
    for (int win0 = k0; win0 < k1; win0 += wkeys) {
      const int win1 = min(k1, win0 + wkeys);
      look_up(win0, win1);
#pragma unroll 1
      for (int s = 0; s < kStages - 1 && win0 + s * KT < win1; ++s) {
        find(win0 + s * KT, win0, win1);
        issue(win0 + s * KT, s);
      }
      find(win0 + (kStages - 1) * KT, win0, win1);
      int stage = 0;
      for (int x = win0; x < win1; x += KT) {
        // this wave's loads of the tile have landed; after the barrier everyone's have, and
        // everyone is done with the tile before
        const int ahead = win1 - x - 1;           // / KT: younger tiles on their way, at most kStages - 2
        if (uniform(ahead >= (kStages - 2) * KT)) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 2) * LPW) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_barrier();
        if (uniform(ahead >= (kStages - 1) * KT)) {
          issue(x + (kStages - 1) * KT, stage == 0 ? kStages - 1 : stage - 1);
          find(x + kStages * KT, win0, win1);
        }
        on_tile(smem + stage * 2 * TILEB, x, win0);
        stage = stage == kStages - 1 ? 0 : stage + 1;
      }
    }
  };
  if (idle) walk([](const char*, int, int) {});
  else walk(work_on);
  int* const again = slots;                       // (free: a window is looked up anew)
  __syncthreads();
  if (threadIdx.x == 0) *again = 0;
  __syncthreads();
  if (left_out && lane == 0) *again = 1;
  __syncthreads();
  if (uniform(*again)) {
    __syncthreads();
    if (idle) walk([](const char*, int, int) {});
    else walk(add_left_out);
  }

  l = groups_sum(l);
  if (kLse) lx = groups_sum(lx);
  if (idle || !ok) return;
  if (it.pid < 0) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const size_t at = (size_t)(it.q0 + j) * a.nh + h;
#pragma unroll
    for (int d = 0; d < HD / 16; ++d)
      *reinterpret_cast<uint2*>(a.out + at * HD + 16 * d + 4 * g) =
          l == 0.0f ? make_uint2(0u, 0u)
                    : make_uint2(pack_bf16x2(o[d][0] * inv, o[d][1] * inv), pack_bf16x2(o[d][2] * inv, o[d][3] * inv));
    if (kLse && g == 0) a.lse[at] = row_lse(m, lx, w.c);
  } else {
    const size_t at = ((size_t)it.pid * w.unit + rest) * (16 * RT) + 16 * wave + c;
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) *reinterpret_cast<floatx4*>(w.part_o + at * HD + 16 * d + 4 * g) = o[d];
    if (g == 0) w.part_ml[at] = floatx4{m, l, lx, 0.0f};
  }
}

// ------------------------------------------------------------------ large trees, long contexts
// The same work where it is the products that bound it: a wave takes 32 rows
// (v_mfma_f32_32x32x16_bf16; lane (h, n) = (lane / 32, lane % 32) holds row n and the keys
// 8 (i / 4) + 4 h + i % 4 of each 32), a workgroup 256, so that one reading of the cache serves
// a tree of 64 nodes with four heads on a kv head.  Tiles are of 64 keys.  A wave holds the weights
// of one tile and the scores of the next at once, so that the first product of the next tile runs
// beside the exponentials of this one.  K is read one tile ahead of V; four LDS buffers of K and
// three of V are filled straight from memory, two tiles ahead of their use.  The tiles of the
// context, which every row sees whole, come first; the tree's own, masked, last.
// 64 trees of 64 nodes over 4096 keys each, 32/8 heads of 128: 350 us, 0.77 PFLOP/s, 485 by shared
// tiles; the matrix units are busy 0.39 of the time, a third of the waves' goes by at barriers
// and loads, 0.30 waiting for the product before.  Smaller trees leave waves idle: of 64 trees of 9
// to 64 nodes over up to 8192 keys (291 us) 39% of the waves' tiles are only loaded.
template <int HD>
__device__ __forceinline__ int swizzle32(int r) {
  if constexpr (HD == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  return ((r & 3) << 2) | ((r >> 2) & 3);
}

__device__ __forceinline__ float halves_sum(float v) {
  uint32_t lo, hi;
  halves_pair(__float_as_uint(v), lo, hi);
  return __uint_as_float(lo) + __uint_as_float(hi);
}

constexpr int kWideWaves = 8, kWideTile = 64;
template <int HD>
constexpr int wide_lds() { return 7 * kWideTile * HD * 2 + kWindow * 4; }

template <int HD, bool kSlots, bool kLse>
__global__ __launch_bounds__(64 * kWideWaves, 2) void paged_wide(Work w) {
  constexpr int NW = kWideWaves, WT = kWideTile, SB = WT / 32, UG = WT / 16, kWideRows = 32 * NW;
  constexpr int ROWB = HD * 2, TILEB = WT * ROWB, PIECES = HD / 8;
  constexpr int LOADS = TILEB / 1024 / NW;        // 1 KB loads of a wave for one tile of K (or V)
  constexpr int LR = 64 / PIECES;                 // rows of one load
  extern __shared__ __attribute__((aligned(16))) char smem[];   // four K tiles, three V tiles, slots
  int32_t* slots = reinterpret_cast<int32_t*>(smem + 7 * TILEB);
  const PagedArgs& a = w.a;
  const int u = blockIdx.x / w.unit, rest = blockIdx.x % w.unit;
  const int kvh = rest % a.nkv, rb = rest / a.nkv;
  Item it;
  if (!find_item<kTree>(w, u, it)) return;
  const int nq = min(it.n, a.max_q), row0 = rb * kWideRows;
  if (nq * w.G <= row0) return;                   // (no row of this block exists)
  if (it.pid >= w.pid_cap) return;                // (the workspace holds every range)

  const int lane = threadIdx.x & 63, col = lane & 31, hh = lane >> 5;
  const int wave = uniform(threadIdx.x >> 6);
  const int r0 = row0 + 32 * wave, j = (r0 + col) / w.G, h = kvh * w.G + (r0 + col) % w.G;
  const bool idle = uniform(r0 >= nq * w.G) != 0;  // a wave without rows only loads
  const bool ok = j < nq;
  const Row row = row_of<kTree>(a, it, j, ok);
  const int ctx = it.kv - it.n;
  bf16x8 qf[HD / 16];
  {
    const uint16_t* src = a.q + (size_t)(it.q0 + (ok ? j : 0)) * a.q_stride + (size_t)(ok ? h : 0) * HD;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 16 * kk + 8 * hh);
      qf[kk] = __builtin_bit_cast(bf16x8, ok ? v : make_uint4(0, 0, 0, 0));
    }
  }
  floatx16 o[HD / 32];                            // dims 32 d + 8 (i / 4) + 4 h + i % 4 of row n
#pragma unroll
  for (int d = 0; d < HD / 32; ++d) o[d] = floatx16{};
  // m: running maximum, in units of the row's factor rc; mb: m, or 0 while the row has seen
  // nothing; lx: l of unrounded weights
  float m = -INFINITY, mb = 0.0f, l = 0.0f, lx = 0.0f, rc = w.c;

  const int32_t* table = a.page_table + (size_t)it.b * a.width;
  const int64_t rbytes = (int64_t)a.nkv * ROWB;   // bytes between slots
  const int pmask = (1 << a.page_shift) - 1;
  const char* kbase = reinterpret_cast<const char*>(a.k_cache + kvh * HD);
  const char* vbase = reinterpret_cast<const char*>(a.v_cache + kvh * HD);
  const uint32_t lds0 = lds_address(smem);
  int gaps = 0;                                   // a key of the window has no slot

  // This wave's loads of a tile: load q takes LR rows of one group of 16.  Where the rows of a
  // tile lie is found once, for K; V's loads of that tile follow a tile later.
  uint32_t off[LOADS];                            // byte offset behind the group's first slot
  int group[LOADS], tile_row[LOADS];
#pragma unroll
  for (int q = 0; q < LOADS; ++q) {
    const int f = uniform(q * NW + wave), r = f * LR + lane / PIECES;
    group[q] = f * LR >> 4;
    tile_row[q] = r;
    off[q] = (uint32_t)(lane % PIECES ^ swizzle32<HD>(r)) << 4;
    if (!kSlots) off[q] += (uint32_t)(r & 15) * (uint32_t)rbytes;
  }
  struct Place {
    int slot[LOADS];                              // the group's first (kSlots: a lane's own row's), or below 0
  };
  auto find = [&](int key0, int win0, int win1) {  // (read a while before it is settled)
    Place p;
#pragma unroll
    for (int q = 0; q < LOADS; ++q)
      p.slot[q] = kSlots ? slots[min(key0 + tile_row[q], win1 - 1) - win0] : slots[(min(key0 + 16 * group[q], win1 - 1) - win0) >> 4];
    return p;
  };
  auto settle = [&](Place p) {
#pragma unroll
    for (int q = 0; q < LOADS; ++q)
      if (!kSlots) p.slot[q] = uniform(p.slot[q]);
    return p;
  };
  auto issue = [&](const char* base, const Place& p, int q, int key0, uint32_t tile) {
    const uint32_t lds = uniform(tile + (q * NW + wave) * 1024);
    const char* at = base + (int64_t)max(p.slot[q], 0) * rbytes;
    uint32_t o = off[q];
    if constexpr (kSlots) {
      load_to_lds16(at + o, lds);
    } else {
      if (uniform(gaps || key0 + WT > it.kv)) {   // a key that does not exist reads an existing row
        const int r = tile_row[q] & 15;
        o -= (uint32_t)max(r - (p.slot[q] < 0 ? 0 : clampi(it.kv - 1 - key0 - 16 * group[q], 0, 15)), 0) * (uint32_t)rbytes;
      }
      load_to_lds16(at, o, lds);
    }
  };
  auto kbuf_of = [&](int t) { return (t & 3) * TILEB; };
  auto vbuf_of = [&](int t) { return (4 + t % 3) * TILEB; };

  int koff = col * ROWB + ((hh ^ swizzle32<HD>(col)) << 4);   // K operand kk of 32 rows: this lane's row, piece 2 kk + hh
  int voff[2];                                    // V operand (u, d): keys 16 u + 8 e + 4 hh .. + 3, dim 32 d + col
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 8 * e + 4 * hh + ((lane & 15) >> 2), dim = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    voff[e] = r * ROWB + (((dim >> 3) ^ swizzle32<HD>(r)) << 4) + ((dim & 4) << 1);
  }
  union VFrag {
    shortx4 s[2];
    uint32_t w[4];
    bf16x8 v;
  };
  auto key_frag = [&](const char* kb, int s, int kk) {
    return *reinterpret_cast<const bf16x8*>(kb + ((koff ^ (kk << 5)) + 32 * s * ROWB));
  };
  auto value_frag = [&](const char* vb, int u, int d) {
    VFrag f;
#pragma unroll
    for (int e = 0; e < 2; ++e) f.s[e] = lds_read_tr(vb + ((voff[e] ^ (d << 6)) + 16 * u * ROWB));
    return f;
  };
  auto scores = [&](floatx16 (&sc)[SB], const char* kb) {
#pragma unroll
    for (int s = 0; s < SB; ++s) {
      sc[s] = floatx16{};
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        sc[s] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_frag(kb, s, kk), qf[kk], sc[s], 0, 0, 0);
    }
  };
  auto row_max = [&](const floatx16 (&sc)[SB]) {
    float top = sc[0][0];
#pragma unroll
    for (int s = 0; s < SB; ++s)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[s][e]);
    uint32_t lo, hi;
    halves_pair(__float_as_uint(top), lo, hi);
    return fmaxf(__uint_as_float(lo), __uint_as_float(hi));
  };
  // raise the maxima that the scores exceed by too much
  auto raise = [&](float top) {
    const bool up = top * rc > m + kRaise;
    if (uniform(__any(up))) {
      if (up) rc = row_factor(top, w.c);
      const float mn = up ? top * rc : m;
      const float al = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      mb = mn == -INFINITY ? 0.0f : mn;
      l *= al;
      lx *= al;
#pragma unroll
      for (int d = 0; d < HD / 32; ++d) o[d] *= al;
    }
  };
  // weights of keys 16 u + 8 half .. of the tile, rounded to bf16 (the second product's operand
  // type), and their sums
  auto weights = [&](const floatx16 (&sc)[SB], int u, int half, uint32_t (&p)[4]) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(sc[u >> 1][8 * (u & 1) + 4 * half + e], rc, -mb));
    if (kLse) lx += (x[0] + x[1]) + (x[2] + x[3]);
    p[2 * half] = pack_bf16x2(x[0], x[1]);
    p[2 * half + 1] = pack_bf16x2(x[2], x[3]);
    l = add_bf16x2(p[2 * half + 1], add_bf16x2(p[2 * half], l));
    asm volatile("" : "+v"(p[2 * half]), "+v"(p[2 * half + 1]));
  };
  auto as_frag = [](const uint32_t (&p)[4]) { return __builtin_bit_cast(bf16x8, make_uint4(p[0], p[1], p[2], p[3])); };

  constexpr int wkeys = kSlots ? kWindow : kWindow * 16;
  for (int win0 = it.k0; win0 < it.k1; win0 += wkeys) {
    const int win1 = min(it.k1, win0 + wkeys);
    __syncthreads();
    {
      const int entries = kSlots ? win1 - win0 : (win1 - win0 + 15) >> 4;
      int missing = 0;
      for (int e = threadIdx.x; e < entries; e += 64 * NW) {
        const int key = win0 + (kSlots ? e : e << 4), page = table[key >> a.page_shift];
        const int slot = page >= 0 && page < a.num_pages ? (page << a.page_shift) + (key & pmask) : -1;
        slots[e] = slot;
        missing |= slot < 0;
      }
      gaps = uniform(__syncthreads_or(missing));
    }
    const int nt = (win1 - win0 + WT - 1) / WT;
    const int nfull = gaps ? 0 : clampi((min(win1, ctx) - win0) / WT, 0, nt);
    int t = 0;
    // At tile t the loads of K t + 3 and V t + 2 are issued; those of the tile before may be on
    // their way, older ones (K t + 1 and V t, and all before) have landed, everyone's after the
    // barrier, and everyone is done with the tile before.
    auto open_tile = [&]() {
      if (uniform(t + 2 < nt)) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * LOADS) : "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      lds_barrier();
    };
    Place next, last;                             // of K t + 3, of V t + 2
    {
      const Place p0 = settle(find(win0, win0, win1)), p1 = settle(find(win0 + WT, win0, win1));
      next = settle(find(win0 + 2 * WT, win0, win1));
#pragma unroll
      for (int q = 0; q < LOADS; ++q) issue(kbase, p0, q, win0 + 0 * WT, lds0 + kbuf_of(0));
#pragma unroll
      for (int q = 0; q < LOADS; ++q)
        if (nt > 1) issue(kbase, p1, q, win0 + 1 * WT, lds0 + kbuf_of(1));
#pragma unroll
      for (int q = 0; q < LOADS; ++q) issue(vbase, p0, q, win0 + 0 * WT, lds0 + vbuf_of(0));
#pragma unroll
      for (int q = 0; q < LOADS; ++q)
        if (nt > 2) issue(kbase, next, q, win0 + 2 * WT, lds0 + kbuf_of(2));
#pragma unroll
      for (int q = 0; q < LOADS; ++q)
        if (nt > 1) issue(vbase, p1, q, win0 + 1 * WT, lds0 + vbuf_of(1));
      last = next;
      next = settle(find(win0 + 3 * WT, win0, win1));
    }
    auto issue_k = [&](int q) {
      if (uniform(t + 3 < nt)) issue(kbase, next, q, win0 + (t + 3) * WT, lds0 + kbuf_of(t + 3));
    };
    auto issue_v = [&](int q) {
      if (uniform(t + 2 < nt)) issue(vbase, last, q, win0 + (t + 2) * WT, lds0 + vbuf_of(t + 2));
    };
    auto advance = [&](const Place& found) {
      ++t;
      last = next;
      next = settle(found);
    };
    auto find_next = [&]() { return find(win0 + (t + 4) * WT, win0, win1); };

    // tiles that every row sees whole: cur holds tile t's scores, nxt takes the next tile's (of no
    // use after the last)
    constexpr int KG = SB * (HD / 16) / 4, VG = HD / 32;
    auto step = [&](floatx16 (&cur)[SB], floatx16 (&nxt)[SB]) {
      open_tile();
      const Place found = find_next();
      asm volatile("" : "+v"(koff), "+v"(voff[0]), "+v"(voff[1]));   // (flipped offsets are cheaper than registers)
      const char* kb = smem + kbuf_of(t + 1);
      const char* vb = smem + vbuf_of(t);
      bf16x8 kf[2][KG];
      uint32_t p[UG][4];
      VFrag vf[2][VG];
#pragma unroll
      for (int i = 0; i < KG; ++i) kf[0][i] = key_frag(kb, i % SB, i / SB);
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) {
        if (gq < 3) {
#pragma unroll
          for (int i = 0; i < KG; ++i) {
            const int f = (gq + 1) * KG + i;
            kf[(gq + 1) & 1][i] = key_frag(kb, f % SB, f / SB);
          }
        } else {
#pragma unroll
          for (int i = 0; i < VG; ++i) vf[0][i] = value_frag(vb, 0, i);
        }
        if (gq == 0)
#pragma unroll
          for (int s = 0; s < SB; ++s) nxt[s] = floatx16{};
        weights(cur, gq >> 1, gq & 1, p[gq >> 1]);
#pragma unroll
        for (int i = 0; i < KG; ++i) {
          const int f = gq * KG + i;
          nxt[f % SB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[gq & 1][i], qf[f / SB], nxt[f % SB], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
          if (q * 4 / LOADS == gq) issue_k(q);
      }
      float tm = 0.0f;
#pragma unroll
      for (int u = 0; u < UG; ++u) {
        if (u < UG - 1)
#pragma unroll
          for (int i = 0; i < VG; ++i) vf[(u + 1) & 1][i] = value_frag(vb, u + 1, i);
        if (UG > 2 && u == 0) {
          weights(cur, 2, 0, p[2]);
          weights(cur, 2, 1, p[2]);
        } else if (UG > 2 && u < 3) {
          weights(cur, 3, u - 1, p[3]);
        }
        if (u == UG - 1) tm = row_max(nxt);
#pragma unroll
        for (int i = 0; i < VG; ++i)
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[u & 1][i].v, as_frag(p[u]), o[i], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
          if (q * UG / LOADS == u) issue_v(q);
      }
      advance(found);
      if (uniform(t < nfull)) raise(tm);          // (the scores of a tile seen in part are formed again, masked)
    };
    auto only_load = [&]() {
      open_tile();
      const Place found = find_next();
#pragma unroll
      for (int q = 0; q < LOADS; ++q) {
        issue_k(q);
        issue_v(q);
      }
      advance(found);
    };
    if (idle) {
      if (nfull > 0) open_tile();
      while (t < nt) only_load();
      continue;
    }
    floatx16 sa[SB];
    if (uniform(nfull > 0)) {
      floatx16 sb[SB];
      open_tile();
      scores(sa, smem + kbuf_of(0));
      raise(row_max(sa));
      while (true) {
        step(sa, sb);
        if (uniform(t >= nfull)) break;
        step(sb, sa);
        if (uniform(t >= nfull)) break;
      }
    }
    // the others, one product after the other
    while (t < nt) {
      const int key0 = win0 + t * WT;
      const char* kb = smem + kbuf_of(t);
      const char* vb = smem + vbuf_of(t);
      open_tile();
      const Place found = find_next();
#pragma unroll
      for (int q = 0; q < LOADS; ++q) {
        issue_k(q);
        issue_v(q);
      }
      scores(sa, kb);
      uint32_t held[SB], sees[SB];                // bit i of block s: key 32 s + i exists, the row sees it
#pragma unroll
      for (int s = 0; s < SB; ++s) {
        const int x = key0 + 32 * s, e = max(min(x + (lane & 31), it.kv - 1) - win0, 0);
        const bool there = x + (lane & 31) < it.kv && slots[kSlots ? e : e >> 4] >= 0;
        held[s] = (uint32_t)uniform((int)(uint32_t)__ballot(there));
        sees[s] = held[s] & seen_of<kTree>(a, row, x);
        const uint32_t mine = sees[s] >> (4 * hh);
#pragma unroll
        for (int e = 0; e < 16; ++e) sa[s][e] = where_bit(mine, 8 * (e >> 2) + (e & 3), sa[s][e]);
      }
      raise(row_max(sa));
#pragma unroll
      for (int u = 0; u < UG; ++u) {
        const uint32_t hold = held[u >> 1] >> (16 * (u & 1)), see = sees[u >> 1] >> (16 * (u & 1));
        if (!uniform((int)(hold & 0xFFFFu))) continue;
        VFrag f[VG];
        uint32_t pw[4], top = 0;                  // top: the largest exponent, in the high half
        weights(sa, u, 0, pw);
        weights(sa, u, 1, pw);
        const bf16x8 p = as_frag(pw);
#pragma unroll
        for (int d = 0; d < VG; ++d) f[d] = value_frag(vb, u, d);
        // a value that is not finite must not meet the zero weight of a row that does not see it
#pragma unroll
        for (int d = 0; d < VG; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t e = f[d].w[k] & 0x7F807F80u;
            top = max(top, max(e, e << 16));
          }
        if (!uniform(__any(top >= 0x7F800000u))) {
#pragma unroll
          for (int d = 0; d < VG; ++d) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[d].v, p, o[d], 0, 0, 0);
        } else {
          // key by key, added only to the rows that see it
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {
            if (!((hold >> k) & 1u)) continue;
            const int jj = (k & 3) | ((k >> 3) << 2);
            const uint32_t half = jj & 1 ? 0xFFFF0000u : 0x0000FFFFu;
            const uint32_t keep = hh == ((k >> 2) & 1) ? half : 0u;
#pragma unroll
            for (int d = 0; d < VG; ++d) {
              const bf16x8 one = __builtin_bit_cast(
                  bf16x8, make_uint4(jj / 2 == 0 ? f[d].w[0] & keep : 0u, jj / 2 == 1 ? f[d].w[1] & keep : 0u,
                                     jj / 2 == 2 ? f[d].w[2] & keep : 0u, jj / 2 == 3 ? f[d].w[3] & keep : 0u));
              const floatx16 add = __builtin_amdgcn_mfma_f32_32x32x16_bf16(one, p, floatx16{}, 0, 0, 0);
              if ((see >> k) & 1u) o[d] += add;
            }
          }
        }
      }
      advance(found);
    }
  }

  l = halves_sum(l);
  if (kLse) lx = halves_sum(lx);
  if (idle || !ok) return;
  if (it.pid < 0) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const size_t at = (size_t)(it.q0 + j) * a.nh + h;
#pragma unroll
    for (int d = 0; d < HD / 32; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint2*>(a.out + at * HD + 32 * d + 8 * q + 4 * hh) =
            l == 0.0f ? make_uint2(0u, 0u)
                      : make_uint2(pack_bf16x2(o[d][4 * q] * inv, o[d][4 * q + 1] * inv),
                                   pack_bf16x2(o[d][4 * q + 2] * inv, o[d][4 * q + 3] * inv));
    if (kLse && hh == 0) a.lse[at] = row_lse(m, lx, w.c);
  } else {
    const size_t at = ((size_t)it.pid * w.unit + rest) * kWideRows + 32 * wave + col;
#pragma unroll
    for (int d = 0; d < HD / 32; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<floatx4*>(w.part_o + at * HD + 32 * d + 8 * q + 4 * hh) =
            floatx4{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
    if (hh == 0) w.part_ml[at] = floatx4{m, l, lx, 0.0f};
  }
}

// The ranges of split requests, joined in their order.  A workgroup takes `step` rows of one
// (request, row block, kv head); hd / 4 threads take a row, four dims each.  Up to kFew
// ranges they do so alone, every row of the workgroup at once; of more ranges the
// 256 / (hd / 4) groups take every so many each, row after row, and LDS joins the groups.
constexpr int kFew = 16;

struct Joined {
  float m, l, lx;
  floatx4 acc;
};

// ranges first, first + hop, .. of row at0 (partials `stride` rows apart)
__device__ __forceinline__ Joined join_ranges(const Work& w, size_t at0, size_t stride, int ns, int first, int hop, int hd, int d) {
  Joined t{-INFINITY, 0.0f, 0.0f, floatx4{0.f, 0.f, 0.f, 0.f}};
  for (int s0 = first; s0 < ns; s0 += 4 * hop) {
    floatx4 ml[4], v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int s = s0 + q * hop;
      const size_t at = at0 + (size_t)min(s, ns - 1) * stride;
      ml[q] = w.part_ml[at];
      v[q] = *reinterpret_cast<const floatx4*>(w.part_o + at * hd + 4 * d);
      if (s >= ns) ml[q][0] = -INFINITY;
    }
    float mn = t.m;
#pragma unroll
    for (int q = 0; q < 4; ++q) mn = fmaxf(mn, ml[q][0]);
    const float ms = mn == -INFINITY ? 0.0f : mn;
    const float f0 = __builtin_amdgcn_exp2f(t.m - ms);
    t.l *= f0;
    t.lx *= f0;
    t.acc *= f0;
    t.m = mn;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float f = __builtin_amdgcn_exp2f(ml[q][0] - ms);
      if (s0 + q * hop < ns) {                    // (a range of weight 0 too: its sums may be NaN)
        t.l += ml[q][1] * f;
        t.lx += ml[q][2] * f;
        t.acc += v[q] * f;
      }
    }
  }
  return t;
}

template <int HD, int RT>
__global__ __launch_bounds__(256) void paged_join(Work w, int step) {
  const PagedArgs& a = w.a;
  const int b = blockIdx.x / w.unit, rest = blockIdx.x % w.unit;
  const int kvh = rest % a.nkv, rb = rest / a.nkv;
  int q0, n, kv;
  request(a, b, q0, n, kv);
  const int rows = min(16 * RT, min(n, a.max_q) * w.G - rb * 16 * RT), first = blockIdx.y * step;
  if (first >= rows) return;
  const int2 rq = w.req[b];
  if (rq.y <= 1) return;
  const int ns = min(rq.y, w.pid_cap - rq.x), last = min(rows, first + step);
  constexpr int TPR = HD / 4, GR = 256 / TPR;
  __shared__ floatx4 part[GR][TPR];
  __shared__ float gm[GR], gl[GR], gx[GR];
  const int d = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const size_t stride = (size_t)w.unit * (16 * RT), base = ((size_t)rq.x * w.unit + rest) * (16 * RT);
  auto finish = [&](int r, const Joined& t) {
    const int R = rb * 16 * RT + r;
    const size_t at = (size_t)(q0 + R / w.G) * a.nh + kvh * w.G + R % w.G;
    const float inv = t.l == 0.0f ? 0.0f : 1.0f / t.l;
    uint2 pk = make_uint2(0u, 0u);
    if (t.l != 0.0f) pk = make_uint2(pack_bf16x2(t.acc[0] * inv, t.acc[1] * inv), pack_bf16x2(t.acc[2] * inv, t.acc[3] * inv));
    *reinterpret_cast<uint2*>(a.out + at * HD + 4 * d) = pk;
    if (a.lse && d == 0) a.lse[at] = row_lse(t.m, t.lx, w.c);
  };
  if (ns <= kFew) {
    for (int r = first + grp; r < last; r += GR) finish(r, join_ranges(w, base + r, stride, ns, 0, 1, HD, d));
    return;
  }
  for (int r = first; r < last; ++r) {
    Joined t = join_ranges(w, base + r, stride, ns, grp, GR, HD, d);
    __syncthreads();
    part[grp][d] = t.acc;
    if (d == 0) {
      gm[grp] = t.m;
      gl[grp] = t.l;
      gx[grp] = t.lx;
    }
    __syncthreads();
    if (grp == 0) {
      t.m = -INFINITY;
#pragma unroll
      for (int q = 0; q < GR; ++q) t.m = fmaxf(t.m, gm[q]);
      const float ms = t.m == -INFINITY ? 0.0f : t.m;
      t.l = t.lx = 0.0f;
      t.acc = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const float f = __builtin_amdgcn_exp2f(gm[q] - ms);
        t.l += gl[q] * f;
        t.lx += gx[q] * f;
        t.acc += part[q][d] * f;
      }
      finish(r, t);
    }
  }
}

struct Shape {
  bool wide;
  int RT, RB, G, unit, target, min_chunk, whole, pid_cap;
  size_t off_o, off_ml, off_req, off_plan, off_count, bytes;
};

template <int kSeen>
Shape shape_of(int B, int max_q, int nh, int nkv, int hd, int64_t keys) {
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  Shape s;
  s.G = nh / nkv;
  const int rows = max_q * s.G;
  // Waves of 16 rows a workgroup: 64 requests over 100..4000 keys, 32/8 heads of 128, take
  // 114 us with 4 rows by paged_rows and 126 by shared tiles, 118 and 130 with 16; 20 rows
  // 130 us with four waves (two of them only load) and 131 with two, 40 rows 135 with four
  // and 144 with eight, 68 rows 166 with eight and 190 with four.
  s.RT = rows <= 16 ? 1 : rows <= 64 ? 4 : 8;
  // Large trees: workgroups of 256 rows (paged_wide) where there may be 2048 keys for every
  // compute unit.  They take longer to start and to end, and go faster in between.  Against shared
  // tiles, 32/8 heads of 128, in us in a captured graph: trees of 64 nodes, 64 requests of 4096 keys
  // 350 and 485, of 2048 205 and 244, of 1024 137 and 136; one request of 65536 keys 111 and 129.
  // Trees of 32 nodes (128 rows) gained 6% at most by them.  Heads of 256 leave no registers.
  // The host knows what the tables have room for, not the lengths: short contexts under wide tables
  // pay.  64 requests of 512 keys under a table of 32768, 105 and 86 us, one of 8192 keys under one of
  // 131072, 52 and 39, one of 613 33 and 21.
  s.wide = kSeen == kTree && hd <= 128 && rows > 128 && keys * nkv >= (int64_t)2048 * kCus;
  if (s.wide) s.RT = 16;
  s.RB = (rows + 16 * s.RT - 1) / (16 * s.RT);
  s.unit = nkv * s.RB;
  // items aimed at: two workgroups on each compute unit (one with heads of 256) draw all
  // that memory gives, and shorter ranges cost more in starting and joining than they
  // even out: 64 blocks of 16 x 4 rows over 100..4000 keys take 145 us so, 150 at twice
  // and 163 us at four times as many; one token over 131071 keys 104, 110 and 118 us
  s.target = kCus * (hd > 128 ? 1 : 2);
  if (s.wide) s.target = kCus;                    // (twice as many: 345 us for the 64 ragged trees' 291)
  // A shorter range costs more to start and join than it takes.  A tile of 32 keys takes a
  // workgroup of shared tiles about 0.9 us alone, four tiles the waves of paged_rows; the
  // joining pass, about 5 us.  Calls that leave most of the card idle cut finer: 9 tokens
  // over 512 keys of one request 11 us so and 18 us whole, of 64 requests 38 and 32 us.
  s.min_chunk = s.RT == 1 ? 512 : B * s.unit <= kCus / 4 ? 128 : 256;
  s.whole = 2 * s.min_chunk;
  // a split request has more keys than a range, so its ranges are fewer than twice its
  // keys over the range's length, and all of them together at most 2 target / unit
  s.pid_cap = 2 * (s.target / s.unit + 1) + 1;
  s.off_req = 0;
  s.off_count = al((size_t)B * sizeof(int2));
  s.off_plan = s.off_count + 256;
  s.off_ml = s.off_plan + al(((size_t)s.target / s.unit + B + 2) * sizeof(Item));
  s.off_o = s.off_ml + al((size_t)s.pid_cap * s.unit * 16 * s.RT * sizeof(floatx4));
  s.bytes = s.off_o + al((size_t)s.pid_cap * s.unit * 16 * s.RT * hd * sizeof(float));
  return s;
}

template <int HD, int RT, bool kWide, bool kSlots, bool kLse, int kSeen>
hipError_t launch_rows(const Work& w, int grid, hipStream_t stream) {
  if constexpr (kWide) {
    static_assert(kSeen == kTree, "the only rule whose keys are seen whole from the first on");
    static_assert(16 * RT == 32 * kWideWaves, "rows of a block");
    constexpr int lds = wide_lds<HD>();
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&paged_wide<HD, kSlots, kLse>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((paged_wide<HD, kSlots, kLse>), dim3(grid), dim3(64 * kWideWaves), lds, stream, w);
  } else if constexpr (RT > 1) {
    constexpr int lds = shared_lds<HD>();
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&paged_shared<HD, RT, kSlots, kLse, kSeen>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((paged_shared<HD, RT, kSlots, kLse, kSeen>), dim3(grid), dim3(64 * RT), lds, stream, w);
  } else {
    // Eight waves where no compute unit gets a second workgroup: one token over 517 keys, 32/8
    // heads of 128, 9.2 us with eight and 10.2 with four, 32 of them 13.6 and 15.4.  Heads of 256
    // leave registers for four.
    constexpr int most = HD > 128 ? 4 : 8;
    if (grid <= kCus) hipLaunchKernelGGL((paged_rows<HD, most, kSlots, kLse, kSeen>), dim3(grid), dim3(64 * most), 0, stream, w);
    else hipLaunchKernelGGL((paged_rows<HD, 4, kSlots, kLse, kSeen>), dim3(grid), dim3(64 * 4), 0, stream, w);
  }
  return hipGetLastError();
}

template <int HD, int RT, bool kWide, int kSeen>
hipError_t launch(const Work& w, int grid, hipStream_t stream) {
  const bool slots = w.a.page_shift < 4, lse = w.a.lse != nullptr;
  const hipError_t e = slots ? lse ? launch_rows<HD, RT, kWide, true, true, kSeen>(w, grid, stream) : launch_rows<HD, RT, kWide, true, false, kSeen>(w, grid, stream)
                       : lse ? launch_rows<HD, RT, kWide, false, true, kSeen>(w, grid, stream)
                             : launch_rows<HD, RT, kWide, false, false, kSeen>(w, grid, stream);
  if (e != hipSuccess || !w.cut) return e;
  const int rows = std::min(16 * RT, w.a.max_q * w.G);
  const int step = std::max(1, std::min(rows, (int)((int64_t)w.a.B * w.unit * rows / kJoinGroups)));
  hipLaunchKernelGGL((paged_join<HD, RT>), dim3(w.a.B * w.unit, (rows + step - 1) / step), dim3(256), 0, stream, w, step);
  return hipGetLastError();
}

template <int HD, int kSeen>
hipError_t launch_rt(const Work& w, const Shape& s, int grid, hipStream_t stream) {
  if constexpr (kSeen == kTree && HD <= 128)
    if (s.wide) return launch<HD, 16, true, kSeen>(w, grid, stream);
  switch (s.RT) {
    case 1: return launch<HD, 1, false, kSeen>(w, grid, stream);
    case 4: return launch<HD, 4, false, kSeen>(w, grid, stream);
    default: return launch<HD, 8, false, kSeen>(w, grid, stream);
  }
}

template <int kSeen>
hipError_t launch_seen(const PagedArgs& a, int hd, void* workspace, hipStream_t stream) {
  const Shape s = shape_of<kSeen>(a.B, a.max_q, a.nh, a.nkv, hd, (int64_t)a.B * ((int64_t)a.width << a.page_shift));
  Work w;
  w.a = a;
  w.G = s.G;
  w.RB = s.RB;
  w.unit = s.unit;
  w.target_log2 = __builtin_ctz((unsigned)s.target);
  w.min_chunk = s.min_chunk;
  w.pid_cap = s.pid_cap;
  w.c = a.scale * kLog2e;
  char* base = static_cast<char*>(workspace);
  w.req = reinterpret_cast<int2*>(base + s.off_req);
  w.part_ml = reinterpret_cast<floatx4*>(base + s.off_ml);
  w.part_o = reinterpret_cast<float*>(base + s.off_o);
  w.plan = nullptr;
  w.count = reinterpret_cast<int*>(base + s.off_count);
  // The table's width is the host's only bound on the lengths, so that a wide one costs the
  // plan, the join and surplus workgroups: one token over 517 keys 8.7 us under a table of that
  // length and 11.0 under one of 131072 keys, 64 requests of up to 512 keys 15.8 and 21.7.  A
  // window bounds the span too: its keys, the block's, the sinks', and what completes a group.
  // (A block longer than max_q may pass that: it is one range then, or there is room for its ranges.)
  const int held = a.width << a.page_shift;
  auto bound = [&](int block) {
    return kSeen != kRecent ? held : (int)std::min<int64_t>(held, (int64_t)a.sink_keys + a.window + block + 16);
  };
  w.cut = bound(a.max_q) > s.whole;
  if (kSeen == kRecent) {
    // Under a window requests are about as long as each other, and where they alone fill the card,
    // cutting them costs the plan and the join for nothing: 16 requests of one token under a window of
    // 2048, 32/8 heads of 128, in us in a captured graph, 39.6 whole and 41.7 cut, 64 of 17 tokens under one
    // of 512 46 and 52, of 2048 129 and 135; but 4 of one token under 2048 27 and 20, 32 of 17 tokens under
    // 2048 107 and 85, 16 of one token under 8192 130 and 110.  Large calls even out by the cut what their
    // uneven ends cost: 256 of 1 to 17 tokens under 1024 247 and 267, 1500 337 and 339, 2048 440 and
    // 440, 2600 543 and 541, 3500 713 and 702, 4096 820 and 813, 8192 1570 and 1486.  The last condition's
    // bound lies at about 2500 of these, where the two are within a hundredth.
    const int64_t groups = (int64_t)a.B * s.unit, span = bound(a.max_q);
    const bool fill = s.RT == 1 ? span <= 32 * groups : span <= 2 * groups || groups >= 2 * kCus;
    if (fill && groups * span <= (5 << 20)) w.cut = 0;
  }
  // at most one range per request, plus the ones the balancing adds
  const int64_t most = (int64_t)a.B * s.unit * (w.cut ? (bound(a.T) + s.min_chunk - 1) / s.min_chunk : 1);
  const int64_t items = std::min(most, (int64_t)a.B * s.unit + s.target + s.unit);
  if (a.B > 1 && w.cut) {
    w.plan = reinterpret_cast<Item*>(base + s.off_plan);
    hipLaunchKernelGGL(paged_plan<kSeen>, dim3(1), dim3(a.B <= 1024 ? 256 : kPlanThreads), 0, stream, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  switch (hd) {
    case 64: return launch_rt<64, kSeen>(w, s, (int)items, stream);
    case 128: return launch_rt<128, kSeen>(w, s, (int)items, stream);
    case 256: return launch_rt<256, kSeen>(w, s, (int)items, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

}  // namespace dspark
