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

// a range of one request's keys: the work of a workgroup for every (row block, kv head)
struct __attribute__((aligned(16))) Item {
  int b, k0, k1;       // request, its keys k0 .. k1 - 1
  int pid;             // partial to leave, or -1: the request's only range
  int q0, n, kv;       // the request's first query token, their number, its keys
  int pad;
};

struct Work {
  PagedArgs a;
  int G, RB, unit;     // heads per kv head, row blocks, nkv * RB
  int target_log2;     // items aimed at, a power of two
  int min_chunk;       // keys of a range, at least
  int whole;           // no request is cut where none can be longer than this
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
__device__ __forceinline__ bool find_item(const Work& w, int u, Item& it) {
  const PagedArgs& a = w.a;
  if (w.plan) {
    if (u >= *w.count) return false;
    it = w.plan[u];
  } else if (a.B == 1 && (a.width << a.page_shift) > w.whole) {
    request(a, 0, it.q0, it.n, it.kv);
    const int chunk = chunk_of(w, it.kv);
    const int len = range_len(it.kv, max(1, (it.kv + chunk - 1) / chunk));
    const int ranges = len > 0 ? (it.kv + len - 1) / len : 1;
    if (u >= ranges || it.n == 0) return false;
    it.b = 0;
    it.k0 = u * len;
    it.k1 = min(it.kv, it.k0 + len);
    it.pid = ranges > 1 ? u : -1;
    if (u == 0 && threadIdx.x == 0) w.req[0] = make_int2(0, ranges);
  } else {
    request(a, u, it.q0, it.n, it.kv);
    if (it.n == 0) return false;
    it.b = u;
    it.k0 = 0;
    it.k1 = it.kv;
    it.pid = -1;
  }
  it.b = uniform(it.b);
  it.k0 = uniform(it.k0);
  it.k1 = uniform(it.k1);
  it.pid = uniform(it.pid);
  it.q0 = uniform(it.q0);
  it.n = uniform(it.n);
  it.kv = uniform(it.kv);
  return true;
}

// The plan of a call with several requests: one workgroup cuts the requests into ranges
// and lists them by falling length (to a 256th of the longest), so that the dearest start
// first.  The order among equals is that of the atomics and decides nothing but time: a
// range's place among the partials comes from the requests alone.
constexpr int kPlanThreads = 1024, kPlanEach = 4;   // 256 threads are enough for 1024 requests

__global__ __launch_bounds__(kPlanThreads) void paged_plan(Work w) {
  const PagedArgs& a = w.a;
  __shared__ int64_t sums[kPlanThreads / 64];
  __shared__ int offs[kPlanThreads / 64], bins[256], cursor[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x;
  int q0[kPlanEach], n[kPlanEach], kv[kPlanEach], ranges[kPlanEach], len[kPlanEach];
  int64_t total = 0;
#pragma unroll
  for (int e = 0; e < kPlanEach; ++e) {
    const int b = e * threads + tid;
    q0[e] = n[e] = kv[e] = 0;
    if (b < a.B) request(a, b, q0[e], n[e], kv[e]);
    if (n[e] > 0) total += kv[e];
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
      len[e] = range_len(kv[e], max(1, (kv[e] + chunk - 1) / chunk));
      ranges[e] = len[e] > 0 ? (kv[e] + len[e] - 1) / len[e] : 1;
      if (ranges[e] > 1) {
        split += ranges[e];
        atomicAdd(&bins[bin(len[e])], ranges[e] - 1);
      }
      atomicAdd(&bins[bin(kv[e] - (ranges[e] - 1) * len[e])], 1);
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
        w.plan[at + r] = Item{b, r * len[e], (r + 1) * len[e], pid + r, q0[e], n[e], kv[e], 0};
    }
    const int at = atomicAdd(&cursor[bin(kv[e] - full * len[e])], 1);
    w.plan[at] = Item{b, full * len[e], kv[e], full > 0 ? pid + full : -1, q0[e], n[e], kv[e], 0};
    if (full > 0) pid += ranges[e];
  }
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
template <int HD, int NW, bool kSlots, bool kLse>
__global__ __launch_bounds__(64 * NW) void paged_rows(Work w) {
  using D = Dims<HD>;
  constexpr int ODIM = 16 * D::VD;                // dims of one group
  const PagedArgs& a = w.a;
  __shared__ float obuf[NW][16][ODIM + 4];
  __shared__ float mbuf[NW][16], lbuf[NW][16], xbuf[NW][16];

  const int u = blockIdx.x / w.unit, kvh = blockIdx.x % w.unit;
  Item it;
  if (!find_item(w, u, it)) return;
  if (it.pid >= w.pid_cap) return;                // (the workspace holds every range)
  const int nq = min(it.n, a.max_q);

  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);

  // queries: the B operand of S^T, row c, dims 32 kk + 8 g ..
  const int qj = c / w.G;
  const bool ok = qj < nq;
  const int lim = ok && a.causal ? it.kv - it.n + qj + 1 : it.kv;   // keys below lim are seen
  const int minlim = a.causal ? it.kv - it.n + 1 : it.kv;
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
  auto find = [&](int key0) {
    if constexpr (kSlots) {
      where[0] = table[min(key0 + (lane & 31), it.kv - 1) >> a.page_shift];
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) where[s] = table[min(key0 + 16 * s, it.kv - 1) >> a.page_shift];
    }
  };
  if (it.k0 + KT * wave < it.k1) find(it.k0 + KT * wave);
  for (int key0 = it.k0 + KT * wave; key0 < it.k1; key0 += KT * NW) {
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
    find(key0 + KT * NW);
    held = (uint32_t)uniform((int)held);
    const bool partial = uniform(held != 0xFFFFFFFFu || key0 + KT > minlim) != 0;

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
    if (partial) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = 16 * (e >> 2) + 4 * g + (e & 3);
        if (!((held >> i) & 1u) || key0 + i >= lim) sc[e >> 2][e & 3] = -INFINITY;
      }
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
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(sc[e >> 2][e & 3], rc, -mb));
    // the weights' rounding to bf16, the second product's operand type
    const bf16x8 p = pack_weights<kLse>(x, l, lx);

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
            if (key0 + k < lim) o[y][t] += add;
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

template <int HD, int RT, bool kSlots, bool kLse>
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
  if (!find_item(w, u, it)) return;
  const int nq = min(it.n, a.max_q), row0 = rb * 16 * RT;
  if (nq * w.G <= row0) return;                                 // (no row of this block exists)
  if (it.pid >= w.pid_cap) return;                // (the workspace holds every range)

  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const bool idle = uniform(row0 + 16 * wave >= nq * w.G) != 0;  // a wave without rows only loads
  const int row = row0 + 16 * wave + c, j = row / w.G, h = kvh * w.G + row % w.G;
  const bool ok = j < nq;
  const int lim = ok && a.causal ? it.kv - it.n + j + 1 : it.kv;        // keys below lim are seen
  const int minlim = a.causal ? it.kv - it.n + 1 + (row0 + 16 * wave) / w.G : it.kv;
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
  int half[LPW], row_of[LPW];                     // which 16 keys; this lane's row of the tile
#pragma unroll
  for (int q = 0; q < LPW; ++q) {
    const int f = uniform(q * RT + wave), fk = f % (LOADS / 2), r = fk * LR + lrow;
    from[q] = f < LOADS / 2 ? kbase : vbase;
    to[q] = f * 1024;
    half[q] = fk * LR >> 4;
    row_of[q] = r;
    off[q] = (uint32_t)(lslot ^ swizzle<HD>(r)) << 4;
    if (!kSlots) off[q] += (uint32_t)(r & 15) * (uint32_t)rbytes;
  }
  // Where a tile lies is read from LDS a tile ahead; a key that does not exist reads an
  // existing row.
  int slot[kSlots ? LPW : 2];                     // of this lane's rows; of the two first keys
  auto find = [&](int key0, int win0, int win1) {
    if constexpr (kSlots) {
#pragma unroll
      for (int q = 0; q < LPW; ++q) slot[q] = slots[min(key0 + row_of[q], win1 - 1) - win0];
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) slot[s] = slots[(min(key0 + 16 * s, win1 - 1) - win0) >> 4];
    }
  };
  auto issue = [&](int key0, int stage) {
    const uint32_t lds = lds0 + stage * 2 * TILEB;
    if constexpr (kSlots) {
#pragma unroll
      for (int q = 0; q < LPW; ++q) load_to_lds16(from[q] + (int64_t)max(slot[q], 0) * rbytes + off[q], uniform(lds + to[q]));
    } else {
      int64_t at[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) at[s] = (int64_t)max(uniform(slot[s]), 0) * rbytes;
      const bool tail = uniform(gaps || key0 + KT > it.kv) != 0;
#pragma unroll
      for (int q = 0; q < LPW; ++q) {
        uint32_t o = off[q];
        if (tail) {
          const int first = half[q] ? uniform(slot[1]) : uniform(slot[0]), r = row_of[q] & 15;
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

  // bit i: key key0 + i exists
  auto held_of = [&](int key0, int win0) {
    const int key = min(key0 + (lane & 31), it.kv - 1), e = key - win0;
    const bool there = slots[kSlots ? e : e >> 4] >= 0 && key0 + (lane & 31) < it.kv;
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
  auto mask = [&](floatx4 (&sc)[2], uint32_t held, int key0) {
    held >>= 4 * g;
    const int left = lim - key0 - 4 * g;          // keys below this are seen
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      constexpr int at[8] = {0, 1, 2, 3, 16, 17, 18, 19};
      if (!((held >> at[e]) & 1u) || at[e] >= left) sc[e >> 2][e & 3] = -INFINITY;
    }
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
  auto work_on = [&](const char* kb, int key0, int win0) {
    const char* vb = kb + TILEB;
    asm volatile("" : "+v"(koff), "+v"(voff[0]), "+v"(voff[1]));   // (flipped offsets are cheaper than registers)
    floatx4 sc[2];
    scores(kb, sc);
    int whole = 1;
    if (uniform(gaps || key0 + KT > minlim)) {
      mask(sc, held_of(key0, win0), key0);
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
  auto add_left_out = [&](const char* kb, int key0, int win0) {
    const char* vb = kb + TILEB;
    if (!uniform(gaps || key0 + KT > minlim) || finite(vb)) return;
    const uint32_t held = held_of(key0, win0);
    floatx4 sc[2];
    float counted = 0.0f;                         // (its weights are in the sums already)
    scores(kb, sc);
    mask(sc, held, key0);
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
        if (key0 + k < lim) o[d] += add;
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
      const int key = win0 + (kSlots ? e : e << 4);
      const int page = table[key >> a.page_shift];
      slots[e] = page >= 0 && page < a.num_pages ? (page << a.page_shift) + (key & pmask) : -1;
      missing |= slots[e] < 0;
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
      for (int key0 = win0; key0 < win1; key0 += KT) {
        // this wave's loads of the tile have landed; after the barrier everyone's have, and
        // everyone is done with the tile before
        const int ahead = win1 - key0 - 1;        // / KT: younger tiles on their way, at most kStages - 2
        if (uniform(ahead >= (kStages - 2) * KT)) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 2) * LPW) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_barrier();
        if (uniform(ahead >= (kStages - 1) * KT)) {
          issue(key0 + (kStages - 1) * KT, stage == 0 ? kStages - 1 : stage - 1);
          find(key0 + kStages * KT, win0, win1);
        }
        on_tile(smem + stage * 2 * TILEB, key0, win0);
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
  int RT, RB, G, unit, target, min_chunk, whole, pid_cap;
  size_t off_o, off_ml, off_req, off_plan, off_count, bytes;
};

Shape shape_of(int B, int max_q, int nh, int nkv, int hd) {
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  Shape s;
  s.G = nh / nkv;
  const int rows = max_q * s.G;
  // Waves of 16 rows a workgroup: 64 requests over 100..4000 keys, 32/8 heads of 128, take
  // 114 us with 4 rows by paged_rows and 126 by shared tiles, 118 and 130 with 16; 20 rows
  // 130 us with four waves (two of them only load) and 131 with two, 40 rows 135 with four
  // and 144 with eight, 68 rows 166 with eight and 190 with four.
  s.RT = rows <= 16 ? 1 : rows <= 64 ? 4 : 8;
  s.RB = (rows + 16 * s.RT - 1) / (16 * s.RT);
  s.unit = nkv * s.RB;
  // items aimed at: two workgroups on each compute unit (one with heads of 256) draw all
  // that memory gives, and shorter ranges cost more in starting and joining than they
  // even out: 64 blocks of 16 x 4 rows over 100..4000 keys take 145 us so, 150 at twice
  // and 163 us at four times as many; one token over 131071 keys 104, 110 and 118 us
  s.target = kCus * (hd > 128 ? 1 : 2);
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

template <int HD, int RT, bool kSlots, bool kLse>
hipError_t launch_rows(const Work& w, int grid, hipStream_t stream) {
  if constexpr (RT > 1) {
    constexpr int lds = shared_lds<HD>();
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&paged_shared<HD, RT, kSlots, kLse>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((paged_shared<HD, RT, kSlots, kLse>), dim3(grid), dim3(64 * RT), lds, stream, w);
  } else {
    // Eight waves where no compute unit gets a second workgroup: one token over 517 keys, 32/8
    // heads of 128, 9.2 us with eight and 10.2 with four, 32 of them 13.6 and 15.4.  Heads of 256
    // leave registers for four.
    constexpr int most = HD > 128 ? 4 : 8;
    if (grid <= kCus) hipLaunchKernelGGL((paged_rows<HD, most, kSlots, kLse>), dim3(grid), dim3(64 * most), 0, stream, w);
    else hipLaunchKernelGGL((paged_rows<HD, 4, kSlots, kLse>), dim3(grid), dim3(64 * 4), 0, stream, w);
  }
  return hipGetLastError();
}

template <int HD, int RT>
hipError_t launch(const Work& w, int64_t items, int max_kv, hipStream_t stream) {
  const int grid = (int)items;
  const bool slots = w.a.page_shift < 4, lse = w.a.lse != nullptr;
  const hipError_t e = slots ? lse ? launch_rows<HD, RT, true, true>(w, grid, stream) : launch_rows<HD, RT, true, false>(w, grid, stream)
                       : lse ? launch_rows<HD, RT, false, true>(w, grid, stream)
                             : launch_rows<HD, RT, false, false>(w, grid, stream);
  if (e != hipSuccess || max_kv <= w.whole) return e;
  const int rows = std::min(16 * RT, w.a.max_q * w.G);
  const int step = std::max(1, std::min(rows, (int)((int64_t)w.a.B * w.unit * rows / kJoinGroups)));
  hipLaunchKernelGGL((paged_join<HD, RT>), dim3(w.a.B * w.unit, (rows + step - 1) / step), dim3(256), 0, stream, w, step);
  return hipGetLastError();
}

template <int HD>
hipError_t launch_rt(const Work& w, int RT, int64_t items, int max_kv, hipStream_t stream) {
  switch (RT) {
    case 1: return launch<HD, 1>(w, items, max_kv, stream);
    case 4: return launch<HD, 4>(w, items, max_kv, stream);
    default: return launch<HD, 8>(w, items, max_kv, stream);
  }
}

}  // namespace

size_t paged_attention_workspace_bytes(int T, int B, int max_q, int nh, int nkv, int hd) {
  (void)T;
  return shape_of(B, max_q, nh, nkv, hd).bytes;
}

hipError_t launch_paged_attention(const PagedArgs& a, int hd, void* workspace, hipStream_t stream) {
  const Shape s = shape_of(a.B, a.max_q, a.nh, a.nkv, hd);
  Work w;
  w.a = a;
  w.G = s.G;
  w.RB = s.RB;
  w.unit = s.unit;
  w.target_log2 = __builtin_ctz((unsigned)s.target);
  w.min_chunk = s.min_chunk;
  w.whole = s.whole;
  w.pid_cap = s.pid_cap;
  w.c = a.scale * kLog2e;
  char* base = static_cast<char*>(workspace);
  w.req = reinterpret_cast<int2*>(base + s.off_req);
  w.part_ml = reinterpret_cast<floatx4*>(base + s.off_ml);
  w.part_o = reinterpret_cast<float*>(base + s.off_o);
  w.plan = nullptr;
  w.count = reinterpret_cast<int*>(base + s.off_count);
  // at most one range per request, plus the ones the balancing adds.  The table's width is the
  // host's only bound on the lengths, so that a wide one costs the plan, the join and surplus
  // workgroups: one token over 517 keys 8.7 us under a table of that length and 11.0 under one of
  // 131072 keys, 64 requests of up to 512 keys 15.8 and 21.7.
  const int max_kv = a.width << a.page_shift;
  const int64_t most = (int64_t)a.B * s.unit * (max_kv <= s.whole ? 1 : (max_kv + s.min_chunk - 1) / s.min_chunk);
  const int64_t items = std::min(most, (int64_t)a.B * s.unit + s.target + s.unit);
  if (a.B > 1 && max_kv > s.whole) {
    w.plan = reinterpret_cast<Item*>(base + s.off_plan);
    hipLaunchKernelGGL(paged_plan, dim3(1), dim3(a.B <= 1024 ? 256 : kPlanThreads), 0, stream, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  switch (hd) {
    case 64: return launch_rt<64>(w, s.RT, items, max_kv, stream);
    case 128: return launch_rt<128>(w, s.RT, items, max_kv, stream);
    case 256: return launch_rt<256>(w, s.RT, items, max_kv, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dspark
