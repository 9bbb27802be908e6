// Attention of a few query tokens per request over its pages of the key-value cache.
//
//   out[r] = sum_s exp2(x_rs - m_r) v_s / sum_s exp2(x_rs - m_r),   x_rs = q_r . k_s * scale * log2 e
//
// over the keys s row r sees, in one pass with a running maximum m_r and sum.  The nh / nkv
// query heads that share a kv head, times the request's query tokens, are the rows of one
// product, so a key or value is read from memory once per kv head (row blocks of 16 RT).
//
// Each wave takes tiles of 32 keys, all by itself in registers (no LDS in the loop: no
// other wave needs its keys).  Scores are formed transposed, S^T = K Q^T, with
// v_mfma_f32_16x16x32_bf16: lane (g, c) = (lane / 16, lane % 16) then holds row c and the
// keys 16 s + 4 g + i (s = 0, 1; i = 0..3).  The second product O^T = V^T P^T may take its
// 32 keys in any order as long as both operands agree, so those eight scores, rounded to
// bf16, are its B operand as they stand.  Its A operand needs eight keys of one dim per
// lane: a lane loads 8 consecutive dims of its eight keys (16 lanes cover a row, 16 bytes
// each) and transposes the 8 x 8 block with byte permutes; product t then covers the
// dims 8 c + t.
//
// Work items (request, range of its keys, row block, kv head) come from the lengths on
// the device: ranges are all of one length, chosen so that all items together are about
// `target`, and a request shorter than that is one item, written straight to the output.
// The others leave a maximum, a sum and an unnormalised row each, joined by
// paged_join in the order of the ranges.
#include <algorithm>

#include "attention.hpp"
#include "kernels.hpp"

namespace dspark {

namespace {

// The running maximum is raised only when a row's scores exceed it by kRaise (weights up
// to 2^kRaise, which neither float nor bf16 minds): the accumulators are rescaled on a
// row's first tile and hardly ever after.
constexpr float kRaise = 8.0f;

constexpr int NW = 4;          // waves per workgroup; they take tiles in turn
constexpr int KT = 32;         // keys per tile
constexpr int kMinChunk = 512; // keys of a range, at least
constexpr int kCus = 256;      // compute units of the card
constexpr int kJoinGroups = 2048;   // workgroups of the joining pass aimed at

struct Work {
  PagedArgs a;
  int G, RB, unit;     // heads per kv head, row blocks, nkv * RB
  int target;          // items aimed at
  int pid_cap;         // ranges the workspace has room for
  float c;             // scale * log2 e
  float* part_o;       // [pid_cap, unit, 16 RT, hd]
  float* part_ml;      // [pid_cap, unit, 16 RT, 2]
  int2* req;           // [B]: first range and number of ranges of a split request
};

struct Item {
  int b, q0, n, kv, split, nsplit, pid, chunk;
};

// n counts all of the request's query tokens; the first max_q of them are computed
__device__ __forceinline__ void request(const PagedArgs& a, int b, int& q0, int& n, int& kv) {
  q0 = clampi(a.cu_q[b], 0, a.T);
  n = clampi(a.cu_q[b + 1], q0, a.T) - q0;
  kv = clampi(a.kv_len[b], 0, a.width << a.page_shift);
}

__device__ __forceinline__ int wave_incl_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// the u-th (request, range) of the call; every wave finds it for itself
__device__ bool find_item(const Work& w, int u, Item& it) {
  const PagedArgs& a = w.a;
  const int lane = threadIdx.x & 63;
  const int step = KT * NW;
  if (a.B == 1) {
    request(a, 0, it.q0, it.n, it.kv);
    if (it.n == 0) return false;
    const int64_t per = ((int64_t)it.kv * w.unit + w.target - 1) / w.target;
    it.chunk = max(kMinChunk, (int)((per + step - 1) / step * step));
    it.b = 0;
    it.nsplit = max(1, (it.kv + it.chunk - 1) / it.chunk);
    it.split = u;
    it.pid = u;
    return u < it.nsplit;
  }
  int q0, n, kv;
  int64_t total = 0;
  for (int base = 0; base < a.B; base += 64) {
    if (base + lane < a.B) {
      request(a, base + lane, q0, n, kv);
      if (n > 0) total += kv;
    }
  }
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  const int64_t per = (total * w.unit + w.target - 1) / w.target;
  const int64_t up = (per + step - 1) / step * step;
  it.chunk = (int)(up < kMinChunk ? kMinChunk : up > (1 << 30) ? (1 << 30) : up);
  int before = 0, pids = 0;
  for (int base = 0; base < a.B; base += 64) {
    int cnt = 0;
    q0 = n = kv = 0;
    if (base + lane < a.B) {
      request(a, base + lane, q0, n, kv);
      if (n > 0) cnt = max(1, (kv + it.chunk - 1) / it.chunk);
    }
    const int split_cnt = cnt > 1 ? cnt : 0;
    const int inc = wave_incl_scan(cnt, lane), pinc = wave_incl_scan(split_cnt, lane);
    const uint64_t hit = __ballot(before + inc > u);
    if (hit) {
      const int s = __builtin_ctzll(hit);
      it.b = __builtin_amdgcn_readfirstlane(base + s);
      it.q0 = __builtin_amdgcn_readlane(q0, s);
      it.n = __builtin_amdgcn_readlane(n, s);
      it.kv = __builtin_amdgcn_readlane(kv, s);
      it.nsplit = __builtin_amdgcn_readlane(cnt, s);
      it.split = u - before - (__builtin_amdgcn_readlane(inc, s) - it.nsplit);
      it.pid = pids + __builtin_amdgcn_readlane(pinc, s) - __builtin_amdgcn_readlane(split_cnt, s) + it.split;
      return true;
    }
    before += __builtin_amdgcn_readlane(inc, 63);
    pids += __builtin_amdgcn_readlane(pinc, 63);
  }
  return false;
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

template <int HD>
struct Dims {
  static constexpr int VD = HD >= 128 ? 8 : 4;    // dims a lane loads of a value row, per group of 16 VD
  static constexpr int VU = HD / (16 * VD);       // such groups
  static constexpr int VW = VD / 2;               // their 32-bit words
};

// kSlots: pages smaller than 16, so the slot of every key is looked up by a lane of its
// own; otherwise 16 aligned keys lie in one page and the wave looks up two
template <int HD, int RT, bool kSlots>
__global__ __launch_bounds__(64 * NW) void paged_rows(Work w) {
  using D = Dims<HD>;
  constexpr int ODIM = 16 * D::VD;                // dims of one group
  const PagedArgs& a = w.a;
  __shared__ float obuf[NW][16][ODIM + 4];
  __shared__ float mbuf[NW][16], lbuf[NW][16];

  const int u = blockIdx.x / w.unit, rest = blockIdx.x % w.unit;
  const int kvh = rest % a.nkv, rb = rest / a.nkv;
  Item it;
  if (!find_item(w, u, it)) return;
  it.b = uniform(it.b);
  it.q0 = uniform(it.q0);
  it.n = uniform(it.n);
  it.kv = uniform(it.kv);
  it.chunk = uniform(it.chunk);
  it.split = uniform(it.split);
  it.nsplit = uniform(it.nsplit);
  it.pid = uniform(it.pid);
  if (rest == 0 && it.split == 0 && threadIdx.x == 0)
    w.req[it.b] = make_int2(it.pid, it.nsplit);
  const int nq = min(it.n, a.max_q);
  const int rows = nq * w.G - rb * 16 * RT;       // rows of this block, possibly none
  if (rows <= 0) return;
  if (it.nsplit > 1 && it.pid >= w.pid_cap) return;   // (the workspace holds every range)

  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // queries: the B operand of S^T, row 16 rt + c, dims 32 kk + 8 g ..
  bf16x8 qf[RT][HD / 32];
  int lim[RT];                                    // keys below lim are seen
  int minlim = it.kv;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = rb * 16 * RT + 16 * rt + c;
    const int j = r / w.G, h = kvh * w.G + r % w.G;
    const bool ok = j < nq;
    lim[rt] = ok && a.causal ? it.kv - it.n + j + 1 : it.kv;
    const uint16_t* src = a.q + (size_t)(it.q0 + (ok ? j : 0)) * a.q_stride + (size_t)(ok ? h : 0) * HD;
#pragma unroll
    for (int kk = 0; kk < HD / 32; ++kk) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 32 * kk + 8 * g);
      qf[rt][kk] = __builtin_bit_cast(bf16x8, ok ? v : make_uint4(0, 0, 0, 0));
    }
  }
  if (a.causal) minlim = it.kv - it.n + 1 + (rb * 16 * RT) / w.G;

  floatx4 o[RT][D::VU][D::VD];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY;
    l[rt] = 0.0f;
#pragma unroll
    for (int x = 0; x < D::VU; ++x)
#pragma unroll
      for (int t = 0; t < D::VD; ++t) o[rt][x][t] = floatx4{0.f, 0.f, 0.f, 0.f};
  }

  const int k0 = it.split * it.chunk, k1 = min(it.kv, k0 + it.chunk);
  const int32_t* table = a.page_table + (size_t)it.b * a.width;
  const int rstride = a.nkv * HD;                 // elements between slots
  const int pmask = (1 << a.page_shift) - 1;

  for (int key0 = k0 + KT * wave; key0 < k1; key0 += KT * NW) {
    // the tile's keys and values; a key that does not exist reads an existing row
    uint32_t held;                                // bit i: key key0 + i exists
    uint32_t kf[2][HD / 32][4], vf[D::VU][8][D::VW];
    if constexpr (kSlots) {
      const int key = min(key0 + (lane & 31), it.kv - 1);
      const int page = table[key >> a.page_shift];
      const bool ok = key0 + (lane & 31) < it.kv && page >= 0 && page < a.num_pages;
      const int slot = (page >= 0 && page < a.num_pages ? page << a.page_shift : 0) + (key & pmask);
      held = (uint32_t)__ballot(ok);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint16_t* src = a.k_cache + ((size_t)__shfl(slot, 16 * s + c) * rstride + kvh * HD);
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)
          *reinterpret_cast<uint4*>(kf[s][kk]) = *reinterpret_cast<const uint4*>(src + 32 * kk + 8 * g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint16_t* src = a.v_cache + ((size_t)__shfl(slot, 16 * (j >> 2) + 4 * g + (j & 3)) * rstride + kvh * HD);
#pragma unroll
        for (int x = 0; x < D::VU; ++x)
          if constexpr (D::VD == 8)
            *reinterpret_cast<uint4*>(vf[x][j]) = *reinterpret_cast<const uint4*>(src + ODIM * x + 8 * c);
          else
            *reinterpret_cast<uint2*>(vf[x][j]) = *reinterpret_cast<const uint2*>(src + ODIM * x + 4 * c);
      }
    } else {
      held = 0;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int ks = key0 + 16 * s;
        int cnt = min(16, it.kv - ks);            // keys of this half, possibly <= 0
        int page = uniform(table[min(ks, it.kv - 1) >> a.page_shift]);
        if (page < 0 || page >= a.num_pages) {
          page = 0;
          cnt = 0;
        }
        cnt = max(cnt, 0);
        held |= ((1u << cnt) - 1u) << (16 * s);
        const size_t slot = ((size_t)page << a.page_shift) + (ks & pmask);
        const uint16_t* kb = a.k_cache + (slot * rstride + kvh * HD);
        const uint16_t* vb = a.v_cache + (slot * rstride + kvh * HD);
        const int last = max(cnt - 1, 0);
        const uint16_t* src = kb + min(c, last) * rstride;
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)
          *reinterpret_cast<uint4*>(kf[s][kk]) = *reinterpret_cast<const uint4*>(src + 32 * kk + 8 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint16_t* vs = vb + min(4 * g + j, last) * rstride;
#pragma unroll
          for (int x = 0; x < D::VU; ++x)
            if constexpr (D::VD == 8)
              *reinterpret_cast<uint4*>(vf[x][4 * s + j]) = *reinterpret_cast<const uint4*>(vs + ODIM * x + 8 * c);
            else
              *reinterpret_cast<uint2*>(vf[x][4 * s + j]) = *reinterpret_cast<const uint2*>(vs + ODIM * x + 4 * c);
        }
      }
    }
    held = (uint32_t)uniform((int)held);
    const bool partial = uniform(held != 0xFFFFFFFFu || key0 + KT > minlim) != 0;

    // scores, and from them the weights: registers only
    bf16x8 p[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (16 * rt >= rows) break;
      floatx4 sc[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        sc[s] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)
          sc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, *reinterpret_cast<uint4*>(kf[s][kk])), qf[rt][kk], sc[s], 0, 0, 0);
      }
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = sc[e >> 2][e & 3] * w.c;
      if (partial) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = 16 * (e >> 2) + 4 * g + (e & 3);
          if (!((held >> i) & 1u) || key0 + i >= lim[rt]) x[e] = -INFINITY;
        }
      }
      float tm = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) tm = fmaxf(tm, x[e]);
      tm = groups_max(tm);
      const float mn = fmaxf(m[rt], tm);
      const float ms = mn == -INFINITY ? 0.0f : mn;   // a row that has seen nothing yet
      const float al = __builtin_amdgcn_exp2f(m[rt] - ms);
      m[rt] = mn;
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = __builtin_amdgcn_exp2f(x[e] - ms);
        sum += x[e];
      }
      l[rt] = l[rt] * al + sum;
      // the weights' rounding to bf16, the second product's operand type
      p[rt] = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                    pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
      if (__any(al != 1.0f)) {
#pragma unroll
        for (int y = 0; y < D::VU; ++y)
#pragma unroll
          for (int t = 0; t < D::VD; ++t) o[rt][y][t] *= al;
      }
    }

    // in a tile some row does not see whole, a value that is not finite must not meet
    // that row's zero weight
    int odd = 0;
    if (partial) {
      bool any = false;
#pragma unroll
      for (int y = 0; y < D::VU; ++y)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int d = 0; d < D::VW; ++d) any |= bf16x2_nonfinite(vf[y][j][d]);
      odd = __any(any);
    }
    odd = uniform(odd);
#pragma unroll
    for (int y = 0; y < D::VU; ++y) {
#pragma unroll
      for (int t = 0; t < D::VD; ++t) {
        const uint32_t sel = t & 1 ? 0x07060302u : 0x05040100u;
        uint32_t vt[4];
#pragma unroll
        for (int d = 0; d < 4; ++d)
          vt[d] = __builtin_amdgcn_perm(vf[y][2 * d + 1][t >> 1], vf[y][2 * d][t >> 1], sel);
        if (!odd) {
          const bf16x8 va = __builtin_bit_cast(bf16x8, make_uint4(vt[0], vt[1], vt[2], vt[3]));
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            if (16 * rt < rows) o[rt][y][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, p[rt], o[rt][y][t], 0, 0, 0);
        } else {
          // key by key, added only to the rows that see it
          for (int k = 0; k < KT; ++k) {
            if (!((held >> k) & 1u)) continue;
            const int j = (k & 3) | ((k >> 4) << 2);
            const uint32_t half = j & 1 ? 0xFFFF0000u : 0x0000FFFFu;
            const bool mine = g == ((k >> 2) & 3);
            const bf16x8 va = __builtin_bit_cast(
                bf16x8, make_uint4(mine && j / 2 == 0 ? vt[0] & half : 0u, mine && j / 2 == 1 ? vt[1] & half : 0u,
                                   mine && j / 2 == 2 ? vt[2] & half : 0u, mine && j / 2 == 3 ? vt[3] & half : 0u));
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              if (16 * rt >= rows) break;
              const floatx4 add = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, p[rt], (floatx4{0.f, 0.f, 0.f, 0.f}), 0, 0, 0);
              if (key0 + k < lim[rt]) o[rt][y][t] += add;
            }
          }
        }
      }
    }
  }

  // join the four waves, 16 rows and one dim group at a time
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (16 * rt >= rows) break;
    const float lt = groups_sum(l[rt]);
#pragma unroll
    for (int y = 0; y < D::VU; ++y) {
      __syncthreads();
      if (g == 0 && y == 0) {
        mbuf[wave][c] = m[rt];
        lbuf[wave][c] = lt;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < D::VD; t += 4)
          *reinterpret_cast<floatx4*>(&obuf[wave][c][D::VD * (4 * g + i) + t]) =
              floatx4{o[rt][y][t][i], o[rt][y][t + 1][i], o[rt][y][t + 2][i], o[rt][y][t + 3][i]};
      __syncthreads();
      float mm = -INFINITY, ll = 0.0f, f[NW], acc[D::VD];
#pragma unroll
      for (int v = 0; v < NW; ++v) mm = fmaxf(mm, mbuf[v][tr]);
      const float ms = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        f[v] = __builtin_amdgcn_exp2f(mbuf[v][tr] - ms);
        ll += lbuf[v][tr] * f[v];
      }
#pragma unroll
      for (int t = 0; t < D::VD; ++t) {
        acc[t] = 0.0f;
#pragma unroll
        for (int v = 0; v < NW; ++v) acc[t] += obuf[v][tr][D::VD * tc + t] * f[v];
      }
      const int r = rb * 16 * RT + 16 * rt + tr;
      const int j = r / w.G, h = kvh * w.G + r % w.G;
      if (j >= nq) continue;
      if (it.nsplit == 1) {
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        const size_t at = (size_t)(it.q0 + j) * a.nh + h;
        uint32_t pk[D::VW];
#pragma unroll
        for (int t = 0; t < D::VW; ++t) pk[t] = ll == 0.0f ? 0u : pack_bf16x2(acc[2 * t] * inv, acc[2 * t + 1] * inv);
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + at * HD + ODIM * y + D::VD * tc);
#pragma unroll
        for (int t = 0; t < D::VW; ++t) dst[t] = pk[t];
        if (a.lse && y == 0 && tc == 0) a.lse[at] = row_lse(mm, ll);
      } else {
        const size_t at = ((size_t)it.pid * w.unit + rest) * (16 * RT) + 16 * rt + tr;
        float* dst = w.part_o + at * HD + ODIM * y + D::VD * tc;
#pragma unroll
        for (int t = 0; t < D::VD; t += 4)
          *reinterpret_cast<floatx4*>(dst + t) = floatx4{acc[t], acc[t + 1], acc[t + 2], acc[t + 3]};
        if (y == 0 && tc == 0) {
          w.part_ml[2 * at] = mm;
          w.part_ml[2 * at + 1] = ll;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ many rows
// The same work for more than 16 rows: a wave takes 16 rows, and all waves of the
// workgroup share the keys, which pass through three LDS buffers of 32 (one worked on, two
// filling straight from memory).  Rows lie there in 16-byte pieces permuted (piece p of
// row r at p ^ swizzle(r)) so that the K reads (16 rows, one piece) and the transposing V
// reads (8 rows, two pieces) touch every bank once.  The slots of kWindow keys (small
// pages) or groups of 16 keys are looked up ahead into LDS by the whole workgroup.  Few
// registers and 52 KB of LDS leave room for three workgroups on a compute unit, which
// cover each other's waits.
constexpr int kWindow = 1024;
constexpr int kStages = 3;

template <int HD>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (HD == 64) return (((r >> 1) & 3) << 1) | ((r >> 3) & 1);
  return ((r & 7) << 1) | ((r >> 3) & 1);
}

template <int HD>
constexpr int shared_lds() {
  return kStages * 2 * KT * HD * 2 + kWindow * 4;
}

template <int HD, int RT, bool kSlots>
__global__ __launch_bounds__(64 * RT, HD > 128 || RT == 2 ? 2 : RT == 8 ? 4 : 3) void paged_shared(Work w) {
  constexpr int ROWB = HD * 2, TILEB = KT * ROWB, PIECES = HD / 8;
  constexpr int LOADS = 2 * TILEB / 1024;         // 1 KB loads of one tile, K then V
  constexpr int LPW = (LOADS + RT - 1) / RT;      // of a wave (the last wave's may repeat the last load)
  constexpr int LR = 64 / PIECES;                 // rows of one load
  extern __shared__ __attribute__((aligned(16))) char smem[];
  int32_t* slots = reinterpret_cast<int32_t*>(smem + kStages * 2 * TILEB);
  const PagedArgs& a = w.a;
  const int u = blockIdx.x / w.unit, rest = blockIdx.x % w.unit;
  const int kvh = rest % a.nkv, rb = rest / a.nkv;
  Item it;
  if (!find_item(w, u, it)) return;
  it.b = uniform(it.b);
  it.q0 = uniform(it.q0);
  it.n = uniform(it.n);
  it.kv = uniform(it.kv);
  it.chunk = uniform(it.chunk);
  it.split = uniform(it.split);
  it.nsplit = uniform(it.nsplit);
  it.pid = uniform(it.pid);
  if (rest == 0 && it.split == 0 && threadIdx.x == 0) w.req[it.b] = make_int2(it.pid, it.nsplit);
  const int nq = min(it.n, a.max_q), row0 = rb * 16 * RT;
  if (nq * w.G <= row0) return;                                 // (no row of this block exists)
  if (it.nsplit > 1 && it.pid >= w.pid_cap) return;             // (the workspace holds every range)

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
  float m = -INFINITY, mb = 0.0f, l = 0.0f;       // mb: m, or 0 while the row has seen nothing

  const int k0 = it.split * it.chunk, k1 = min(it.kv, k0 + it.chunk);
  const int32_t* table = a.page_table + (size_t)it.b * a.width;
  const int64_t rbytes = (int64_t)a.nkv * ROWB;   // bytes between slots
  const int pmask = (1 << a.page_shift) - 1;
  const char* kbase = reinterpret_cast<const char*>(a.k_cache + kvh * HD);
  const char* vbase = reinterpret_cast<const char*>(a.v_cache + kvh * HD);
  const int lrow = lane / PIECES, lslot = lane % PIECES;
  const uint32_t lds0 = lds_address(smem);

  // this wave's loads of a tile; a key that does not exist reads an existing row
  auto issue = [&](int key0, int win0, int stage) {
#pragma unroll
    for (int q = 0; q < LPW; ++q) {
      const int f = min(q * RT + wave, LOADS - 1), fk = f % (LOADS / 2);
      const char* base = f < LOADS / 2 ? kbase : vbase;
      const int r = fk * LR + lrow;               // row of the tile
      const uint32_t piece = (uint32_t)(lslot ^ swizzle<HD>(r)) << 4;
      const uint32_t lds = lds0 + stage * 2 * TILEB + f * 1024;
      if constexpr (kSlots) {
        const int64_t slot = max(slots[min(key0 + r, it.kv - 1) - win0], 0);
        load_to_lds16(base + slot * rbytes + piece, uniform(lds));
      } else {
        const int ks = key0 + (fk * LR & 16);     // the 16 keys of one page it falls in
        const int first = uniform(slots[(min(ks, it.kv - 1) - win0) >> 4]);
        const int last = first < 0 ? 0 : clampi(it.kv - 1 - ks, 0, 15);
        load_to_lds16(base + (int64_t)max(first, 0) * rbytes, (uint32_t)min(r & 15, last) * (uint32_t)rbytes + piece,
                      uniform(lds));
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

  auto work_on = [&](const char* kb, int key0, int win0) {
    const char* vb = kb + TILEB;
    asm volatile("" : "+v"(koff), "+v"(voff[0]), "+v"(voff[1]));   // (flipped offsets are cheaper than registers)
    bool there = key0 + (lane & 31) < it.kv;
    if (there) {
      const int e = key0 + (lane & 31) - win0;
      there = slots[kSlots ? e : e >> 4] >= 0;
    }
    floatx4 sc[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      sc[s] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < HD / 32; ++kk) {
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(kb + ((koff ^ (kk << 6)) + 16 * s * ROWB));
        sc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[kk], sc[s], 0, 0, 0);
      }
    }
    const uint32_t held = (uint32_t)uniform((int)(uint32_t)__ballot(there));   // bit i: key key0 + i exists
    const bool partial = uniform(held != 0xFFFFFFFFu || key0 + KT > minlim) != 0;
    uint32_t top = 0;                             // the largest exponent of a value, in the high half
    if (partial) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = 16 * (e >> 2) + 4 * g + (e & 3);
        if (!((held >> i) & 1u) || key0 + i >= lim) sc[e >> 2][e & 3] = -INFINITY;
      }
      for (int q = 0; q < TILEB / 1024; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(vb + q * 1024 + lane * 16);
        const uint32_t x[4] = {v.x & 0x7F807F80u, v.y & 0x7F807F80u, v.z & 0x7F807F80u, v.w & 0x7F807F80u};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(x[k], x[k] << 16));
      }
    }
    float hi = sc[0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) hi = fmaxf(hi, sc[e >> 2][e & 3]);
    const float tm = groups_max(hi) * w.c;
    if (uniform(__any(tm > m + kRaise))) {
      const float mn = tm > m + kRaise ? tm : m;
      const float al = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      mb = mn == -INFINITY ? 0.0f : mn;
      l *= al;
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) o[d] *= al;
    }
    // weights, rounded to bf16 (the second product's operand type), and their sum
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(sc[e >> 2][e & 3], w.c, -mb));
    l += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    const bf16x8 p = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                           pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
    // in a tile some row does not see whole, a value that is not finite must not meet
    // that row's zero weight
    if (!uniform(__any(top >= 0x7F800000u))) {
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(value_frag(vb, d).v, p, o[d], 0, 0, 0);
    } else {
      // key by key, added only to the rows that see it
#pragma unroll 1
      for (int k = 0; k < KT; ++k) {
        if (!((held >> k) & 1u)) continue;
        const int jj = (k & 3) | ((k >> 4) << 2);
        const uint32_t half = jj & 1 ? 0xFFFF0000u : 0x0000FFFFu;
        const uint32_t keep = g == ((k >> 2) & 3) ? half : 0u;
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
    }
  };

  constexpr int wkeys = kSlots ? kWindow : kWindow * 16;
  for (int win0 = k0; win0 < k1; win0 += wkeys) {
    const int win1 = min(k1, win0 + wkeys);
    __syncthreads();
    const int entries = kSlots ? win1 - win0 : (win1 - win0 + 15) >> 4;
    for (int e = threadIdx.x; e < entries; e += 64 * RT) {
      const int key = win0 + (kSlots ? e : e << 4);
      const int page = table[key >> a.page_shift];
      slots[e] = page >= 0 && page < a.num_pages ? (page << a.page_shift) + (key & pmask) : -1;
    }
    __syncthreads();
    issue(win0, win0, 0);
    if (win0 + KT < win1) issue(win0 + KT, win0, 1);
    int stage = 0;
    for (int key0 = win0; key0 < win1; key0 += KT) {
      // this wave's loads of the tile have landed; after the barrier everyone's have, and
      // everyone is done with the tile before
      if (uniform(key0 + KT < win1)) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LPW) : "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      lds_barrier();
      if (uniform(key0 + 2 * KT < win1)) issue(key0 + 2 * KT, win0, stage == 0 ? 2 : stage - 1);
      if (!idle) work_on(smem + stage * 2 * TILEB, key0, win0);
      stage = stage == 2 ? 0 : stage + 1;
    }
  }

  l = groups_sum(l);
  if (idle || !ok) return;
  if (it.nsplit == 1) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const size_t at = (size_t)(it.q0 + j) * a.nh + h;
#pragma unroll
    for (int d = 0; d < HD / 16; ++d)
      *reinterpret_cast<uint2*>(a.out + at * HD + 16 * d + 4 * g) =
          l == 0.0f ? make_uint2(0u, 0u)
                    : make_uint2(pack_bf16x2(o[d][0] * inv, o[d][1] * inv), pack_bf16x2(o[d][2] * inv, o[d][3] * inv));
    if (a.lse && g == 0) a.lse[at] = row_lse(m, l);
  } else {
    const size_t at = ((size_t)it.pid * w.unit + rest) * (16 * RT) + 16 * wave + c;
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) *reinterpret_cast<floatx4*>(w.part_o + at * HD + 16 * d + 4 * g) = o[d];
    if (g == 0) {
      w.part_ml[2 * at] = m;
      w.part_ml[2 * at + 1] = l;
    }
  }
}

// The ranges of split requests, joined in their order.  A workgroup takes `step` rows of one
// (request, row block, kv head); hd / 4 threads take a row, four dims each.  Up to kFew
// ranges they do so alone, every row of the workgroup at once; of more ranges the
// 256 / (hd / 4) groups take every so many each, row after row, and LDS joins the groups.
constexpr int kFew = 16;

struct Joined {
  float m, l;
  floatx4 acc;
};

// ranges first, first + hop, .. of row at0 (partials `stride` rows apart)
__device__ __forceinline__ Joined join_ranges(const Work& w, size_t at0, size_t stride, int ns, int first, int hop, int hd, int d) {
  Joined t{-INFINITY, 0.0f, floatx4{0.f, 0.f, 0.f, 0.f}};
  for (int s0 = first; s0 < ns; s0 += 4 * hop) {
    floatx2 ml[4];
    floatx4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int s = s0 + q * hop;
      const size_t at = at0 + (size_t)min(s, ns - 1) * stride;
      ml[q] = *reinterpret_cast<const floatx2*>(w.part_ml + 2 * at);
      v[q] = *reinterpret_cast<const floatx4*>(w.part_o + at * hd + 4 * d);
      if (s >= ns) ml[q] = floatx2{-INFINITY, 0.0f};
    }
    float mn = t.m;
#pragma unroll
    for (int q = 0; q < 4; ++q) mn = fmaxf(mn, ml[q][0]);
    const float ms = mn == -INFINITY ? 0.0f : mn;
    const float f0 = __builtin_amdgcn_exp2f(t.m - ms);
    t.l *= f0;
    t.acc *= f0;
    t.m = mn;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float f = __builtin_amdgcn_exp2f(ml[q][0] - ms);
      if (f != 0.0f) {                            // (a range behind the last has weight 0, whatever lies there)
        t.l += ml[q][1] * f;
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
  __shared__ float gm[GR], gl[GR];
  const int d = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const size_t stride = (size_t)w.unit * (16 * RT), base = ((size_t)rq.x * w.unit + rest) * (16 * RT);
  auto finish = [&](int r, const Joined& t) {
    const int R = rb * 16 * RT + r;
    const size_t at = (size_t)(q0 + R / w.G) * a.nh + kvh * w.G + R % w.G;
    const float inv = t.l == 0.0f ? 0.0f : 1.0f / t.l;
    uint2 pk = make_uint2(0u, 0u);
    if (t.l != 0.0f) pk = make_uint2(pack_bf16x2(t.acc[0] * inv, t.acc[1] * inv), pack_bf16x2(t.acc[2] * inv, t.acc[3] * inv));
    *reinterpret_cast<uint2*>(a.out + at * HD + 4 * d) = pk;
    if (a.lse && d == 0) a.lse[at] = row_lse(t.m, t.l);
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
    }
    __syncthreads();
    if (grp == 0) {
      t.m = -INFINITY;
#pragma unroll
      for (int q = 0; q < GR; ++q) t.m = fmaxf(t.m, gm[q]);
      const float ms = t.m == -INFINITY ? 0.0f : t.m;
      t.l = 0.0f;
      t.acc = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < GR; ++q) {
        const float f = __builtin_amdgcn_exp2f(gm[q] - ms);
        t.l += gl[q] * f;
        t.acc += part[q][d] * f;
      }
      finish(r, t);
    }
  }
}

struct Shape {
  int RT, RB, G, unit, target, pid_cap;
  size_t off_o, off_ml, off_req, bytes;
};

Shape shape_of(int B, int max_q, int nh, int nkv, int hd) {
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  Shape s;
  s.G = nh / nkv;
  const int rows = max_q * s.G;
  s.RT = rows <= 64 ? (rows + 15) / 16 : 8;
  s.RB = (rows + 16 * s.RT - 1) / (16 * s.RT);
  s.unit = nkv * s.RB;
  // Items aimed at: whole rounds of the workgroups that fit the card at once (`slots`), less
  // the half range that every request adds on average.
  const int slots = kCus * (s.RT == 1 || s.RT == 8 || hd > 128 ? 2 : 3), pairs = B * s.unit;
  s.target = std::max(slots / 2, (pairs / slots + 1) * slots - pairs / 2);
  // a split request has more keys than a range, so its ranges are fewer than twice its
  // keys over the range's length, and all of them together at most 2 target / unit
  s.pid_cap = 2 * (s.target / s.unit + 1) + 1;
  s.off_req = 0;
  s.off_ml = al((size_t)B * sizeof(int2));
  s.off_o = s.off_ml + al((size_t)s.pid_cap * s.unit * 16 * s.RT * 2 * sizeof(float));
  s.bytes = s.off_o + al((size_t)s.pid_cap * s.unit * 16 * s.RT * hd * sizeof(float));
  return s;
}

template <int HD, int RT, bool kSlots>
hipError_t launch_rows(const Work& w, int grid, hipStream_t stream) {
#ifndef STREAM_FROM
#define STREAM_FROM 2
#endif
  if constexpr (RT >= STREAM_FROM) {
    constexpr int lds = shared_lds<HD>();
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&paged_shared<HD, RT, kSlots>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((paged_shared<HD, RT, kSlots>), dim3(grid), dim3(64 * RT), lds, stream, w);
  } else {
    hipLaunchKernelGGL((paged_rows<HD, RT, kSlots>), dim3(grid), dim3(64 * NW), 0, stream, w);
  }
  return hipGetLastError();
}

template <int HD, int RT>
hipError_t launch(const Work& w, int64_t items, int max_kv, hipStream_t stream) {
  const int grid = (int)items;
  const hipError_t e = w.a.page_shift < 4 ? launch_rows<HD, RT, true>(w, grid, stream) : launch_rows<HD, RT, false>(w, grid, stream);
  if (e != hipSuccess || max_kv <= kMinChunk) return e;
  const int rows = std::min(16 * RT, w.a.max_q * w.G);
  const int step = std::max(1, std::min(rows, (int)((int64_t)w.a.B * w.unit * rows / kJoinGroups)));
  hipLaunchKernelGGL((paged_join<HD, RT>), dim3(w.a.B * w.unit, (rows + step - 1) / step), dim3(256), 0, stream, w, step);
  return hipGetLastError();
}

template <int HD>
hipError_t launch_rt(const Work& w, int RT, int64_t items, int max_kv, hipStream_t stream) {
  switch (RT) {
    case 1: return launch<HD, 1>(w, items, max_kv, stream);
    case 2: return launch<HD, 2>(w, items, max_kv, stream);
    case 3: return launch<HD, 3>(w, items, max_kv, stream);
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
  w.target = s.target;
  w.pid_cap = s.pid_cap;
  w.c = a.scale * kLog2e;
  char* base = static_cast<char*>(workspace);
  w.req = reinterpret_cast<int2*>(base + s.off_req);
  w.part_ml = reinterpret_cast<float*>(base + s.off_ml);
  w.part_o = reinterpret_cast<float*>(base + s.off_o);
  // at most one range per request, plus the ones the balancing adds
  const int max_kv = a.width << a.page_shift;
  const int64_t most = (int64_t)a.B * s.unit * std::max(1, (max_kv + kMinChunk - 1) / kMinChunk);
  const int64_t items = std::min(most, (int64_t)a.B * s.unit + s.target + s.unit);
  switch (hd) {
    case 64: return launch_rt<64>(w, s.RT, items, max_kv, stream);
    case 128: return launch_rt<128>(w, s.RT, items, max_kv, stream);
    case 256: return launch_rt<256>(w, s.RT, items, max_kv, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dspark
