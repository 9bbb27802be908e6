// Attention over whole packed prompts, causal or full, with grouped heads.
//
//   out[r] = sum_s exp2(x_rs - m_r) v_s / sum_s exp2(x_rs - m_r),   x_rs = q_r . k_s * scale * log2 e
//
// in one pass over a sequence's keys with a running maximum and sum.  The rows of a
// product are (token, head) pairs of one kv head, token-major: the nh / nkv heads that
// share keys share their tiles too.  A workgroup takes 32 NW rows, a wave 32, and keys
// and values pass through LDS in tiles of KT tokens.  One causal prompt of 8192 tokens, 32/8
// heads of 128: 530 to 565 us by the machine, 1040 to 975 TFLOP/s (1100 to 1015 without the
// mask), bound by the matrix pipe and the exponentials and packing beside it; short sequences
// by their loads and stores.
//
// Scores are formed transposed, S^T = K Q^T, with v_mfma_f32_32x32x16_bf16: lane
// (h, n) = (lane / 32, lane % 32) holds row n and the keys 8 (i / 4) + 4 h + i % 4 of
// each 32.  Rounded to bf16, eight of them are the B operand of O^T = V^T P^T as they
// stand, if V's operand takes its keys in the same order: two transposing LDS reads of
// four keys each.  LDS rows are permuted by 16-byte pieces (piece p of row r lies at
// p ^ swizzle(r)) so that both the K reads (16 rows, one piece) and the V reads (4 rows,
// four pieces) touch every bank once.
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

// 32 rows a wave.  One pass of the loop holds the weights of tile t and the scores of tile
// t + 1 at once, so that the first product of the next tile (matrix pipe) runs beside the
// exponentials of this one (vector pipe).  K is read one tile ahead of V; four LDS buffers
// of K and two of V are filled straight from memory while the others are in use, with one
// barrier a tile.  The running maximum is raised only when a row's scores exceed it by
// kRaise (weights up to 2^kRaise, more where the maximum itself is rounded by more than that,
// which neither float nor bf16 minds): the accumulators are rescaled on a row's first tile and
// hardly ever after.
constexpr float kRaise = 8.0f;

template <int HD, int NW, int KT, bool kCausal, bool kLse>
__global__ __launch_bounds__(64 * NW, HD > 128 ? 1 : 2) void prompt_rows(Work w) {
  constexpr int SB = KT / 32, UG = KT / 16; // score blocks of a tile of KT keys, its groups of 16 keys
  constexpr int PIECES = HD / 8;            // 16-byte pieces of a row
  constexpr int ROWB = HD * 2;
  constexpr int TILEB = KT * ROWB;
  constexpr int WGROWS = 32 * NW;
  constexpr int LOADS = KT * PIECES / (64 * NW);   // 1 KB loads of a wave for one tile of K (or V)
  const PromptArgs& a = w.a;
  extern __shared__ __attribute__((aligned(16))) char smem[];   // four K tiles, two V tiles

  const int kvh = blockIdx.x % a.nkv;
  int start, n, tile;
  if (!find_tile(w, blockIdx.x / a.nkv, WGROWS, start, n, tile)) return;
  const int lane = threadIdx.x & 63, col = lane & 31, hh = lane >> 5;
  const int wave = uniform(threadIdx.x >> 6);
  const int r0 = tile * WGROWS, w0 = r0 + 32 * wave;        // first row of the workgroup, of the wave
  const int ghigh = kCausal ? min(n, (r0 + WGROWS - 1) / w.G + 1) : n;
  const int nt = (ghigh + KT - 1) / KT;
  // tiles every row of the wave sees whole, and tiles some row sees at all
  const int wlow = kCausal ? min(n, w0 / w.G + 1) : n;
  const int whigh = w0 / w.G >= n ? 0 : kCausal ? min(n, (w0 + 31) / w.G + 1) : n;
  const int nsome = (whigh + KT - 1) / KT, nfull = min(wlow / KT, nsome);

  const int row = w0 + col, row_j = row / w.G, row_h = kvh * w.G + row % w.G;
  const bool ok = row_j < n;
  const int lim = kCausal && ok ? row_j + 1 : n;                 // keys below lim are seen

  // LDS slot q of a tile (row q / PIECES) takes the piece swizzled into it.  The tile's
  // base is a scalar, a lane's offset into it 32 bits (token strides stay below 2^24); a
  // key behind the sequence reads its last row
  uint32_t koffs[LOADS], voffs[LOADS];
#pragma unroll
  for (int q = 0; q < LOADS; ++q) {
    const int slot = (q * NW + wave) * 64 + lane, r = slot / PIECES, piece = (slot % PIECES) ^ swizzle<HD>(r);
    koffs[q] = (uint32_t)r * (uint32_t)(a.k_stride * 2) + piece * 16;
    voffs[q] = (uint32_t)r * (uint32_t)(a.v_stride * 2) + piece * 16;
  }
  // the tile that the sequence ends in: its offsets are cut once, before its load
  auto cut = [&](uint32_t (&offs)[LOADS], int64_t stride, int t) {
#pragma unroll
    for (int q = 0; q < LOADS; ++q) {
      const int r = ((q * NW + wave) * 64 + lane) / PIECES, over = max(r - (n - 1 - t * KT), 0);
      offs[q] -= (uint32_t)over * (uint32_t)(stride * 2);
    }
  };
  auto fetch_one = [&](const uint16_t* base, int64_t stride, const uint32_t (&offs)[LOADS], int t, char* lds, int q) {
    const char* tb = reinterpret_cast<const char*>(base + (size_t)t * KT * stride);
    load_to_lds16(tb, offs[q], uniform(lds_address(lds) + (q * NW + wave) * 1024));
  };
  auto fetch = [&](const uint16_t* base, int64_t stride, uint32_t (&offs)[LOADS], int t, char* lds) {
    if (uniform((t + 1) * KT > n)) cut(offs, stride, t);
#pragma unroll
    for (int q = 0; q < LOADS; ++q) fetch_one(base, stride, offs, t, lds, q);
  };
  const uint16_t* kbase = a.k + (size_t)start * a.k_stride + (size_t)kvh * HD;
  const uint16_t* vbase = a.v + (size_t)start * a.v_stride + (size_t)kvh * HD;

  // K tile t lies in buffer t % 4, V tile t in buffer t % 2; during tile t the loads of
  // K t + 3 and V t + 1 are in flight
  char* const vbuf = smem + 4 * TILEB;
  auto kbuf_of = [&](int t) { return smem + (t & 3) * TILEB; };
  auto vbuf_of = [&](int t) { return vbuf + (t & 1) * TILEB; };
  fetch(kbase, a.k_stride, koffs, 0, kbuf_of(0));
  if (nt > 1) fetch(kbase, a.k_stride, koffs, 1, kbuf_of(1));
  if (nt > 2) fetch(kbase, a.k_stride, koffs, 2, kbuf_of(2));
  fetch(vbase, a.v_stride, voffs, 0, vbuf_of(0));
  bf16x8 qf[HD / 16];
  {
    const uint16_t* src = a.q + (size_t)(start + (ok ? row_j : 0)) * a.q_stride + (size_t)(ok ? row_h : 0) * HD;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 16 * kk + 8 * hh);
      qf[kk] = __builtin_bit_cast(bf16x8, ok ? v : make_uint4(0, 0, 0, 0));
    }
  }

  floatx16 o[HD / 32];
  // m: running maximum, in units of the row's factor rc; mb: m, or 0 while a row has seen
  // nothing; lx: l of unrounded weights
  float m = -INFINITY, mb = 0.0f, l = 0.0f, lx = 0.0f, rc = w.c;
#pragma unroll
  for (int d = 0; d < HD / 32; ++d) o[d] = floatx16{};

  // K operand kk of 32 rows: this lane's row, piece 2 kk + hh; the swizzle repeats every 16
  // rows, so the second 32 rows are a constant further, and kk only flips bits
  int koff = col * ROWB + ((hh ^ swizzle<HD>(col)) << 4);
  auto key_frag = [&](const char* kb, int s, int kk) {
    return *reinterpret_cast<const bf16x8*>(kb + ((koff ^ (kk << 5)) + 32 * s * ROWB));
  };
  auto scores = [&](floatx16 (&sc)[SB], const char* kb, int keys) {   // of blocks that begin below `keys`
#pragma unroll
    for (int s = 0; s < SB; ++s) {
      sc[s] = floatx16{};
      if (s > 0 && uniform(32 * s >= keys)) continue;
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
  auto mask = [&](floatx16 (&sc)[SB], int t) {
#pragma unroll
    for (int s = 0; s < SB; ++s)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (t * KT + 32 * s + 8 * (e >> 2) + 4 * hh + (e & 3) >= lim) sc[s][e] = -INFINITY;
  };
  // raise the maxima that tile t's scores exceed by too much
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
  // weights of keys 16 u .. 16 u + 15 of the tile, rounded to bf16 (the second product's
  // operand type), and their sum
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
  union VFrag {
    shortx4 s[2];
    uint32_t w[4];
    bf16x8 v;
  };
  // V operand (u, d): keys 16 u + 8 e + 4 hh .. + 3 (e = 0, 1), dim 32 d + col
  int voff[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 8 * e + 4 * hh + ((lane & 15) >> 2), dim = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    voff[e] = r * ROWB + (((dim >> 3) ^ swizzle<HD>(r)) << 4) + ((dim & 4) << 1);
  }
  auto value_frag = [&](const char* vb, int u, int d) {
    VFrag f;
#pragma unroll
    for (int e = 0; e < 2; ++e) f.s[e] = lds_read_tr(vb + ((voff[e] ^ (d << 6)) + 16 * u * ROWB));
    return f;
  };

  int t = 0;
  auto open_tile = [&]() {                  // tile t: its operands have landed, its buffers-to-be are free
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };
  // keeps the flipped offsets out of registers across the loop: they are one instruction
  auto fresh = [&]() { asm volatile("" : "+v"(koff), "+v"(voff[0]), "+v"(voff[1])); };

  // tiles that every row of the wave sees whole: cur holds tile t's scores, nxt takes the
  // next tile's (of no use after the last).  Four groups of the first product and UG of
  // the second, each with its operands read one group ahead (the first group's before the
  // barrier) and an equal share of the vector work
  constexpr int KG = SB * (HD / 16) / 4, DH = HD > 128 ? 2 : 1, VG = HD / 32 / DH, OG = UG * DH;
  bf16x8 kf[2][KG];
  auto step = [&](floatx16 (&cur)[SB], floatx16 (&nxt)[SB]) {
    open_tile();
    if (uniform((t + 4) * KT > n && t + 3 < nt)) cut(koffs, a.k_stride, t + 3);
    if (uniform((t + 2) * KT > n && t + 1 < nt)) cut(voffs, a.v_stride, t + 1);
    fresh();
    const char* kb = kbuf_of(t + 1);
    const char* vb = vbuf_of(t);
    uint32_t p[UG][4];
    float tm = 0.0f;
    VFrag vf[2][VG];
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
      // the loads to come, spread over the tile: all at once they would hold up every wave
      if (uniform(t + 3 < nt)) {
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
          if (q * 4 / LOADS == gq) fetch_one(kbase, a.k_stride, koffs, t + 3, kbuf_of(t + 3), q);
      }
    }
#pragma unroll
    for (int gq = 0; gq < OG; ++gq) {
      const int u = gq / DH, d0 = gq % DH * VG;
      if (gq < OG - 1) {
#pragma unroll
        for (int i = 0; i < VG; ++i) vf[(gq + 1) & 1][i] = value_frag(vb, (gq + 1) / DH, (gq + 1) % DH * VG + i);
      } else {
#pragma unroll
        for (int i = 0; i < KG; ++i) kf[0][i] = key_frag(kbuf_of(t + 2), i % SB, i / SB);
      }
      if (UG > 2 && u == 0) {
        weights(cur, 2, 0, p[2]);
        weights(cur, 2, 1, p[2]);
      } else if (UG > 2 && u < 3) {
        weights(cur, 3, u - 1, p[3]);
      }
      if (gq == OG - 1) tm = row_max(nxt);
#pragma unroll
      for (int i = 0; i < VG; ++i)
        o[d0 + i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[gq & 1][i].v, as_frag(p[u]), o[d0 + i], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (uniform(t + 1 < nt)) {
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
          if (q * OG / LOADS == gq) fetch_one(vbase, a.v_stride, voffs, t + 1, vbuf_of(t + 1), q);
      }
    }
    ++t;
    if (uniform(t < nfull)) raise(tm);      // (the scores of a tile seen in part are formed again, masked)
  };
  floatx16 sa[SB];
  open_tile();
  if (uniform(nfull > 0)) {
    floatx16 sb[SB];
    scores(sa, kbuf_of(0), KT);
    raise(row_max(sa));
#pragma unroll
    for (int i = 0; i < KG; ++i) kf[0][i] = key_frag(kbuf_of(1), i % SB, i / SB);
    while (true) {
      step(sa, sb);
      if (uniform(t >= nfull)) break;
      step(sb, sa);
      if (uniform(t >= nfull)) break;
    }
  }
  // tiles that some row sees only in part, one product after the other; groups of keys
  // that no row of the wave sees are left out
  for (; t < nt; ++t) {
    open_tile();
    if (t + 3 < nt) fetch(kbase, a.k_stride, koffs, t + 3, kbuf_of(t + 3));
    if (t + 1 < nt) fetch(vbase, a.v_stride, voffs, t + 1, vbuf_of(t + 1));
    if (uniform(t < nsome)) {
      const char* vb = vbuf_of(t);
      scores(sa, kbuf_of(t), whigh - t * KT);
      mask(sa, t);
      raise(row_max(sa));
#pragma unroll
      for (int u = 0; u < UG; ++u) {
        const int first = t * KT + 16 * u;
        if (uniform(first >= whigh)) continue;
        VFrag f[HD / 32];
        uint32_t pw[4], top = 0;            // top: the largest exponent, in the high half
        weights(sa, u, 0, pw);
        weights(sa, u, 1, pw);
        const bf16x8 p = as_frag(pw);
#pragma unroll
        for (int d = 0; d < HD / 32; ++d) f[d] = value_frag(vb, u, d);
        if (uniform(first + 16 > wlow)) {
          // a value that is not finite must not meet the zero weight of a row that does not see it
#pragma unroll
          for (int d = 0; d < HD / 32; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t e = f[d].w[k] & 0x7F807F80u;
              top = max(top, max(e, e << 16));
            }
        }
        if (!uniform(__any(top >= 0x7F800000u))) {
#pragma unroll
          for (int d = 0; d < HD / 32; ++d) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[d].v, p, o[d], 0, 0, 0);
        } else {
          // key by key, added only to the rows that see it
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {
            const int jj = (k & 3) | ((k >> 3) << 2);
            const uint32_t half = jj & 1 ? 0xFFFF0000u : 0x0000FFFFu;
            const uint32_t keep = hh == ((k >> 2) & 1) ? half : 0u;
#pragma unroll
            for (int d = 0; d < HD / 32; ++d) {
              const bf16x8 one = __builtin_bit_cast(
                  bf16x8, make_uint4(jj / 2 == 0 ? f[d].w[0] & keep : 0u, jj / 2 == 1 ? f[d].w[1] & keep : 0u,
                                     jj / 2 == 2 ? f[d].w[2] & keep : 0u, jj / 2 == 3 ? f[d].w[3] & keep : 0u));
              const floatx16 add = __builtin_amdgcn_mfma_f32_32x32x16_bf16(one, p, floatx16{}, 0, 0, 0);
              if (first + k < lim) o[d] += add;
            }
          }
        }
      }
    }
  }

  // The rows leave through LDS, a region of this wave's own once all are done with the
  // tiles, so that a store writes whole rows.  Row r's dims 8 p + 4 h .. lie in its piece
  // p ^ (r % 16), halves exchanged in the upper 16 rows: no bank twice.
  const float lt = halves_sum(l), lxt = kLse ? halves_sum(lx) : 0.0f;
  const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
  const int at = ok ? (start + row_j) * a.nh + row_h : -1;
  if (kLse && ok && hh == 0) a.lse[at] = row_lse(m, lxt, w.c);
  __syncthreads();
  char* const mine = smem + wave * 32 * ROWB;
#pragma unroll
  for (int d = 0; d < HD / 32; ++d)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint2*>(mine + col * ROWB + ((4 * d + q) ^ (col & (PIECES < 16 ? PIECES - 1 : 15))) * 16 + (hh ^ (col >> 4)) * 8) =
          lt == 0.0f ? make_uint2(0u, 0u)
                     : make_uint2(pack_bf16x2(o[d][4 * q] * inv, o[d][4 * q + 1] * inv),
                                  pack_bf16x2(o[d][4 * q + 2] * inv, o[d][4 * q + 3] * inv));
  constexpr int RPI = 64 / PIECES;          // rows of one store
#pragma unroll
  for (int i = 0; i < 32 / RPI; ++i) {
    const int r = i * RPI + lane / PIECES, p = lane % PIECES, to = __shfl(at, r);
    uint4 v = *reinterpret_cast<const uint4*>(mine + r * ROWB + (p ^ (r & (PIECES < 16 ? PIECES - 1 : 15))) * 16);
    if (r >= 16) v = make_uint4(v.z, v.w, v.x, v.y);
    if (to >= 0) *reinterpret_cast<uint4*>(a.out + (size_t)to * HD + 8 * p) = v;
  }
}

template <int HD, int NW, int KT, bool kCausal, bool kLse>
hipError_t launch_one(const Work& w, hipStream_t stream) {
  const PromptArgs& a = w.a;
  constexpr int rows = 32 * NW, lds = 6 * KT * HD * 2;
  const int64_t tiles = ((int64_t)a.T * w.G + rows - 1) / rows + a.B;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&prompt_rows<HD, NW, KT, kCausal, kLse>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((prompt_rows<HD, NW, KT, kCausal, kLse>), dim3((unsigned)(tiles * a.nkv)), dim3(64 * NW), lds, stream, w);
  return hipGetLastError();
}

template <int HD, int NW, int KT>
hipError_t launch(const Work& w, hipStream_t stream) {
  if (w.a.lse)
    return w.a.causal ? launch_one<HD, NW, KT, true, true>(w, stream) : launch_one<HD, NW, KT, false, true>(w, stream);
  return w.a.causal ? launch_one<HD, NW, KT, true, false>(w, stream) : launch_one<HD, NW, KT, false, false>(w, stream);
}

}  // namespace

hipError_t launch_prompt_attention(const PromptArgs& a, int hd, hipStream_t stream) {
  Work w;
  w.a = a;
  w.G = a.nh / a.nkv;
  w.c = a.scale * kLog2e;
  // Workgroups of four waves, two on a compute unit, where sequences are short: one begins
  // or ends, which is memory's time, while the other multiplies.  Eight waves where they are
  // long: half the tiles to load.  32/8 heads of 128, causal, four waves against eight: 192
  // sequences of 64 59 and 76 us, 24 of 512 107 and 112, 12 of 1024 170 and 161, one of 8192
  // 611 and 536; 16/2 heads of 64: 64 of 256 35 and 36 us, one of 1024 18 and 23, two of 4096
  // 100 and 92.  Heads of 256 leave registers for four waves only.  The host knows the mean
  // length alone, and these were equal lengths: one of 8192 among 31 of some 100 takes 641 us by
  // four waves, 560 alone by eight and the others 23.
  switch (hd) {
    case 64: return a.T <= (int64_t)1024 * a.B ? launch<64, 4, 64>(w, stream) : launch<64, 8, 64>(w, stream);
    case 128: return a.T <= (int64_t)512 * a.B ? launch<128, 4, 32>(w, stream) : launch<128, 8, 64>(w, stream);
    case 256: return launch<256, 4, 32>(w, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dspark
