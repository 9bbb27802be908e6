// Attention over whole packed prompts, causal or full, with grouped heads.
//
//   out[r] = sum_s exp2(x_rs - m_r) v_s / sum_s exp2(x_rs - m_r),   x_rs = q_r . k_s * scale * log2 e
//
// in one pass over a sequence's keys with a running maximum and sum.  The rows of a
// product are (token, head) pairs of one kv head, token-major: the nh / nkv heads that
// share keys share their tiles too.  A workgroup takes 32 NW rows, a wave 32, and keys
// and values pass through LDS in tiles of 64 tokens.
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

constexpr int KT = 64;   // keys per tile

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

// the sequence and row tile of item u; every wave finds them for itself
__device__ bool find_tile(const Work& w, int u, int rows, int& start, int& n, int& tile) {
  const PromptArgs& a = w.a;
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < a.B; base += 64) {
    int s = 0, len = 0, cnt = 0;
    if (base + lane < a.B) {
      sequence(a, base + lane, s, len);
      cnt = (int)(((int64_t)len * w.G + rows - 1) / rows);
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
      tile = before + __builtin_amdgcn_readlane(inc, q) - 1 - u;   // a sequence's last tile first
      return true;
    }
    before += __builtin_amdgcn_readlane(inc, 63);
  }
  return false;
}

template <int HD, int NW, bool kCausal>
__global__ __launch_bounds__(64 * NW) void prompt_rows(Work w) {
  constexpr int PIECES = HD / 8;            // 16-byte pieces of a row
  constexpr int ROWB = HD * 2;
  const PromptArgs& a = w.a;
  __shared__ __attribute__((aligned(16))) char kbuf[KT * ROWB];
  __shared__ __attribute__((aligned(16))) char vbuf[KT * ROWB];

  const int kvh = blockIdx.x % a.nkv;
  int start, n, tile;
  if (!find_tile(w, blockIdx.x / a.nkv, 32 * NW, start, n, tile)) return;
  const int lane = threadIdx.x & 63, col = lane & 31, hh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r0 = tile * 32 * NW;            // first row of the workgroup
  const int row = r0 + 32 * wave + col;
  const int j = row / w.G, h = kvh * w.G + row % w.G;
  const bool ok = j < n;
  const int lim = kCausal && ok ? j + 1 : n;                     // keys below lim are seen
  const int wlow = kCausal ? min(n, (r0 + 32 * wave) / w.G + 1) : n;       // the wave's smallest limit
  const int whigh = kCausal ? min(n, (r0 + 32 * wave + 31) / w.G + 1) : n; // and its largest
  const int ghigh = kCausal ? min(n, (r0 + 32 * NW - 1) / w.G + 1) : n;
  const bool idle = (r0 + 32 * wave) / w.G >= n;                 // no row of this wave exists

  bf16x8 qf[HD / 16];
  {
    const uint16_t* src = a.q + (size_t)(start + (ok ? j : 0)) * a.q_stride + (size_t)(ok ? h : 0) * HD;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 16 * kk + 8 * hh);
      qf[kk] = __builtin_bit_cast(bf16x8, ok ? v : make_uint4(0, 0, 0, 0));
    }
  }
  floatx16 o[HD / 32];
#pragma unroll
  for (int d = 0; d < HD / 32; ++d) o[d] = floatx16{};
  float m = -INFINITY, l = 0.0f;

  for (int key0 = 0; key0 < ghigh; key0 += KT) {
    __syncthreads();
    // stage: LDS slot q of the tile (row q / PIECES) takes the piece swizzled into it;
    // a key behind the sequence reads its last row
#pragma unroll
    for (int q = 0; q < KT * PIECES / (64 * NW); ++q) {
      const int blk = q * NW + wave, slot = blk * 64 + lane;
      const int r = slot / PIECES, piece = (slot % PIECES) ^ (swizzle<HD>(r));
      const size_t t = start + min(key0 + r, n - 1);
      load_to_lds16(a.k + t * a.k_stride + (size_t)kvh * HD + piece * 8, kbuf + blk * 1024);
      load_to_lds16(a.v + t * a.v_stride + (size_t)kvh * HD + piece * 8, vbuf + blk * 1024);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (uniform(idle || key0 >= whigh)) continue;

    floatx16 sc[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      sc[s] = floatx16{};
      const int r = 32 * s + col;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(kbuf + r * ROWB + (((2 * kk + hh) ^ swizzle<HD>(r)) << 4));
        sc[s] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[kk], sc[s], 0, 0, 0);
      }
    }
    const bool partial = uniform(key0 + KT > wlow) != 0;
    float x[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = sc[e >> 4][e & 15] * w.c;
    if (partial) {
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int i = 32 * (e >> 4) + 8 * ((e & 15) >> 2) + 4 * hh + (e & 3);
        if (key0 + i >= lim) x[e] = -INFINITY;
      }
    }
    float tm = x[0];
#pragma unroll
    for (int e = 1; e < 32; ++e) tm = fmaxf(tm, x[e]);
    {
      uint32_t lo, hi;
      halves_pair(__float_as_uint(tm), lo, hi);
      tm = fmaxf(__uint_as_float(lo), __uint_as_float(hi));
    }
    const float mn = fmaxf(m, tm);
    const float ms = mn == -INFINITY ? 0.0f : mn;     // a row that has seen nothing yet
    const float al = __builtin_amdgcn_exp2f(m - ms);
    m = mn;
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      x[e] = __builtin_amdgcn_exp2f(x[e] - ms);
      sum += x[e];
    }
    l = l * al + sum;
    // the weights' rounding to bf16, the second product's operand type
    bf16x8 p[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      p[u] = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16x2(x[8 * u], x[8 * u + 1]), pack_bf16x2(x[8 * u + 2], x[8 * u + 3]),
                                                   pack_bf16x2(x[8 * u + 4], x[8 * u + 5]), pack_bf16x2(x[8 * u + 6], x[8 * u + 7])));
    if (__any(al != 1.0f)) {
#pragma unroll
      for (int d = 0; d < HD / 32; ++d) o[d] *= al;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int d = 0; d < HD / 32; ++d) {
        // keys 16 u + 4 hh .. + 3 and 8 more on, dim 32 d + col
        union {
          shortx4 s[2];
          uint32_t w[4];
          bf16x8 v;
        } vt;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * u + 8 * e + 4 * hh + ((lane & 15) >> 2);
          const int dim = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
          const char* at = vbuf + r * ROWB + (((dim >> 3) ^ swizzle<HD>(r)) << 4) + ((dim & 4) << 1);
          vt.s[e] = lds_read_tr(at);
        }
        int odd = 0;
        if (partial) {
          // in a tile some row does not see whole, a value that is not finite must not
          // meet that row's zero weight
          const bool any =
              bf16x2_nonfinite(vt.w[0]) || bf16x2_nonfinite(vt.w[1]) || bf16x2_nonfinite(vt.w[2]) ||
                bf16x2_nonfinite(vt.w[3]);
          odd = __any(any);
        }
        odd = uniform(odd);
        if (!odd) {
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vt.v, p[u], o[d], 0, 0, 0);
        } else {
          // key by key, added only to the rows that see it
          for (int k = 0; k < 16; ++k) {
            const int jj = (k & 3) | ((k >> 3) << 2);
            const uint32_t half = jj & 1 ? 0xFFFF0000u : 0x0000FFFFu;
            const bool mine = hh == ((k >> 2) & 1);
            const bf16x8 one = __builtin_bit_cast(
                bf16x8, make_uint4(mine && jj / 2 == 0 ? vt.w[0] & half : 0u, mine && jj / 2 == 1 ? vt.w[1] & half : 0u,
                                   mine && jj / 2 == 2 ? vt.w[2] & half : 0u, mine && jj / 2 == 3 ? vt.w[3] & half : 0u));
            const floatx16 add = __builtin_amdgcn_mfma_f32_32x32x16_bf16(one, p[u], floatx16{}, 0, 0, 0);
            if (key0 + 16 * u + k < lim) o[d] += add;
          }
        }
      }
    }
  }

  {
    uint32_t lo, hi;
    halves_pair(__float_as_uint(l), lo, hi);
    l = __uint_as_float(lo) + __uint_as_float(hi);
  }
  if (!ok) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t at = (size_t)(start + j) * a.nh + h;
#pragma unroll
  for (int d = 0; d < HD / 32; ++d)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint2*>(a.out + at * HD + 32 * d + 8 * q + 4 * hh) =
          l == 0.0f ? make_uint2(0u, 0u)
                    : make_uint2(pack_bf16x2(o[d][4 * q] * inv, o[d][4 * q + 1] * inv),
                                 pack_bf16x2(o[d][4 * q + 2] * inv, o[d][4 * q + 3] * inv));
  if (a.lse && hh == 0) a.lse[at] = row_lse(m, l);
}

template <int HD, int NW>
hipError_t launch(const Work& w, hipStream_t stream) {
  const PromptArgs& a = w.a;
  const int64_t tiles = ((int64_t)a.T * w.G + 32 * NW - 1) / (32 * NW) + a.B;
  const dim3 grid((unsigned)(tiles * a.nkv));
  if (a.causal)
    hipLaunchKernelGGL((prompt_rows<HD, NW, true>), grid, dim3(64 * NW), 0, stream, w);
  else
    hipLaunchKernelGGL((prompt_rows<HD, NW, false>), grid, dim3(64 * NW), 0, stream, w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prompt_attention(const PromptArgs& a, int hd, hipStream_t stream) {
  Work w;
  w.a = a;
  w.G = a.nh / a.nkv;
  w.c = a.scale * kLog2e;
  switch (hd) {
    case 64: return launch<64, 4>(w, stream);
    case 128: return launch<128, 4>(w, stream);
    case 256: return launch<256, 4>(w, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dspark
