// Appending a layer's new tokens to the key-value cache, with the head norms and the
// rotation applied on the way.  For token m and head h of q or k:
//   x = x / sqrt(mean_i x_i^2 + eps) * w                      (where w is given)
//   for i < hd/2 the pair (x_i, x_{i+hd/2}) turned by positions[m] * theta^(-2i/hd)
// k and v then go to slot slots[m] of the caches, q to q_out, k (if asked for) to k_out.
//
// One workgroup per token.  Its first hd/2 threads form the token's angles once (every
// head shares them) while the loads of the heads are in flight; a head is hd/16 lanes,
// each holding the eight pairs i = 8c .. 8c+7 of it, so a pair never leaves its lane
// and a head's sum of squares is a butterfly over hd/16 neighbouring lanes.  Every byte
// moves once: 8192 tokens with 32/8 heads of 128 and packed rotated keys, 218 MB in 44 us,
// 4.9 TB/s, the rate of a plain copy; 9 tokens take 4 us, the time of a launch.
#include "device.hpp"
#include "kernels.hpp"

namespace dspark {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// eight floats to bf16, round to nearest even: the one rounding of every output
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{f[2 * k], f[2 * k + 1]}), bf16x2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int HD>
__global__ __launch_bounds__(512) void kv_append_rows(AppendArgs a) {
  constexpr int LPH = HD / 16;              // lanes per head
  __shared__ float cs[HD / 2], sn[HD / 2];
  const int m = blockIdx.x;
  const int64_t slot = a.slots[m];
  const bool in_cache = slot >= 0 && slot < a.num_slots;
  if (threadIdx.x < HD / 2) {
    // the angle in turns, reduced to half a turn in double, so that far positions keep
    // the accuracy of near ones; sine and cosine of the remainder in float
    const double turns = (double)a.positions[m] *
                         (exp2(-2.0 * (double)threadIdx.x / (double)HD * a.log2_theta) * 0.15915494309189533577);
    const float r = (float)(2.0 * (turns - rint(turns)));
    float s, c;
    sincospif(r, &s, &c);
    cs[threadIdx.x] = c;
    sn[threadIdx.x] = s;
  }
  __syncthreads();
  const int c = threadIdx.x % LPH;
  const int heads = a.nh + 2 * a.nkv;
  for (int hh = threadIdx.x / LPH; hh < heads; hh += blockDim.x / LPH) {
    if (hh >= a.nh + a.nkv) {               // a head of v: copied
      if (!in_cache) continue;
      const int h = hh - a.nh - a.nkv;
      const uint4* src = reinterpret_cast<const uint4*>(a.v + (size_t)m * a.v_stride + (size_t)h * HD);
      uint4* dst = reinterpret_cast<uint4*>(a.v_cache + ((size_t)slot * a.nkv + h) * HD);
      dst[c] = src[c];
      dst[c + LPH] = src[c + LPH];
      continue;
    }
    const bool isq = hh < a.nh;
    const int h = isq ? hh : hh - a.nh;
    const uint16_t* src = isq ? a.q + (size_t)m * a.q_stride + (size_t)h * HD
                              : a.k + (size_t)m * a.k_stride + (size_t)h * HD;
    const uint16_t* w = isq ? a.qnorm_w : a.knorm_w;
    float x[8], y[8];
    unpack8(reinterpret_cast<const uint4*>(src)[c], x);
    unpack8(reinterpret_cast<const uint4*>(src)[c + LPH], y);
    if (w) {
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], fmaf(y[k], y[k], ss));
      ss = group_sum(ss, LPH);
      const float inv = 1.0f / sqrtf(ss / (float)HD + a.eps);
      float wx[8], wy[8];
      unpack8(reinterpret_cast<const uint4*>(w)[c], wx);
      unpack8(reinterpret_cast<const uint4*>(w)[c + LPH], wy);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = x[k] * inv * wx[k];
        y[k] = y[k] * inv * wy[k];
      }
    }
    float lo[8], hi[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float co = cs[8 * c + k], si = sn[8 * c + k];
      lo[k] = x[k] * co - y[k] * si;
      hi[k] = y[k] * co + x[k] * si;
    }
    const uint4 plo = pack8(lo), phi = pack8(hi);
    if (isq) {
      uint4* dst = reinterpret_cast<uint4*>(a.q_out + (size_t)m * a.q_out_stride + (size_t)h * HD);
      dst[c] = plo;
      dst[c + LPH] = phi;
      continue;
    }
    if (a.k_out) {
      uint4* dst = reinterpret_cast<uint4*>(a.k_out + (size_t)m * a.k_out_stride + (size_t)h * HD);
      dst[c] = plo;
      dst[c + LPH] = phi;
    }
    if (in_cache) {
      uint4* dst = reinterpret_cast<uint4*>(a.k_cache + ((size_t)slot * a.nkv + h) * HD);
      dst[c] = plo;
      dst[c + LPH] = phi;
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, int M, int hd, hipStream_t stream) {
  if (M <= 0) return hipSuccess;
  const int lanes = (a.nh + 2 * a.nkv) * (hd / 16);
  const int threads = lanes >= 512 ? 512 : lanes <= 128 ? 128 : (lanes + 63) / 64 * 64;
  switch (hd) {
    case 32: hipLaunchKernelGGL(kv_append_rows<32>, dim3(M), dim3(threads), 0, stream, a); break;
    case 64: hipLaunchKernelGGL(kv_append_rows<64>, dim3(M), dim3(threads), 0, stream, a); break;
    case 128: hipLaunchKernelGGL(kv_append_rows<128>, dim3(M), dim3(threads), 0, stream, a); break;
    case 256: hipLaunchKernelGGL(kv_append_rows<256>, dim3(M), dim3(threads), 0, stream, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace dspark
