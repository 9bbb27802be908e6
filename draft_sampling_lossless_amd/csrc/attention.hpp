// Building blocks of the two attention kernels: bf16 packing, loads into LDS, transposing
// LDS reads, wave-uniform values.
#pragma once

#include "device.hpp"

namespace dspark {

typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short shortx4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// two floats to packed bf16, round to nearest even (one instruction on gfx950)
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{a, b}), bf16x2));
}

// c + the two bf16 of a pair, in float.  The output divides by the sum of the weights as
// they are multiplied, rounded: a row that one key dominates then keeps that key's value
// exactly, whatever its weight was rounded to.  The log-sum-exp takes the unrounded sum.
__device__ __forceinline__ float add_bf16x2(uint32_t w, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, 0x3F803F80u), c, false);
}

// transposing LDS read: the 16 lanes of a quarter wave name four rows of 16 bf16 (lane i
// the 8 bytes i % 4 of row i / 4); lane i gets column i of them, four values
typedef __attribute__((address_space(3))) shortx4 lds_shortx4;
__device__ __forceinline__ shortx4 lds_read_tr(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4*)p);
}

// global -> LDS without registers: lane i's 16 bytes at base + off go to LDS byte address
// lds + 16 i (base and lds uniform).  Written in assembly because the compiler otherwise
// makes every later LDS read wait for every such load; the callers wait themselves
// (s_waitcnt vmcnt, then a barrier) before a buffer is read.  It has no register result.
// The compiler warns that it does not keep m0 across the statement: it has nothing there, LDS
// instructions of gfx950 do not read m0, and nothing else in the kernels that use this writes it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds16(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
// the same with an address of its own for every lane
__device__ __forceinline__ void load_to_lds16(const char* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// A wave-uniform value as a scalar.  MFMA instructions ignore the execution mask, so a
// branch around one has to be a scalar branch: its condition goes through here.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The least power of two that is not below c (c normal, below 2^127)
__device__ __forceinline__ float power_above(float c) {
  return __uint_as_float((__float_as_uint(c) + 0x7FFFFFu) & 0x7F800000u);
}

// The factor of a row's scores, given its maximum: c = scale * log2 e, but the power of two
// above it where the maximum passes 2^30 in magnitude.  score * c - maximum is one fused
// operation against the rounded maximum, whose half unit in the last place is the exponent of
// the largest weight: up to 32 below 2^30, without bound beyond.  There scores that differ at
// all differ by 64 and more, so that any factor near c leaves the same weights, and a power of
// two makes the maximum exact.  As it is not below c, a maximum of the one factor and one of
// the other compare as their scores do, and lie 64 and more apart: a row that changes its
// factor, and waves and ranges of different factors, are rescaled and joined as if there were one.
__device__ __forceinline__ float row_factor(float top, float c) {
  return fabsf(top * c) < 0x1p30f ? c : power_above(c);
}

// log(sum exp) of a row from its base-2 maximum, which is in units of row_factor's, and sum;
// -inf for a row that saw nothing
__device__ __forceinline__ float row_lse(float m, float l, float c) {
  if (fabsf(m) >= 0x1p30f) m *= c / power_above(c);
  return l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : l == 0.0f ? -INFINITY : l;
}

}  // namespace dspark
