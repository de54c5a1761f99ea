// The 8-bit checkpoint format: blocks of 32 consecutive elements of a row,
// each e4m3 codes under one power of two.
//
// The block's scale is 2^(b - 127), b one byte: the smallest power of two
// that brings the block's largest finite magnitude to at most 448 (e4m3's
// largest value), or 2^-127 when that is smaller still.  Dividing by a power
// of two is exact, so an element is rounded once, to the nearest code (ties
// to even): off by at most half a step, 2^-4 of the value for normal codes.
// The largest element never saturates.  Elements that are not finite become
// NaN codes and take no part in the scale.
//
// Eight consecutive elements per thread, four neighbouring lanes per block.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fas.h"
#include "vec8.cuh"

namespace fas {
namespace ckpt {

constexpr int kBlock = FAS_CHECKPOINT_BLOCK;

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// The scale byte for a block whose largest finite magnitude is amax = m 2^E
// (1 <= m < 2): 448 = 1.75 * 2^8, so the power is E - 8, or E - 7 for m > 1.75.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return b > 0 ? (uint32_t)b : 0u;
}

// 2^(b - 127) and its inverse (b <= 247 for finite blocks).
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }
__device__ __forceinline__ float inv_scale_of(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Two e4m3 codes (x0 in the low byte), nearest even.
__device__ __forceinline__ uint32_t encode2(float x0, float x1) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}

// This lane's eight elements of a block as codes (first element in the low
// byte) and the block's scale byte.  All lanes of the warp take part; the
// block is the four lanes 4i .. 4i + 3.
__device__ __forceinline__ uint2 encode8(const vec::P2 (&p)[4], uint32_t& byte) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = vec::lo(p[e]);
    x[2 * e + 1] = vec::hi(p[e]);
  }
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite(x[e]) ? fabsf(x[e]) : 0.f);
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  byte = scale_byte(amax);
  const float inv = inv_scale_of(byte);
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = finite(x[e]) ? x[e] * inv : __uint_as_float(0x7FC00000u);
  return make_uint2(encode2(y[0], y[1]) | encode2(y[2], y[3]) << 16, encode2(y[4], y[5]) | encode2(y[6], y[7]) << 16);
}

// The eight values that codes c under the scale byte stand for (exact).
__device__ __forceinline__ void decode8(uint2 c, uint32_t byte, vec::P2 (&x)[4]) {
  const vec::P2 s = vec::both(scale_of(byte));
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i >> 1] >> ((i & 1) * 16))));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h2));
    x[i] = vec::mul2(vec::pair(lo, hi), s);
  }
}

}  // namespace ckpt
}  // namespace fas
