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

constexpr uint32_t kInfBits = 0x7F800000u;

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
// block is the four lanes 4i .. 4i + 3.  Magnitudes are compared as integers,
// which orders finite ones below infinity and NaN, so a warp learns from the
// maximum whether it holds any that are not finite.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
__device__ __forceinline__ uint2 encode8(const vec::P2 (&p)[4], uint32_t& byte) {
  vec::P2 x[4];
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = p[e];
    m = max(m, max((uint32_t)x[e].v & 0x7FFFFFFFu, (uint32_t)(x[e].v >> 32) & 0x7FFFFFFFu));
  }
  uint32_t amax = block_max(m);
  if (__any_sync(0xffffffffu, amax >= kInfBits)) {
    m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t lo = (uint32_t)x[e].v, hi = (uint32_t)(x[e].v >> 32);
      if ((lo & 0x7FFFFFFFu) >= kInfBits) lo = 0x7FC00000u; else m = max(m, lo & 0x7FFFFFFFu);
      if ((hi & 0x7FFFFFFFu) >= kInfBits) hi = 0x7FC00000u; else m = max(m, hi & 0x7FFFFFFFu);
      x[e] = vec::pair(__uint_as_float(lo), __uint_as_float(hi));
    }
    amax = block_max(m);
  }
  byte = scale_byte(__uint_as_float(amax));
  const vec::P2 inv = vec::both(inv_scale_of(byte));
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const vec::P2 y = vec::mul2(x[e], inv);
    c[e] = encode2(vec::lo(y), vec::hi(y));
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
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
