// Eight consecutive elements of a row in registers: bf16 (one 16-byte
// access) or fp32 (two), converted to fp32 for arithmetic.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"

namespace fas {
namespace vec {

struct Bf16 {
  uint4 a;
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
  // Rounds to nearest even; x becomes what is stored.
  __device__ __forceinline__ void set(float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = ptx::pack_bf16x2(x[2 * e], x[2 * e + 1]);
    a = make_uint4(w[0], w[1], w[2], w[3]);
    get(x);
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = a;
  }
};

struct F32 {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    a = p[0];
    b = p[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = a;
    p[1] = b;
  }
};

}  // namespace vec
}  // namespace fas
