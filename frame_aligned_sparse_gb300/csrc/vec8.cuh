// Eight consecutive elements of a row in registers: bf16 (one 16-byte
// access) or fp32 (two), converted to fp32 pairs for packed arithmetic (two
// fp32 lanes an instruction, sm_100 family).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"

namespace fas {
namespace vec {

// A pair of fp32 values in one 64-bit register.
struct P2 {
  uint64_t v;
};
__device__ __forceinline__ P2 pair(float lo, float hi) { return {ptx::f32x2(lo, hi)}; }
__device__ __forceinline__ P2 both(float x) { return pair(x, x); }
__device__ __forceinline__ float lo(P2 a) { return __uint_as_float((uint32_t)a.v); }
__device__ __forceinline__ float hi(P2 a) { return __uint_as_float((uint32_t)(a.v >> 32)); }
__device__ __forceinline__ P2 fma2(P2 a, P2 b, P2 c) {
  P2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ P2 mul2(P2 a, P2 b) {
  P2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float sum(P2 a) { return lo(a) + hi(a); }

struct Bf16 {
  uint4 a;
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
  }
  __device__ __forceinline__ void get(P2 (&x)[4]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pair(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void set(const P2 (&x)[4]) {  // nearest even
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = ptx::pack_bf16x2(lo(x[e]), hi(x[e]));
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = a;
  }
};

struct F32 {
  float4 a, b;
  // Two 16-byte accesses leave half of each 32-byte sector to the other; one
  // of 32 bytes, where the address allows it, asks L2 once.
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const float* p = static_cast<const float*>(base) + i;
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w), "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                   : "l"(p));
    } else {
      a = reinterpret_cast<const float4*>(p)[0];
      b = reinterpret_cast<const float4*>(p)[1];
    }
  }
  __device__ __forceinline__ void get(P2 (&x)[4]) const {
    x[0] = pair(a.x, a.y);
    x[1] = pair(a.z, a.w);
    x[2] = pair(b.x, b.y);
    x[3] = pair(b.z, b.w);
  }
  __device__ __forceinline__ void set(const P2 (&x)[4]) {
    a = make_float4(lo(x[0]), hi(x[0]), lo(x[1]), hi(x[1]));
    b = make_float4(lo(x[2]), hi(x[2]), lo(x[3]), hi(x[3]));
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    float* p = static_cast<float*>(base) + i;
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(a.x), "f"(a.y), "f"(a.z),
                   "f"(a.w), "f"(b.x), "f"(b.y), "f"(b.z), "f"(b.w)
                   : "memory");
    } else {
      reinterpret_cast<float4*>(p)[0] = a;
      reinterpret_cast<float4*>(p)[1] = b;
    }
  }
};

}  // namespace vec
}  // namespace fas
