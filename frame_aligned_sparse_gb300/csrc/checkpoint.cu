// Packing a tensor into an 8-bit checkpoint and back (format: checkpoint.cuh).
// Both are one pass over the data, bound by HBM: 16 or 32 bytes in and 8 out
// per thread (or the reverse) and a byte per four threads.

#include <cuda_runtime.h>
#include <stdint.h>

#include "checkpoint.cuh"
#include "kernels.h"
#include "vec8.cuh"

namespace fas {
namespace {

constexpr int kThreadsC = 256;
constexpr int kPerThread = 4;  // vectors of eight a thread: enough bytes in flight to cover HBM's latency

template <class X>
__global__ void __launch_bounds__(kThreadsC) checkpoint_pack(const void* __restrict__ x, uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales, int64_t vecs) {
  const int64_t i0 = blockIdx.x * (int64_t)(kThreadsC * kPerThread) + threadIdx.x;
  X v[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int64_t i = i0 + k * kThreadsC;
    v[k] = X{};
    if (i < vecs) v[k].load(x, i * 8);
  }
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int64_t i = i0 + k * kThreadsC;
    vec::P2 f[4];
    v[k].get(f);
    uint32_t b;
    const uint2 c = ckpt::encode8(f, b);
    if (i < vecs) {
      *reinterpret_cast<uint2*>(codes + i * 8) = c;
      if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
    }
  }
}

template <class X>
__global__ void __launch_bounds__(kThreadsC) checkpoint_unpack(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, void* __restrict__ x,
                                                               int64_t vecs) {
  const int64_t i0 = blockIdx.x * (int64_t)(kThreadsC * kPerThread) + threadIdx.x;
  uint2 c[kPerThread];
  uint32_t b[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int64_t i = i0 + k * kThreadsC;
    if (i < vecs) {
      c[k] = *reinterpret_cast<const uint2*>(codes + i * 8);
      b[k] = scales[i >> 2];
    }
  }
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int64_t i = i0 + k * kThreadsC;
    if (i >= vecs) break;
    vec::P2 f[4];
    ckpt::decode8(c[k], b[k], f);
    X v;
    v.set(f);
    v.store(x, i * 8);
  }
}

int64_t blocks_of(int64_t vecs) { return (vecs + kThreadsC * kPerThread - 1) / (kThreadsC * kPerThread); }

}  // namespace

cudaError_t launch_checkpoint_pack(const void* x, bool f32, uint8_t* codes, uint8_t* scales, int64_t n,
                                   cudaStream_t st) {
  const int64_t vecs = n / 8, blocks = blocks_of(vecs);
  if (f32)
    checkpoint_pack<vec::F32><<<(unsigned)blocks, kThreadsC, 0, st>>>(x, codes, scales, vecs);
  else
    checkpoint_pack<vec::Bf16><<<(unsigned)blocks, kThreadsC, 0, st>>>(x, codes, scales, vecs);
  return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(const uint8_t* codes, const uint8_t* scales, void* x, bool f32, int64_t n,
                                     cudaStream_t st) {
  const int64_t vecs = n / 8, blocks = blocks_of(vecs);
  if (f32)
    checkpoint_unpack<vec::F32><<<(unsigned)blocks, kThreadsC, 0, st>>>(codes, scales, x, vecs);
  else
    checkpoint_unpack<vec::Bf16><<<(unsigned)blocks, kThreadsC, 0, st>>>(codes, scales, x, vecs);
  return cudaGetLastError();
}

}  // namespace fas
