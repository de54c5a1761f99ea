// Rotary positions with several axes, applied on the way from a projection's
// output to the attention's q, k and v, and taken back on the way of their
// gradients.
//
// Token n sits at position p[n, a] on axis a (frame, row, column, ...).  Each
// of a head's d/2 pairs belongs to one axis and turns by angle = p[n, axis] f:
//   (a, b) -> (a cos - b sin, a sin + b cos)
// The turn is orthogonal, so the gradient's way back is the opposite turn.
//
// A thread owns eight pairs (two 16-byte vectors) of one token and keeps
// their cosines and sines in registers over the heads of its tensor: an angle
// is computed once per token, pair and tensor, not once per head, and nothing
// goes through shared memory.  Angles of far positions: the frequency is held
// in turns (f / 2 pi) as a pair of fp32 numbers, the product's whole turns are
// taken off exactly (one fma gives the rounding error of the product) and the
// rest goes to sincospif, which has no argument reduction left to do.  An
// angle of t turns is off by about 2^-47 t turns plus fp32's rounding of the
// remaining fraction.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "ptx.cuh"

namespace fas {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // heads whose loads are in flight at once

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight pairs, whose elements are eight of `x` with eight of `y` (halves) or
// neighbours in x, then in y.
template <bool kHalf>
__device__ __forceinline__ void turn(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
  uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
  if constexpr (kHalf) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a0 = bf16_lo(u[e]), a1 = bf16_hi(u[e]), b0 = bf16_lo(w[e]), b1 = bf16_hi(w[e]);
      u[e] = ptx::pack_bf16x2(a0 * c[2 * e] - b0 * s[2 * e], a1 * c[2 * e + 1] - b1 * s[2 * e + 1]);
      w[e] = ptx::pack_bf16x2(fmaf(a0, s[2 * e], b0 * c[2 * e]), fmaf(a1, s[2 * e + 1], b1 * c[2 * e + 1]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = bf16_lo(u[e]), b = bf16_hi(u[e]);
      u[e] = ptx::pack_bf16x2(a * c[e] - b * s[e], fmaf(a, s[e], b * c[e]));
      a = bf16_lo(w[e]), b = bf16_hi(w[e]);
      w[e] = ptx::pack_bf16x2(a * c[4 + e] - b * s[4 + e], fmaf(a, s[4 + e], b * c[4 + e]));
    }
  }
  x = make_uint4(u[0], u[1], u[2], u[3]);
  y = make_uint4(w[0], w[1], w[2], w[3]);
}

// The same where only the first n of the eight pairs turn: the others keep
// their bits (a turn by zero would not: infinity times the sine is NaN).
template <bool kHalf>
__device__ __forceinline__ void turn(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8], int n) {
  const uint4 x0 = x, y0 = y;
  turn<kHalf>(x, y, c, s);
  if (n == 8) return;
  uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
  const uint32_t u0[4] = {x0.x, x0.y, x0.z, x0.w}, w0[4] = {y0.x, y0.y, y0.z, y0.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (kHalf) {  // pairs 2 e and 2 e + 1 in the halves of both
      const uint32_t turned = (2 * e < n ? 0x0000FFFFu : 0u) | (2 * e + 1 < n ? 0xFFFF0000u : 0u);
      u[e] = (u[e] & turned) | (u0[e] & ~turned);
      w[e] = (w[e] & turned) | (w0[e] & ~turned);
    } else {  // pair e in x, pair 4 + e in y
      if (e >= n) u[e] = u0[e];
      if (4 + e >= n) w[e] = w0[e];
    }
  }
  x = make_uint4(u[0], u[1], u[2], u[3]);
  y = make_uint4(w[0], w[1], w[2], w[3]);
}

// Grid: x over tokens, y over (tensor, run of heads).
template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads) rotary(const __grid_constant__ RotaryParams p) {
  constexpr int kPieces = D / 16;
  const int piece = threadIdx.x % kPieces;
  const int64_t token = (int64_t)blockIdx.x * (kThreads / kPieces) + threadIdx.x / kPieces;
  if (token >= p.tokens) return;
  const int runs = gridDim.y / p.tensors;
  const int tensor = blockIdx.y / runs, run = blockIdx.y % runs;
  const int per = (p.heads + runs - 1) / runs;
  const int h0 = run * per, h1 = min(p.heads, h0 + per);
  const RotaryTensor& t = p.t[tensor];
  const int second = kHalf ? D / 2 : 8;
  const int at = piece * (kHalf ? 8 : 16);
  const uint16_t* in = t.in + token * t.in_token + h0 * t.in_head + at;
  uint16_t* out = t.out + token * t.out_token + h0 * t.out_head + at;
  float c[8], s[8];
  const int pairs = t.turned ? min(8, p.pairs - piece * 8) : 0;  // that turn (0 or less: none)
  if (pairs > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = piece * 8 + e;
      const float pos = p.positions[token * p.axes + p.axis[i]], f = p.turns[i];
      const float whole = pos * f;
      const float rest = fmaf(pos, p.turns_low[i], fmaf(pos, f, -whole));
      sincospif(2.f * ((whole - rintf(whole)) + rest), &s[e], &c[e]);
      s[e] *= p.sign;
    }
  }
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 x[kUnroll], y[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (h + k < h1) {
        x[k] = *reinterpret_cast<const uint4*>(in + k * t.in_head);
        y[k] = *reinterpret_cast<const uint4*>(in + k * t.in_head + second);
      }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (h + k < h1) {
        if (pairs > 0) turn<kHalf>(x[k], y[k], c, s, pairs);
        *reinterpret_cast<uint4*>(out + k * t.out_head) = x[k];
        *reinterpret_cast<uint4*>(out + k * t.out_head + second) = y[k];
      }
    in += kUnroll * t.in_head;
    out += kUnroll * t.out_head;
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int head_dim, bool half, int sms, cudaStream_t stream) {
  const int64_t rows = kThreads / (head_dim / 16);
  const int64_t blocks = (p.tokens + rows - 1) / rows;
  // Runs of heads: all of a tensor's in one where the tokens alone fill the
  // GPU several times over, fewer otherwise (14,960 tokens of 16 heads: 62 us
  // in runs of 16, 59 in runs of 8, 60 in runs of 4).
  int runs = 1;
  while (blocks * p.tensors * runs < (int64_t)sms * 16 && runs * kUnroll < p.heads) runs *= 2;  // at most 1024
  const dim3 grid((unsigned)blocks, (unsigned)(p.tensors * runs));
  auto go = [&](auto kern) {
    kern<<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  };
  if (head_dim == 128) return half ? go(rotary<128, true>) : go(rotary<128, false>);
  return half ? go(rotary<64, true>) : go(rotary<64, false>);
}

}  // namespace fas
