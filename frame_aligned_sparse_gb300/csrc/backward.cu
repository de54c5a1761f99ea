// Backward pass of the frame-aligned sparse attention.
//
// With s = 1/sqrt(d), for row i and the keys j its frame sees:
//   P_ij = exp(s q_i.k_j - lse_i)          (recomputed, lse from the forward)
//   delta_i = sum_c dout_ic out_ic         dS_ij = P_ij (dout_i.v_j - delta_i)
//   dq_i = s sum_j dS_ij k_j    dk_j = s sum_i dS_ij q_i    dv_j = sum_i P_ij dout_i
// Visibility is symmetric in the frames, so the queries that see a key frame
// are the same table ranges that the frame's own queries see.  Two kernels,
// each output row written once by one warp: no atomics, results are
// bit-reproducible.

#include <cuda_runtime.h>
#include <stdint.h>

#include "fas.h"
#include "internal.h"
#include "kernels.h"
#include "ptx.cuh"

namespace fas {
namespace {

constexpr int kWarpsB = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One lane's D / 32 consecutive elements of a bf16 row.
template <int D>
__device__ __forceinline__ void load_row(const uint16_t* p, int lane, float (&x)[D / 32]) {
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(p)[lane * (D / 64) + e];
    x[2 * e] = __uint_as_float(w << 16);
    x[2 * e + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
}
template <int D>
__device__ __forceinline__ void store_row(uint16_t* p, int lane, const float (&x)[D / 32], float scale) {
#pragma unroll
  for (int e = 0; e < D / 64; ++e)
    reinterpret_cast<uint32_t*>(p)[lane * (D / 64) + e] = ptx::pack_bf16x2(x[2 * e] * scale, x[2 * e + 1] * scale);
}

// A warp per row of the tile: query rows (kKeys false: delta and dq) or key
// rows (dk and dv), over the visible tokens of the other side.
template <int D, bool kKeys>
__global__ void __launch_bounds__(32 * kWarpsB) attention_bwd(const BwdParams p) {
  constexpr int E = D / 32;
  const int4 item = p.work[blockIdx.x];
  const int h = item.x, f = item.y;
  const int lane = threadIdx.x % 32;
  const int2 sp = p.spans[f];
  const int4 rng = p.table[f];
  const int64_t hb = (int64_t)h * p.head_stride, lb = (int64_t)h * p.N;
  for (int r = item.z * kQTile + threadIdx.x / 32; r < min((item.z + 1) * kQTile, sp.y); r += kWarpsB) {
    const int64_t row = (int64_t)sp.x + r, at = hb + row * p.row_stride;
    float a[E], b[E], g0[E] = {}, g1[E] = {};  // (q, dout) or (k, v); dq or (dk, dv)
    load_row<D>((kKeys ? p.k : p.q) + at, lane, a);
    load_row<D>((kKeys ? p.v : p.dout) + at, lane, b);
    float lse = 0.f, delta = 0.f;
    if (!kKeys) {
      float o[E];
      load_row<D>(p.out + at, lane, o);
#pragma unroll
      for (int e = 0; e < E; ++e) delta = fmaf(b[e], o[e], delta);
      delta = warp_sum(delta);
      lse = p.lse[lb + row];
      if (lane == 0) p.delta[lb + row] = delta;
    }
    for (int part = 0; part < 2; ++part) {
      const int t0 = part ? rng.z : rng.x, n = part ? rng.w : rng.y;
      for (int t = t0; t < t0 + n; ++t) {
        const int64_t ot = hb + (int64_t)t * p.row_stride;
        float c[E], e2[E];
        load_row<D>((kKeys ? p.q : p.k) + ot, lane, c);
        load_row<D>((kKeys ? p.dout : p.v) + ot, lane, e2);
        if (kKeys) {
          lse = p.lse[lb + t];
          delta = p.delta[lb + t];
        }
        float s = 0.f, dp = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          s = fmaf(a[e], c[e], s);
          dp = fmaf(b[e], e2[e], dp);
        }
        s = warp_sum(s);
        dp = warp_sum(dp);
        const float pr = __expf(s * p.scale - lse), ds = pr * (dp - delta);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          g0[e] = fmaf(ds, c[e], g0[e]);
          if (kKeys) g1[e] = fmaf(pr, e2[e], g1[e]);
        }
      }
    }
    store_row<D>((kKeys ? p.dk : p.dq) + at, lane, g0, p.scale);
    if (kKeys) store_row<D>(p.dv + at, lane, g1, 1.f);
  }
}

template <int D>
int launch(const BwdParams& p, int grid, cudaStream_t st) {
  attention_bwd<D, false><<<grid, 32 * kWarpsB, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -1;
  attention_bwd<D, true><<<grid, 32 * kWarpsB, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? 2 : -1;
}

}  // namespace

int launch_attention_backward(int d, const BwdParams& p, int grid, cudaStream_t stream) {
  if (d == 128) return launch<128>(p, grid, stream);
  if (d == 64) return launch<64>(p, grid, stream);
  return -1;
}

}  // namespace fas
