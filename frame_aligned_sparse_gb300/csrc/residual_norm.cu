// The norms around a block, its gate and its residual, in one pass over the
// data, and their backward pass.
//
// For token n of frame f with a block's output y, the residual stream x, and
// the width C (RMS norms as in the prologue):
//   r_y = 1 / sqrt(mean(y^2) + eps)       x' = x + alpha gate_f (y r_y gamma_post)
//   r_x = 1 / sqrt(mean(x'^2) + eps)      h  = x' r_x gamma_pre
// With yh = y r_y, xh = x' r_x and the gradients dx' and dh:
//   a = dh gamma_pre                      g  = dx' + r_x (a - xh mean(a xh)),  dx = g
//   b = alpha gate_f g gamma_post         dy = r_y (b - yh mean(b yh))
//   Z_f = sum_{n in f} yh g               dgate_f    = alpha gamma_post Z_f
//   dgamma_pre = sum_n dh xh              dgamma_post = sum_f alpha gate_f Z_f
// so both gradients through the post norm need only the frames' sums Z_f.
//
// A row belongs to a group of W warps, eight columns (V times) a thread, so
// a row's values stay in registers from its load to its stores, and the two
// row sums are warp shuffles and one exchange through shared memory each.
// Both kernels are bound by HBM.  Groups are persistent over consecutive
// rows: gamma and gate stay in registers, the next row is loaded while the
// current one is reduced.
//
// Backward: a group's rows never cross frames, so it adds its columns of Z
// and of dgamma_pre in registers and writes one partial row of each at its
// end; a second kernel adds the partials frame by frame and then frame after
// frame, in a fixed order (no atomics on values: results are
// bit-reproducible).

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "checkpoint.cuh"
#include "kernels.h"
#include "vec8.cuh"

namespace fas {
namespace {

constexpr int kMaxGroups = 8;   // row groups per CTA (named barriers 1 .. 8)
constexpr int kMaxWarps = 16;   // warps per row

// Frame of a row and first row of a frame: uniform spans, or a table passed
// with the launch's arguments (no device copy to keep alive).
struct Uniform {
  int64_t span;
  __device__ __forceinline__ int frame(int64_t row) const { return (int)(row / span); }
  __device__ __forceinline__ int64_t end(int f) const { return (f + 1) * span; }
};
struct Ragged {
  int n;
  int32_t start[kNormMaxFrames + 1];
  __device__ __forceinline__ int frame(int64_t row) const {
    int lo = 0, hi = n - 1;  // the last frame that starts at or before row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= row) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  __device__ __forceinline__ int64_t end(int f) const { return start[f + 1]; }
};

// Sum over the W warps of the row group; `slot` alternates so that one
// barrier a sum is enough (a slot is written again two sums later).
__device__ __forceinline__ float group_sum(float v, float (*red)[kMaxWarps], int slot, int warps, int w, int lane,
                                           int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  if (lane == 0) red[slot][w] = v;
  ptx::named_barrier_sync(1 + group, warps * 32);
  float s = 0.f;
  for (int i = 0; i < warps; ++i) s += red[slot][i];
  return s;
}

template <class R, int V, bool kCkpt, class Frames>
__global__ void __launch_bounds__(32 * kMaxWarps)
    residual_norm_fwd(const NormArgs a, const __grid_constant__ Frames frames) {
  __shared__ float red[kMaxGroups][4][kMaxWarps];
  const int W = a.warps, G = a.groups;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int group = warp / W, w = warp % W;
  const int C = a.width;
  const int64_t ngroups = (int64_t)gridDim.x * G, gi = (int64_t)blockIdx.x * G + group;
  const int64_t r0 = a.rows * gi / ngroups, r1 = a.rows * (gi + 1) / ngroups;
  const float inv_c = 1.0f / (float)C;
  int col[V];
  bool in[V];
  float gpost[V][8], gpre[V][8], coef[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = (v * W * 32 + w * 32 + lane) * 8;
    in[v] = col[v] < C;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      gpost[v][e] = in[v] ? a.gamma_post[col[v] + e] * a.alpha : 0.f;
      gpre[v][e] = in[v] ? a.gamma_pre[col[v] + e] : 0.f;
      coef[v][e] = gpost[v][e];
    }
  }
  vec::Bf16 yv[V];
  R xv[V];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (in[v]) {
        yv[v].load(a.y, r * C + col[v]);
        xv[v].load(a.x, r * C + col[v]);
      }
  };
#pragma unroll
  for (int v = 0; v < V; ++v) {
    yv[v] = vec::Bf16{};
    xv[v] = R{};
  }
  if (r0 < r1) load(r0);
  int64_t frame_end = a.gate ? -1 : a.rows;
  int slot = 0;
  for (int64_t r = r0; r < r1; ++r) {
    float y[V][8], x[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      yv[v].get(y[v]);
      xv[v].get(x[v]);
    }
    if (r + 1 < r1) load(r + 1);
    if (r >= frame_end) {
      const int f = frames.frame(r);
      frame_end = frames.end(f);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (in[v])
#pragma unroll
          for (int e = 0; e < 8; ++e) coef[v][e] = gpost[v][e] * a.gate[(int64_t)f * C + col[v] + e];
    }
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[v][e], y[v][e], ss);
    const float ry = rsqrtf(group_sum(ss, red[group], slot, W, w, lane, group) * inv_c + a.eps);
    float sx = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[v][e] = fmaf(y[v][e] * ry, coef[v][e], x[v][e]);
        sx = fmaf(x[v][e], x[v][e], sx);
      }
    const float rx = rsqrtf(group_sum(sx, red[group], slot + 1, W, w, lane, group) * inv_c + a.eps);
    slot ^= 2;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t at = r * C + col[v];
      float h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = x[v][e] * rx * gpre[v][e];
      vec::Bf16 hv;
      R ov;
      hv.set(h);
      ov.set(x[v]);  // x becomes what is stored: the checkpoint is of that
      if (in[v]) {
        hv.store(a.h, at);
        ov.store(a.x_out, at);
      }
      if constexpr (kCkpt) {
        uint32_t by, bx;
        const uint2 cy = ckpt::encode8(y[v], by), cx = ckpt::encode8(x[v], bx);
        if (in[v]) {
          *reinterpret_cast<uint2*>(a.y8 + at) = cy;
          *reinterpret_cast<uint2*>(a.x8 + at) = cx;
          if ((lane & 3) == 0) {
            a.y8_scale[at / ckpt::kBlock] = (uint8_t)by;
            a.x8_scale[at / ckpt::kBlock] = (uint8_t)bx;
          }
        }
      }
    }
    if (w == 0 && lane == 0) {
      a.rstd[r] = ry;
      a.rstd[a.rows + r] = rx;
    }
  }
}

// Backward items: item i covers `chunk` rows (fewer at the end) of one frame.
struct UniformItems {
  int64_t span;
  int per_frame;
  __device__ __forceinline__ int frame(int64_t item) const { return (int)(item / per_frame); }
  __device__ __forceinline__ int64_t first(int f) const { return (int64_t)f * per_frame; }
  __device__ __forceinline__ int64_t start(int f) const { return f * span; }
  __device__ __forceinline__ int64_t end(int f) const { return (f + 1) * span; }
};
struct RaggedItems {
  int n;
  int32_t row[kNormMaxFrames + 1], item[kNormMaxFrames + 1];
  __device__ __forceinline__ int frame(int64_t i) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (item[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  __device__ __forceinline__ int64_t first(int f) const { return item[f]; }
  __device__ __forceinline__ int64_t start(int f) const { return row[f]; }
  __device__ __forceinline__ int64_t end(int f) const { return row[f + 1]; }
};

// y and x' of one thread's eight columns, 16 bits (or fp32 x') or 8 bits.
template <class R, bool k8>
struct Held;
template <class R>
struct Held<R, false> {
  vec::Bf16 y;
  R x;
  __device__ __forceinline__ void load(const NormArgs& a, int64_t at) {
    y.load(a.y, at);
    x.load(a.x, at);
  }
  __device__ __forceinline__ void get(float (&yf)[8], float (&xf)[8]) const {
    y.get(yf);
    x.get(xf);
  }
};
template <class R>
struct Held<R, true> {
  uint2 y, x;
  uint32_t b;
  __device__ __forceinline__ void load(const NormArgs& a, int64_t at) {
    y = *reinterpret_cast<const uint2*>(a.y8 + at);
    x = *reinterpret_cast<const uint2*>(a.x8 + at);
    b = a.y8_scale[at / ckpt::kBlock] | (uint32_t)a.x8_scale[at / ckpt::kBlock] << 8;
  }
  __device__ __forceinline__ void get(float (&yf)[8], float (&xf)[8]) const {
    ckpt::decode8(y, b & 255u, yf);
    ckpt::decode8(x, b >> 8, xf);
  }
};

template <class R, int V, bool k8, class Items>
__global__ void __launch_bounds__(32 * kMaxWarps) residual_norm_bwd(const NormArgs a, const __grid_constant__ Items items) {
  __shared__ float red[kMaxGroups][4][kMaxWarps];
  const int W = a.warps, G = a.groups;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int group = warp / W, w = warp % W;
  const int C = a.width;
  const float inv_c = 1.0f / (float)C;
  // The second kernel's counters (one per column block) start at zero.
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.counters; i += blockDim.x) a.counter[i] = 0u;
  const int64_t item = (int64_t)blockIdx.x * G + group;
  if (item >= a.items) return;  // whole groups: the group's barrier is its own
  const int f = items.frame(item);
  const int64_t r0 = items.start(f) + (item - items.first(f)) * a.chunk;
  const int64_t r1 = min(r0 + a.chunk, items.end(f));
  int col[V];
  bool in[V];
  float coef[V][8], gpre[V][8], z[V][8], dg[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = (v * W * 32 + w * 32 + lane) * 8;
    in[v] = col[v] < C;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      coef[v][e] = in[v] ? a.gamma_post[col[v] + e] * a.alpha : 0.f;
      if (in[v] && a.gate) coef[v][e] *= a.gate[(int64_t)f * C + col[v] + e];
      gpre[v][e] = in[v] ? a.gamma_pre[col[v] + e] : 0.f;
      z[v][e] = dg[v][e] = 0.f;
    }
  }
  vec::Bf16 hv[V];
  R gv[V];
  Held<R, k8> held[V];
  float ry, rx;
  auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (in[v]) {
        const int64_t at = r * C + col[v];
        gv[v].load(a.dx_out, at);
        hv[v].load(a.dh, at);
        held[v].load(a, at);
      }
    ry = a.rstd[r];
    rx = a.rstd[a.rows + r];
  };
#pragma unroll
  for (int v = 0; v < V; ++v) {
    gv[v] = R{};
    hv[v] = vec::Bf16{};
    held[v] = Held<R, k8>{};
  }
  if (r0 < r1) load(r0);
  int slot = 0;
  for (int64_t r = r0; r < r1; ++r) {
    float y[V][8], x[V][8], g[V][8], h[V][8];
    const float ryc = ry, rxc = rx;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      held[v].get(y[v], x[v]);
      gv[v].get(g[v]);
      hv[v].get(h[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[v][e] *= ryc;
        x[v][e] *= rxc;
        dg[v][e] = fmaf(h[v][e], x[v][e], dg[v][e]);
        h[v][e] *= gpre[v][e];
        s = fmaf(h[v][e], x[v][e], s);
      }
    }
    if (r + 1 < r1) load(r + 1);
    const float m1 = group_sum(s, red[group], slot, W, w, lane, group) * inv_c;
    float s2 = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[v][e] = fmaf(rxc, fmaf(-x[v][e], m1, h[v][e]), g[v][e]);
        z[v][e] = fmaf(y[v][e], g[v][e], z[v][e]);
        s2 = fmaf(g[v][e] * coef[v][e], y[v][e], s2);
      }
    const float m2 = group_sum(s2, red[group], slot + 1, W, w, lane, group) * inv_c;
    slot ^= 2;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (in[v]) {
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = ryc * fmaf(-y[v][e], m2, g[v][e] * coef[v][e]);
        vec::Bf16 dv;
        R ov;
        dv.set(d);
        ov.set(g[v]);
        const int64_t at = r * C + col[v];
        dv.store(a.dy, at);
        ov.store(a.dx, at);
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (in[v]) {
      vec::F32 o;
      o.set(z[v]);
      o.store(a.z_part, item * C + col[v]);
      o.set(dg[v]);
      o.store(a.d_part, item * C + col[v]);
    }
}

// Adds the partials: CTA (column block, frame) sums its frame's items, 8
// lanes of items by 32 columns; the last CTA of a column block to arrive
// (a counter) then adds the frames in order.
constexpr int kSumCols = 32, kSumLanes = 8;

template <class Items>
__global__ void __launch_bounds__(kSumCols* kSumLanes)
    residual_norm_sums(const NormArgs a, const __grid_constant__ Items items, int n_frames) {
  __shared__ float red[2][kSumLanes][kSumCols];
  __shared__ bool last;
  const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols;
  const int c = blockIdx.y * kSumCols + tx, f = blockIdx.x, C = a.width;
  const bool in = c < C;
  auto reduce = [&](float z, float d) {
    __syncthreads();
    red[0][ty][tx] = z;
    red[1][ty][tx] = d;
    __syncthreads();
  };
  float z = 0.f, d = 0.f;
  const int64_t i1 = f + 1 < n_frames ? items.first(f + 1) : a.items;
  if (in)
    for (int64_t i = items.first(f) + ty; i < i1; i += kSumLanes) {
      z += a.z_part[i * C + c];
      d += a.d_part[i * C + c];
    }
  reduce(z, d);
  const float post = in ? a.gamma_post[c] : 0.f;
  if (ty == 0 && in) {
    z = d = 0.f;
    for (int l = 0; l < kSumLanes; ++l) {
      z += red[0][l][tx];
      d += red[1][l][tx];
    }
    if (a.gate) a.dgate[(int64_t)f * C + c] = a.alpha * post * z;
    a.z_frame[(int64_t)f * C + c] = a.gate ? a.alpha * a.gate[(int64_t)f * C + c] * z : a.alpha * z;
    a.d_frame[(int64_t)f * C + c] = d;
    __threadfence();
  }
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(&a.counter[blockIdx.y], 1u) == (unsigned)n_frames - 1u;
  __syncthreads();
  if (!last) return;
  __threadfence();
  z = d = 0.f;
  if (in)
    for (int g = ty; g < n_frames; g += kSumLanes) {
      z += __ldcg(a.z_frame + (int64_t)g * C + c);
      d += __ldcg(a.d_frame + (int64_t)g * C + c);
    }
  reduce(z, d);
  if (ty == 0 && in) {
    z = d = 0.f;
    for (int l = 0; l < kSumLanes; ++l) {
      z += red[0][l][tx];
      d += red[1][l][tx];
    }
    a.dgamma_post[c] = z;
    a.dgamma_pre[c] = d;
  }
}

// Warps per row and vectors per thread for a width.
struct Shape {
  int V, W, G;
};
Shape shape_of(int width) {
  const int vecs = width / 8;
  const int V = vecs <= 32 * kMaxWarps ? 1 : vecs <= 64 * kMaxWarps ? 2 : 4;
  const int W = (vecs + 32 * V - 1) / (32 * V);
  return {V, W, std::max(1, kMaxGroups / W)};
}

// Row groups that run at once for a kernel of `threads` a CTA on the device.
template <class K>
int64_t resident_groups(K kern, const Shape& s, int sms) {
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, 32 * s.W * s.G, 0) != cudaSuccess || per_sm < 1)
    return 0;
  return (int64_t)per_sm * sms * s.G;
}

template <class R, int V, bool kCkpt, class Frames>
cudaError_t fwd(NormArgs a, const Frames& fr, const Shape& s, int sms, cudaStream_t st) {
  auto kern = residual_norm_fwd<R, V, kCkpt, Frames>;
  const int64_t res = resident_groups(kern, s, sms);
  if (res == 0) return cudaErrorInvalidConfiguration;
  const int64_t groups = std::min(a.rows, res);
  kern<<<(unsigned)((groups + s.G - 1) / s.G), 32 * s.W * s.G, 0, st>>>(a, fr);
  return cudaGetLastError();
}

template <class R, int V, class Frames>
cudaError_t fwd_c(const NormArgs& a, const Frames& fr, const Shape& s, int sms, cudaStream_t st) {
  return a.y8 ? fwd<R, V, true>(a, fr, s, sms, st) : fwd<R, V, false>(a, fr, s, sms, st);
}
template <class Frames>
cudaError_t fwd_all(const NormArgs& a, const Frames& fr, const Shape& s, int sms, cudaStream_t st) {
  if (s.V == 1) return a.f32 ? fwd_c<vec::F32, 1>(a, fr, s, sms, st) : fwd_c<vec::Bf16, 1>(a, fr, s, sms, st);
  if (s.V == 2) return a.f32 ? fwd_c<vec::F32, 2>(a, fr, s, sms, st) : fwd_c<vec::Bf16, 2>(a, fr, s, sms, st);
  return a.f32 ? fwd_c<vec::F32, 4>(a, fr, s, sms, st) : fwd_c<vec::Bf16, 4>(a, fr, s, sms, st);
}

template <class R, int V, bool k8, class Items>
cudaError_t bwd(const NormArgs& a, const Items& it, const Shape& s, cudaStream_t st) {
  residual_norm_bwd<R, V, k8, Items>
      <<<(unsigned)((a.items + s.G - 1) / s.G), 32 * s.W * s.G, 0, st>>>(a, it);
  return cudaGetLastError();
}
template <class R, int V, class Items>
cudaError_t bwd_c(const NormArgs& a, const Items& it, const Shape& s, cudaStream_t st) {
  return a.y8 ? bwd<R, V, true>(a, it, s, st) : bwd<R, V, false>(a, it, s, st);
}
template <class Items>
cudaError_t bwd_all(const NormArgs& a, const Items& it, int n_frames, const Shape& s, cudaStream_t st) {
  cudaError_t e;
  if (s.V == 1)
    e = a.f32 ? bwd_c<vec::F32, 1>(a, it, s, st) : bwd_c<vec::Bf16, 1>(a, it, s, st);
  else if (s.V == 2)
    e = a.f32 ? bwd_c<vec::F32, 2>(a, it, s, st) : bwd_c<vec::Bf16, 2>(a, it, s, st);
  else
    e = a.f32 ? bwd_c<vec::F32, 4>(a, it, s, st) : bwd_c<vec::Bf16, 4>(a, it, s, st);
  if (e != cudaSuccess) return e;
  residual_norm_sums<Items><<<dim3((unsigned)n_frames, (unsigned)a.counters), kSumCols * kSumLanes, 0, st>>>(a, it,
                                                                                                         n_frames);
  return cudaGetLastError();
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_residual_norm(NormArgs a, const int32_t* spans, int n_frames, int64_t span, int sms,
                                 cudaStream_t st) {
  const Shape s = shape_of(a.width);
  a.warps = s.W;
  a.groups = s.G;
  if (!spans) return fwd_all(a, Uniform{span}, s, sms, st);
  Ragged fr;
  fr.n = n_frames;
  fr.start[0] = 0;
  for (int f = 0; f < n_frames; ++f) fr.start[f + 1] = fr.start[f] + spans[f];
  return fwd_all(a, fr, s, sms, st);
}

// Rows per item: about one item per group that runs at once (kItemGroups a
// SM), and never across frames.  Depends on the shape and the device alone.
constexpr int kItemGroupsPerSm = 2;

NormItems residual_norm_items(int64_t rows, int width, const int32_t* spans, int n_frames, int64_t span, int sms) {
  const Shape s = shape_of(width);
  const int64_t want = std::max<int64_t>(n_frames, (int64_t)kItemGroupsPerSm * sms * s.G);
  auto count = [&](int64_t chunk) {
    if (!spans) return (int64_t)n_frames * ((span + chunk - 1) / chunk);
    int64_t n = 0;
    for (int f = 0; f < n_frames; ++f) n += (spans[f] + chunk - 1) / chunk;
    return n;
  };
  int64_t lo = 1, hi = rows;  // the smallest chunk with at most `want` items
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (count(mid) <= want) hi = mid; else lo = mid + 1;
  }
  NormItems r;
  r.chunk = lo;
  r.items = count(lo);
  r.counters = (width + kSumCols - 1) / kSumCols;
  const int64_t part = align256(r.items * width * 4), frame = align256((int64_t)n_frames * width * 4);
  r.bytes = 2 * part + 2 * frame + align256((int64_t)r.counters * 4);
  return r;
}

cudaError_t launch_residual_norm_backward(NormArgs a, const NormItems& n, const int32_t* spans, int n_frames,
                                          int64_t span, void* workspace, cudaStream_t st) {
  const Shape s = shape_of(a.width);
  a.warps = s.W;
  a.groups = s.G;
  a.items = n.items;
  a.chunk = n.chunk;
  a.counters = n.counters;
  const int64_t part = align256(n.items * a.width * 4), frame = align256((int64_t)n_frames * a.width * 4);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.z_part = reinterpret_cast<float*>(ws);
  a.d_part = reinterpret_cast<float*>(ws + part);
  a.z_frame = reinterpret_cast<float*>(ws + 2 * part);
  a.d_frame = reinterpret_cast<float*>(ws + 2 * part + frame);
  a.counter = reinterpret_cast<unsigned int*>(ws + 2 * part + 2 * frame);
  if (!spans) return bwd_all(a, UniformItems{span, (int)((span + n.chunk - 1) / n.chunk)}, n_frames, s, st);
  RaggedItems it;
  it.n = n_frames;
  it.row[0] = it.item[0] = 0;
  for (int f = 0; f < n_frames; ++f) {
    it.row[f + 1] = it.row[f] + spans[f];
    it.item[f + 1] = it.item[f] + (int32_t)((spans[f] + n.chunk - 1) / n.chunk);
  }
  return bwd_all(a, it, n_frames, s, st);
}

}  // namespace fas
