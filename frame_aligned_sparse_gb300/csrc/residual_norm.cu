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
// Everything is fp32 but the stored results, which are rounded once.
//
// A row belongs to a group of W warps, eight columns a vector and one or two
// vectors a thread (four above 8192 columns), so a row's values stay
// in registers from its arrival to its stores, and a row sum is a warp
// shuffle and one exchange through shared memory.  A group works through its
// item's rows; gamma and gate stay with it, and the next rows are on their way
// into a ring in shared memory.  Each thread copies just the bytes it will
// read itself (cp.async), so the ring needs no barrier.  (One vector a thread
// and rows prefetched into registers: twice the instructions a row, 57 us
// forward and 80 backward at 14,960 x 2048.)
//
// Bound by HBM: forward 41.5 us at 14,960 x 2048 bf16 (5.9 TB/s, 0.87 of the
// measured copy rate), backward 59 us (6.2 TB/s, 0.91) and 7 for its sums;
// 292 us (0.82) from 8-bit checkpoints at 79,200 x 2048, where decoding takes
// issue slots; device time of captured calls.
//
// Backward: a group's rows never cross frames, so it adds its columns of Z
// and of dgamma_pre in registers and writes one partial row of each at its
// end; a second kernel adds the partials frame by frame and then frame after
// frame, in a fixed order (no atomics: results are bit-reproducible).

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "checkpoint.cuh"
#include "kernels.h"
#include "vec8.cuh"

namespace fas {
namespace {

constexpr int kMaxGroups = 4;   // row groups per CTA (named barriers 1 .. 4), and warps of a CTA unless a row needs more
constexpr int kMaxWarps = 16;   // warps per row
// CTAs of four warps per SM: what the registers allow without spilling (16
// warps of 128, 12 of 168).  On 14,960 x 2048: forward 41.5 us with 4, 43 with
// 3, 44 with 5; backward 66 with 3, 74 with 2, 173 with 4, which spills.
constexpr int kFwdPerSm = 4, kBwdPerSm = 3;

// Sums over the row's lanes and the W warps of its group.  `slot` alternates,
// so that one barrier a call is enough (a slot is written again two calls
// later).
template <int N>
struct Exchange {
  float v[2][N][kMaxWarps];
};
// A barrier of one row group.  The numbers are constants: with one in a
// register the kernel would claim all sixteen barriers, and an SM holds
// sixty-four.
__device__ __forceinline__ void group_sync(int group, int threads) {
  switch (group) {
    case 0: asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); break;
    case 1: asm volatile("bar.sync 2, %0;" ::"r"(threads) : "memory"); break;
    case 2: asm volatile("bar.sync 3, %0;" ::"r"(threads) : "memory"); break;
    default: asm volatile("bar.sync 4, %0;" ::"r"(threads) : "memory"); break;
  }
}
template <bool kNarrow, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], Exchange<N>& ex, int slot, int warps, int lanes, int w,
                                           int lane, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (!kNarrow || o < lanes)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (kNarrow || warps == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) ex.v[slot][i][w] = v[i];
  group_sync(group, warps * 32);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int k = 0; k < warps; k += 4)  // the row's tail is zero
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 p = *reinterpret_cast<const float4*>(&ex.v[slot][i][k]);
      v[i] += (p.x + p.y) + (p.z + p.w);
    }
}
template <int N>
__device__ __forceinline__ void clear_exchange(Exchange<N> (&ex)[kMaxGroups]) {
  float* p = reinterpret_cast<float*>(ex);
  for (int i = threadIdx.x; i < (int)(sizeof(ex) / 4); i += blockDim.x) p[i] = 0.f;
  __syncthreads();
}

// Stages of a row ring.  Rows of at most four warps: two (forward) or three
// (backward) cover HBM's latency with the CTAs that fit; wider rows in the
// backward: what shared memory holds beside what else the threads keep there.
template <int V>
constexpr int kRingFwd = V == 4 ? 1 : 2;
// kT: most threads a CTA of the backward has; CTAs of it that share an SM.
template <int kT>
constexpr int kCtas = kT == 128 ? kBwdPerSm : kT == 192 ? 2 : 1;
template <int V, int kT>
constexpr int kKeptPieces = (V == 2 ? 4 : 0) + (V == 2 && kT == 512 ? 4 : 0);  // 16 bytes a vector: Params, Sums
template <int V, int kT, int kVec, bool kF32>
__host__ __device__ constexpr int ring_bwd() {
  if (kT == 128) return kF32 ? 2 : 3;
  const int fit = (232448 / kCtas<kT> - 3072 - kT * 16 * V * kKeptPieces<V, kT>) / (kT * 16 * V * kVec);
  return fit < 1 ? 1 : fit < 4 ? fit : 4;
}

// Asynchronous copies of this thread's bytes into its own shared memory.
// kL1: the other half of the sector is asked for next, so it goes by L1.
template <int kBytes, bool kL1 = kBytes == 8>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (kL1)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A thread's place in the ring: piece i of slot q at base + (q * pieces + i)
// * step, step = 16 bytes a thread of the CTA, so that a warp's accesses are
// consecutive.  `off` is the byte offset of the current slot.
struct RingPos {
  uint32_t off, slot_bytes, end;
  __device__ __forceinline__ RingPos(uint32_t bytes, int slots) : off(0), slot_bytes(bytes), end(bytes * slots) {}
  __device__ __forceinline__ void next() {
    off += slot_bytes;
    if (off == end) off = 0;
  }
};
template <class X>
__device__ __forceinline__ void ring_load(uint32_t dst, uint32_t step, const uint8_t* src) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(X) / 16; ++i) copy_async<16, sizeof(X) == 32>(dst + i * step, src + i * 16);
}
__device__ __forceinline__ uint4 ring_piece(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
template <class X>
__device__ __forceinline__ X ring_read(uint32_t addr, uint32_t step) {
  X x;
  uint4* p = reinterpret_cast<uint4*>(&x);
#pragma unroll
  for (int i = 0; i < (int)sizeof(X) / 16; ++i) p[i] = ring_piece(addr + i * step);
  return x;
}
__device__ __forceinline__ const uint8_t* bytes_of(const void* p) { return static_cast<const uint8_t*>(p); }
__device__ __forceinline__ uint8_t* bytes_of(void* p) { return static_cast<uint8_t*>(p); }

// Eight consecutive fp32 parameters.
__device__ __forceinline__ void load_param(const float* p, vec::P2 (&x)[4]) {
  vec::F32 v;
  v.load(p, 0);
  v.get(x);
}

// Work items: each frame's rows are dealt out to its items in turn (item k of
// n takes rows k, k + n, ...), so that the items of a frame work on
// neighbouring rows at any time.  Frames of equal spans, or a table passed
// with the launch's arguments (no device copy to keep alive).
struct UniformItems {
  int64_t span;
  int per_frame;
  __device__ __forceinline__ int frame(int64_t item) const { return (int)(item / per_frame); }
  __device__ __forceinline__ int64_t first(int f) const { return (int64_t)f * per_frame; }
  __device__ __forceinline__ int count(int) const { return per_frame; }
  __device__ __forceinline__ int64_t start(int f) const { return f * span; }
  __device__ __forceinline__ int64_t rows(int) const { return span; }
};
struct RaggedItems {
  int n;
  int32_t row[kNormMaxFrames + 1], item[kNormMaxFrames + 1];
  __device__ __forceinline__ int frame(int64_t i) const {
    int lo = 0, hi = n - 1;  // the last frame whose items start at or before i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (item[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  __device__ __forceinline__ int64_t first(int f) const { return item[f]; }
  __device__ __forceinline__ int count(int f) const { return item[f + 1] - item[f]; }
  __device__ __forceinline__ int64_t start(int f) const { return row[f]; }
  __device__ __forceinline__ int64_t rows(int f) const { return row[f + 1] - row[f]; }
};

// Where a thread works: its row group's item.  A row has W warps, or (kNarrow:
// up to 128 columns) 4, 8 or 16 lanes of one, whose other lanes have other
// rows: they all go through the longest item's rows together, for the
// shuffles.
struct Place {
  int group, w, lane;  // of the warps that share a row; the lane within the row
  bool on;             // an item of its own
  int64_t item;
  int f, stride, n, turns;  // the item's frame, rows apart, rows; rows of the warp's longest item
  int64_t r0;               // first row
};
template <bool kNarrow, class Items>
__device__ __forceinline__ Place place(const NormArgs& a, const Items& items) {
  Place p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, lanes = kNarrow ? a.lanes : 32;
  p.group = warp / a.warps;
  p.w = warp % a.warps;
  p.lane = lane % lanes;
  const int64_t item = (int64_t)blockIdx.x * a.groups + p.group * (32 / lanes) + lane / lanes;
  p.on = item < a.items;
  p.item = p.on ? item : 0;
  p.f = items.frame(p.item);
  p.stride = items.count(p.f);
  const int first = (int)(p.item - items.first(p.f));
  p.r0 = items.start(p.f) + first;
  p.n = p.on ? (int)((items.rows(p.f) - first + p.stride - 1) / p.stride) : 0;
  p.turns = kNarrow ? (int)__reduce_max_sync(0xffffffffu, (unsigned)p.n) : p.n;
  return p;
}

// kWide: rows of more than four warps (up to 512 threads a CTA); else 128.
template <class R, int V, bool kCkpt, bool kWide, bool kNarrow, class Items>
__global__ void __launch_bounds__(kWide ? 512 : 128, kWide ? 1 : kFwdPerSm)
    residual_norm_fwd(const NormArgs a, const __grid_constant__ Items items) {
  using namespace vec;
  __shared__ __align__(16) Exchange<1> ex[kMaxGroups];
  clear_exchange(ex);
  const Place at = place<kNarrow>(a, items);
  const int W = a.warps, group = at.group, w = at.w, lane = at.lane, C = a.width, n = at.n;
  const int64_t r0 = at.r0, row_step = (int64_t)at.stride * C;  // elements between the item's rows
  const float inv_c = 1.0f / (float)C;
  extern __shared__ uint4 ring[];
  constexpr int S = kRingFwd<V>, kX = sizeof(R) / 16, kVec = 1 + kX, kElem = sizeof(R) / 8;
  const uint32_t step = blockDim.x * 16, base = ptx::smem_addr(ring + threadIdx.x);
  bool in[V];
  int col[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = (v * W * 32 + w * 32 + lane) * 8;
    in[v] = col[v] < C;
  }
  // Pointers to this thread's first vector, advanced row by row.
  const int64_t at0 = r0 * C + col[0];
  const int vstep = W * 32 * 8;  // columns between a thread's vectors
  const uint8_t *py = bytes_of(a.y) + at0 * 2, *px = bytes_of(a.x) + at0 * kElem;
  uint8_t *ph = bytes_of(a.h) + at0 * 2, *po = bytes_of(a.x_out) + at0 * kElem;
  RingPos ld(V * kVec * step, S), rd(V * kVec * step, S);
  int left = n;  // rows not yet asked for
  auto load = [&]() {
    if (left > 0) {
      --left;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (in[v]) {
          const uint32_t dst = base + ld.off + v * kVec * step;
          ring_load<Bf16>(dst, step, py + v * vstep * 2);
          ring_load<R>(dst + step, step, px + v * vstep * kElem);
        }
      py += row_step * 2;
      px += row_step * kElem;
      ld.next();
    }
    copy_commit();
  };
  for (int i = 0; i < S; ++i) load();
  P2 gpre[V][4], coef[V][4];  // coef: alpha gate gamma_post
  const P2 zero = both(0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) gpre[v][e] = coef[v][e] = zero;
    if (in[v]) {
      load_param(a.gamma_pre + col[v], gpre[v]);
      load_param(a.gamma_post + col[v], coef[v]);
      P2 gt[4] = {both(1.f), both(1.f), both(1.f), both(1.f)};
      if (a.gate) load_param(a.gate + (int64_t)at.f * C + col[v], gt);
#pragma unroll
      for (int e = 0; e < 4; ++e) coef[v][e] = mul2(mul2(coef[v][e], both(a.alpha)), gt[e]);
    }
  }
  for (int i = 0; i < at.turns; ++i) {
    const bool live = !kNarrow || i < n;
    copy_wait<S - 1>();
    P2 y[V][4], x[V][4], acc = zero;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Bf16 yv{};
      R xv{};
      if (in[v] && live) {
        const uint32_t src = base + rd.off + v * kVec * step;
        yv = ring_read<Bf16>(src, step);
        xv = ring_read<R>(src + step, step);
      }
      yv.get(y[v]);
      xv.get(x[v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = fma2(y[v][e], y[v][e], acc);
    }
    rd.next();
    load();
    float s[1] = {sum(acc)};
    group_sums<kNarrow>(s, ex[group], 0, W, a.lanes, w, lane, group);
    const float ry = rsqrtf(s[0] * inv_c + a.eps);
    const P2 ry2 = both(ry);
    acc = zero;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[v][e] = fma2(mul2(y[v][e], ry2), coef[v][e], x[v][e]);
        acc = fma2(x[v][e], x[v][e], acc);
      }
    s[0] = sum(acc);
    group_sums<kNarrow>(s, ex[group], 1, W, a.lanes, w, lane, group);
    const float rx = rsqrtf(s[0] * inv_c + a.eps);
    const P2 rx2 = both(rx);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P2 h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = mul2(mul2(x[v][e], rx2), gpre[v][e]);
      Bf16 hv;
      R ov;
      hv.set(h);
      ov.set(x[v]);
      if (in[v] && live) {
        hv.store(ph + v * vstep * 2, 0);
        ov.store(po + v * vstep * kElem, 0);
      }
      if constexpr (kCkpt) {
        ov.get(x[v]);  // the checkpoint is of x' as stored
        uint32_t by, bx;
        const uint2 cy = ckpt::encode8(y[v], by), cx = ckpt::encode8(x[v], bx);
        if (in[v] && live) {
          const int64_t o = r0 * C + i * row_step + col[v];
          *reinterpret_cast<uint2*>(a.y8 + o) = cy;
          *reinterpret_cast<uint2*>(a.x8 + o) = cx;
          if ((lane & 3) == 0) {
            a.y8_scale[o / ckpt::kBlock] = (uint8_t)by;
            a.x8_scale[o / ckpt::kBlock] = (uint8_t)bx;
          }
        }
      }
    }
    ph += row_step * 2;
    po += row_step * kElem;
    if (w == 0 && lane == 0 && live) {
      a.rstd[r0 + (int64_t)i * at.stride] = ry;
      a.rstd[a.rows + r0 + (int64_t)i * at.stride] = rx;
    }
  }
}

// y and x' of one thread's eight columns, 16 bits (or fp32 x') or 8 bits.
template <class R, bool k8>
struct Held;
template <class R>
struct Held<R, false> {
  static constexpr int kPieces = 1 + sizeof(R) / 16, kElem = sizeof(R) / 8;
  const uint8_t *y, *x;
  __device__ __forceinline__ Held(const NormArgs& a, int64_t at) : y(bytes_of(a.y) + at * 2), x(bytes_of(a.x) + at * kElem) {}
  __device__ __forceinline__ void load(uint32_t dst, uint32_t step, int cols) const {
    ring_load<vec::Bf16>(dst, step, y + cols * 2);
    ring_load<R>(dst + step, step, x + cols * kElem);
  }
  __device__ __forceinline__ void next(int64_t c) {
    y += c * 2;
    x += c * kElem;
  }
  static __device__ __forceinline__ void get(uint32_t src, uint32_t step, uint32_t, uint32_t, vec::P2 (&yf)[4],
                                             vec::P2 (&xf)[4]) {
    ring_read<vec::Bf16>(src, step).get(yf);
    ring_read<R>(src + step, step).get(xf);
  }
};
template <class R>
struct Held<R, true> {
  static constexpr int kPieces = 1;  // both codes' eight bytes
  const uint8_t *y, *x;
  __device__ __forceinline__ Held(const NormArgs& a, int64_t at) : y(a.y8 + at), x(a.x8 + at) {}
  __device__ __forceinline__ void load(uint32_t dst, uint32_t, int cols) const {
    copy_async<8>(dst, y + cols);
    copy_async<8>(dst + 8, x + cols);
  }
  __device__ __forceinline__ void next(int64_t c) {
    y += c;
    x += c;
  }
  static __device__ __forceinline__ void get(uint32_t src, uint32_t, uint32_t by, uint32_t bx, vec::P2 (&yf)[4],
                                             vec::P2 (&xf)[4]) {
    const uint4 c = ring_piece(src);
    ckpt::decode8(make_uint2(c.x, c.y), by, yf);
    ckpt::decode8(make_uint2(c.z, c.w), bx, xf);
  }
};

// alpha gate gamma_post and gamma_pre of a thread's columns: in registers, or
// (V = 2, where the two column sums take 64 registers) in shared memory, four
// 16-byte pieces a vector that only this thread reads.  Kept in registers
// there, they left 8 warps an SM, or spilled.
template <int V>
struct Params {
  static constexpr int kPieces = V == 2 ? 4 : 0;
  vec::P2 coef_[V == 2 ? 1 : V][4], gpre_[V == 2 ? 1 : V][4];
  uint32_t at, step;
  __device__ __forceinline__ void set(int v, const vec::P2 (&c)[4], const vec::P2 (&g)[4]) {
    if constexpr (V == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const vec::P2 *x = (i < 2 ? c : g) + (i & 1) * 2;
        asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(at + (v * 4 + i) * step), "l"(x[0].v), "l"(x[1].v) : "memory");
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        coef_[v][e] = c[e];
        gpre_[v][e] = g[e];
      }
    }
  }
  __device__ __forceinline__ void piece(int v, int i, vec::P2 (&x)[4]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x[2 * k].v), "=l"(x[2 * k + 1].v) : "r"(at + (v * 4 + i + k) * step));
  }
  __device__ __forceinline__ void coef(int v, vec::P2 (&x)[4]) const {
    if constexpr (V == 2) {
      piece(v, 0, x);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = coef_[v][e];
    }
  }
  __device__ __forceinline__ void gpre(int v, vec::P2 (&x)[4]) const {
    if constexpr (V == 2) {
      piece(v, 2, x);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = gpre_[v][e];
    }
  }
};

// The two column sums of a thread's columns: in registers, or (V = 2 in rows
// of more than eight warps, 128 registers a thread) in shared memory.
template <int V, bool kSmem>
struct Sums {
  vec::P2 z_[kSmem ? 1 : V][4], d_[kSmem ? 1 : V][4];
  uint32_t at, step;
  __device__ __forceinline__ uint32_t piece(int v, int i) const { return at + (v * 4 + i) * step; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (kSmem) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("st.shared.v2.u64 [%0], {%1, %1};" ::"r"(piece(v, i)), "l"(0ull) : "memory");
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) z_[v][e] = d_[v][e] = vec::both(0.f);
      }
    }
  }
  // The sums' four pairs (which: 0 Z, 1 dgamma_pre) += a * b.
  template <int kWhich>
  __device__ __forceinline__ void add(int v, const vec::P2 (&a)[4], const vec::P2 (&b)[4]) {
    if constexpr (kSmem) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        vec::P2 s0, s1;
        const uint32_t p = piece(v, kWhich * 2 + i);
        asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(s0.v), "=l"(s1.v) : "r"(p));
        s0 = vec::fma2(a[2 * i], b[2 * i], s0);
        s1 = vec::fma2(a[2 * i + 1], b[2 * i + 1], s1);
        asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(p), "l"(s0.v), "l"(s1.v) : "memory");
      }
    } else {
      vec::P2(&s)[4] = kWhich ? d_[v] : z_[v];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = vec::fma2(a[e], b[e], s[e]);
    }
  }
  template <int kWhich>
  __device__ __forceinline__ void get(int v, vec::P2 (&s)[4]) const {
    if constexpr (kSmem) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(s[2 * i].v), "=l"(s[2 * i + 1].v) : "r"(piece(v, kWhich * 2 + i)));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = kWhich ? d_[v][e] : z_[v][e];
    }
  }
};

// Both row means come from one exchange: with t = dx' + r_x a (g = t - r_x xh
// m1), sum(b yh) = sum(coef yh t) - r_x m1 sum(coef yh xh), coef = alpha gate
// gamma_post, so the three sums of a xh, coef yh t and coef yh xh give both.
template <class R, int V, bool k8, int kT, bool kNarrow, class Items>
__global__ void __launch_bounds__(kT, kCtas<kT>)
    residual_norm_bwd(const NormArgs a, const __grid_constant__ Items items) {
  using namespace vec;
  __shared__ __align__(16) Exchange<3> ex[kMaxGroups];
  clear_exchange(ex);
  ptx::grid_launch_next();
  const Place at = place<kNarrow>(a, items);
  const int W = a.warps, group = at.group, w = at.w, lane = at.lane, C = a.width, n = at.n, stride = at.stride;
  const int64_t r0 = at.r0, row_step = (int64_t)stride * C;  // elements between the item's rows
  const float inv_c = 1.0f / (float)C;
  extern __shared__ uint4 ring[];
  using H = Held<R, k8>;
  constexpr int kG = sizeof(R) / 16, kVec = kG + 1 + H::kPieces, kElem = sizeof(R) / 8;
  constexpr int S = ring_bwd<V, kT, kVec, sizeof(R) == 32>();
  const uint32_t step = blockDim.x * 16, base = ptx::smem_addr(ring + threadIdx.x);
  int col[V];
  bool in[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = (v * W * 32 + w * 32 + lane) * 8;
    in[v] = col[v] < C;
  }
  const int64_t at0 = r0 * C + col[0];
  const int vstep = W * 32 * 8;  // columns between a thread's vectors
  const uint8_t *pg = bytes_of(a.dx_out) + at0 * kElem, *ph = bytes_of(a.dh) + at0 * 2;
  uint8_t *pdx = bytes_of(a.dx) + at0 * kElem, *pdy = bytes_of(a.dy) + at0 * 2;
  H held(a, at0);
  RingPos ld(V * kVec * step, S), rd(V * kVec * step, S);
  int left = n;  // rows not yet asked for
  auto load = [&]() {
    if (left > 0) {
      --left;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (in[v]) {
          const uint32_t dst = base + ld.off + v * kVec * step;
          ring_load<R>(dst, step, pg + v * vstep * kElem);
          ring_load<Bf16>(dst + kG * step, step, ph + v * vstep * 2);
          held.load(dst + (kG + 1) * step, step, v * vstep);
        }
      pg += row_step * kElem;
      ph += row_step * 2;
      held.next(row_step);
      ld.next();
    }
    copy_commit();
  };
  for (int i = 0; i < S; ++i) load();
  // The row's small inputs come through registers, two rows ahead, and are
  // not touched before their row (an instruction that uses one waits for it).
  struct Small {
    float ry, rx;
    uint32_t by[V], bx[V];
  };
  const float* pr = a.rstd + r0;
  const uint8_t *sy = nullptr, *sx = nullptr;
  if (k8) {
    sy = a.y8_scale + at0 / ckpt::kBlock;
    sx = a.x8_scale + at0 / ckpt::kBlock;
  }
  auto load_small = [&](int i, Small& s) {
    if (i < n) {
      s.ry = pr[(int64_t)i * stride];
      s.rx = pr[(int64_t)i * stride + a.rows];
      if (k8)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (in[v]) {
            s.by[v] = sy[i * (row_step / ckpt::kBlock) + v * (vstep / ckpt::kBlock)];
            s.bx[v] = sx[i * (row_step / ckpt::kBlock) + v * (vstep / ckpt::kBlock)];
          }
    }
  };
  Small small[2] = {};
  load_small(0, small[0]);
  load_small(1, small[1]);
  const P2 zero = both(0.f);
  Params<V> params;
  params.at = base + S * V * kVec * step;
  params.step = step;
  Sums<V, V == 2 && kT == 512> sums;
  sums.at = params.at + V * Params<V>::kPieces * step;
  sums.step = step;
  sums.clear();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    P2 c[4] = {zero, zero, zero, zero}, g[4] = {zero, zero, zero, zero};
    if (in[v]) {
      load_param(a.gamma_post + col[v], c);
      load_param(a.gamma_pre + col[v], g);
      P2 gt[4] = {both(1.f), both(1.f), both(1.f), both(1.f)};
      if (a.gate) load_param(a.gate + (int64_t)at.f * C + col[v], gt);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = mul2(mul2(c[e], both(a.alpha)), gt[e]);
    }
    params.set(v, c, g);
  }
  auto row = [&](int i, Small& sm, int slot) {
    P2 y[V][4], x[V][4], t[V][4];
    const bool live = !kNarrow || i < n;
    const float ry = live ? sm.ry : 0.f, rx = live ? sm.rx : 0.f;
    const P2 ry2 = both(ry), rx2 = both(rx);
    P2 sa = zero, sb = zero, sc = zero;
    copy_wait<S - 1>();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P2 h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[v][e] = x[v][e] = t[v][e] = h[e] = zero;
      if (in[v] && live) {
        const uint32_t src = base + rd.off + v * kVec * step;
        ring_read<R>(src, step).get(t[v]);
        ring_read<Bf16>(src + kG * step, step).get(h);
        H::get(src + (kG + 1) * step, step, sm.by[v], sm.bx[v], y[v], x[v]);
      }
      P2 coef[4], gpre[4];
      params.coef(v, coef);
      params.gpre(v, gpre);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[v][e] = mul2(y[v][e], ry2);
        x[v][e] = mul2(x[v][e], rx2);
        const P2 ah = mul2(h[e], gpre[e]);
        sa = fma2(ah, x[v][e], sa);
        t[v][e] = fma2(rx2, ah, t[v][e]);
        const P2 cy = mul2(coef[e], y[v][e]);
        sb = fma2(cy, t[v][e], sb);
        sc = fma2(cy, x[v][e], sc);
      }
      sums.template add<1>(v, h, x[v]);
    }
    rd.next();
    load();
    load_small(i + 2, sm);
    float s[3] = {sum(sa), sum(sb), sum(sc)};
    group_sums<kNarrow>(s, ex[group], slot, W, a.lanes, w, lane, group);
    const float rm1 = rx * s[0] * inv_c, m2 = (s[1] - rm1 * s[2]) * inv_c;
    const P2 nrm1 = both(-rm1), nm2 = both(-m2);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P2 d[4], coef[4];
      params.coef(v, coef);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[v][e] = fma2(nrm1, x[v][e], t[v][e]);  // g
        d[e] = mul2(ry2, fma2(nm2, y[v][e], mul2(coef[e], t[v][e])));
      }
      sums.template add<0>(v, y[v], t[v]);
      Bf16 dv;
      R ov;
      dv.set(d);
      ov.set(t[v]);
      if (in[v] && live) {
        dv.store(pdy + v * vstep * 2, 0);
        ov.store(pdx + v * vstep * kElem, 0);
      }
    }
    pdx += row_step * kElem;
    pdy += row_step * 2;
  };
  for (int i = 0; i < at.turns; i += 2) {
    row(i, small[0], 0);
    if (i + 1 < at.turns) row(i + 1, small[1], 1);
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (in[v] && at.on) {
      F32 o;
      P2 s[4];
      sums.template get<0>(v, s);
      o.set(s);
      o.store(a.z_part, at.item * C + col[v]);
      sums.template get<1>(v, s);
      o.set(s);
      o.store(a.d_part, at.item * C + col[v]);
    }
}

// Adds the partials: a CTA per 16 columns, 128 lanes of four-column loads.
// A frame's items are split over `sub` lanes, so that each lane has few loads
// and all are in flight at once; then the frame's lanes are added, and the
// frames, each in a fixed order.
constexpr int kSumCols = 16, kSumLanes = 128, kSumThreads = kSumCols / 4 * kSumLanes, kSumRows = kSumThreads / kSumCols;

template <class Items>
__global__ void __launch_bounds__(kSumThreads)
    residual_norm_sums(const NormArgs a, const __grid_constant__ Items items, int n_frames) {
  __shared__ __align__(16) float zr[kSumLanes][kSumCols], dr[kSumLanes][kSumCols];
  __shared__ float last[2][kSumCols][kSumRows + 1];
  const int tx = threadIdx.x % (kSumCols / 4), lane = threadIdx.x / (kSumCols / 4);
  const int C = a.width, c0 = blockIdx.x * kSumCols;
  const bool in = c0 + tx * 4 < C;  // C is a multiple of 8
  const int sub = n_frames >= kSumLanes ? 1 : kSumLanes / n_frames, par = kSumLanes / sub;
  const int ct = threadIdx.x % kSumCols, wt = threadIdx.x / kSumCols;  // one column a thread
  const bool ct_in = c0 + ct < C;
  // What the first kernel does not write is read before it ends.
  const float post = ct_in ? a.gamma_post[c0 + ct] * a.alpha : 0.f;
  float gate = a.gate && ct_in && wt < n_frames ? a.gate[(int64_t)wt * C + c0 + ct] : 1.f;
  ptx::grid_wait_previous();
  float4 d = {0.f, 0.f, 0.f, 0.f};
  float zs = 0.f;
  for (int f0 = 0; f0 < n_frames; f0 += par) {
    const int f = f0 + lane / sub, s = lane % sub;
    float4 z = {0.f, 0.f, 0.f, 0.f};
    if (in && lane / sub < par && f < n_frames) {
      const int64_t i1 = items.first(f) + items.count(f);
#pragma unroll 4
      for (int64_t i = items.first(f) + s; i < i1; i += sub) {
        const float4 p = *reinterpret_cast<const float4*>(a.z_part + i * C + c0 + tx * 4);
        const float4 q = *reinterpret_cast<const float4*>(a.d_part + i * C + c0 + tx * 4);
        z.x += p.x; z.y += p.y; z.z += p.z; z.w += p.w;
        d.x += q.x; d.y += q.y; d.z += q.z; d.w += q.w;
      }
    }
    *reinterpret_cast<float4*>(&zr[lane][tx * 4]) = z;
    __syncthreads();
    const int nf = n_frames - f0 < par ? n_frames - f0 : par;
    for (int k = wt; k < nf; k += kSumRows) {
      float v = 0.f;
      for (int l = 0; l < sub; ++l) v += zr[k * sub + l][ct];
      if (a.gate && ct_in) {
        const int64_t at = (int64_t)(f0 + k) * C + c0 + ct;
        if (f0 + k != wt) gate = a.gate[at];
        a.dgate[at] = post * v;
      }
      zs = fmaf(gate, v, zs);
    }
    __syncthreads();
  }
  *reinterpret_cast<float4*>(&dr[lane][tx * 4]) = d;
  __syncthreads();
  float ds = 0.f;
#pragma unroll
  for (int l = 0; l < kSumLanes / kSumRows; ++l) ds += dr[wt * (kSumLanes / kSumRows) + l][ct];
  last[0][ct][wt] = zs;
  last[1][ct][wt] = ds;
  __syncthreads();
  // A warp per column adds its 32 shares.
  static_assert(kSumRows == 32 && kSumThreads == 32 * kSumCols, "");
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  float v0 = last[0][w][l], v1 = last[1][w][l];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v0 += __shfl_xor_sync(0xffffffffu, v0, o);
    v1 += __shfl_xor_sync(0xffffffffu, v1, o);
  }
  if (l == 0 && c0 + w < C) {
    a.dgamma_post[c0 + w] = a.alpha * v0;
    a.dgamma_pre[c0 + w] = v1;
  }
}


struct Shape {
  int V, W, L, G;  // vectors a thread, warps and lanes a row, rows a CTA works on
};
// One vector a thread up to 256 columns, four above 8192, else two (half the
// instructions a row that one takes).
Shape shape_of(int width) {
  const int vecs = width / 8;
  const int V = vecs <= 32 ? 1 : vecs <= 64 * kMaxWarps ? 2 : 4;
  const int W = (vecs + 32 * V - 1) / (32 * V);
  const int L = vecs <= 4 ? 4 : vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32;
  return {V, W, L, std::max(1, kMaxGroups / W) * (32 / L)};
}

int warps_of(const Shape& s) { return s.W * std::max(1, kMaxGroups / s.W); }  // of a CTA

// A kernel's ring: its opt-in shared memory, and, for more CTAs than SMs, the
// SM's whole share for it (by itself the driver leaves room for fewer CTAs
// than fit).  Set on every launch: it belongs to the device's context.
template <class K>
cudaError_t allow_ring(K kern, size_t smem, bool many) {
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024)  // up to 48 KB with the static part goes without
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && many)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  return e;
}

template <class R, int V, bool kCkpt, bool kWide, bool kNarrow, class Items>
cudaError_t fwd(const NormArgs& a, const Items& it, const Shape& s, cudaStream_t st) {
  auto kern = residual_norm_fwd<R, V, kCkpt, kWide, kNarrow, Items>;
  const size_t smem = (size_t)32 * warps_of(s) * kRingFwd<V> * V * (16 + sizeof(R));
  const cudaError_t e = allow_ring(kern, smem, a.items / s.G > a.sms);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((a.items + s.G - 1) / s.G), 32 * warps_of(s), smem, st>>>(a, it);
  return cudaGetLastError();
}

template <class R, int V, class Items>
cudaError_t fwd_c(const NormArgs& a, const Items& it, const Shape& s, cudaStream_t st) {
  if constexpr (V == 1)
    if (s.L < 32) return a.y8 ? fwd<R, V, true, false, true>(a, it, s, st) : fwd<R, V, false, false, true>(a, it, s, st);
  if constexpr (V >= 2)
    if (s.W > kMaxGroups) return a.y8 ? fwd<R, V, true, true, false>(a, it, s, st) : fwd<R, V, false, true, false>(a, it, s, st);
  if constexpr (V <= 2)
    return a.y8 ? fwd<R, V, true, false, false>(a, it, s, st) : fwd<R, V, false, false, false>(a, it, s, st);
  return cudaErrorInvalidValue;  // V = 4 has more warps
}
template <class Items>
cudaError_t fwd_all(const NormArgs& a, const Items& it, const Shape& s, cudaStream_t st) {
  if (s.V == 1) return a.f32 ? fwd_c<vec::F32, 1>(a, it, s, st) : fwd_c<vec::Bf16, 1>(a, it, s, st);
  if (s.V == 2) return a.f32 ? fwd_c<vec::F32, 2>(a, it, s, st) : fwd_c<vec::Bf16, 2>(a, it, s, st);
  return a.f32 ? fwd_c<vec::F32, 4>(a, it, s, st) : fwd_c<vec::Bf16, 4>(a, it, s, st);
}

template <class R, int V, bool k8, int kT, bool kNarrow, class Items>
cudaError_t bwd(const NormArgs& a, const Items& it, const Shape& s, cudaStream_t st) {
  auto kern = residual_norm_bwd<R, V, k8, kT, kNarrow, Items>;
  constexpr int kVec = sizeof(R) / 16 + 1 + Held<R, k8>::kPieces;
  const size_t smem = (size_t)32 * warps_of(s) * V * 16 *
                      (ring_bwd<V, kT, kVec, sizeof(R) == 32>() * kVec + kKeptPieces<V, kT>);
  const cudaError_t e = allow_ring(kern, smem, a.items / s.G > a.sms);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((a.items + s.G - 1) / s.G), 32 * warps_of(s), smem, st>>>(a, it);
  return cudaGetLastError();
}
template <class R, int V, class Items>
cudaError_t bwd_c(const NormArgs& a, const Items& it, const Shape& s, cudaStream_t st) {
  auto go = [&](auto t, auto narrow) {
    constexpr int kT = decltype(t)::value;
    constexpr bool kN = decltype(narrow)::value;
    return a.y8 ? bwd<R, V, true, kT, kN>(a, it, s, st) : bwd<R, V, false, kT, kN>(a, it, s, st);
  };
  using std::integral_constant;
  const std::false_type no;
  if constexpr (V == 1) {
    if (s.L < 32) return go(integral_constant<int, 128>(), std::true_type());
    return go(integral_constant<int, 128>(), no);
  } else if constexpr (V == 2) {
    if (s.W <= 4) return go(integral_constant<int, 128>(), no);
    if (s.W <= 6) return go(integral_constant<int, 192>(), no);
    if (s.W <= 8) return go(integral_constant<int, 256>(), no);
    return go(integral_constant<int, 512>(), no);
  } else {
    return go(integral_constant<int, 512>(), no);
  }
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.width + kSumCols - 1) / kSumCols));
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // starts in the first kernel's tail
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, residual_norm_sums<Items>, a, it, n_frames);
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Splits the rows: about one item per row group that runs at once, none
// across frames.  Depends on the shape and the device alone.
NormItems split(int64_t rows, const Shape& s, const int32_t* spans, int n_frames, int64_t span, int sms, int per_sm) {
  // per_sm is in CTAs of four warps (which fix the registers a thread).
  const int ctas = std::max(1, per_sm * kMaxGroups / warps_of(s));
  const int64_t want = std::max<int64_t>(n_frames, (int64_t)ctas * sms * s.G);
  auto count = [&](int64_t chunk) {
    if (!spans) return (int64_t)n_frames * ((span + chunk - 1) / chunk);
    int64_t n = 0;
    for (int f = 0; f < n_frames; ++f) n += (spans[f] + chunk - 1) / chunk;
    return n;
  };
  int64_t lo = 1, hi = rows;  // the fewest rows an item with at most `want` items
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (count(mid) <= want) hi = mid; else lo = mid + 1;
  }
  NormItems r;
  r.chunk = lo;
  r.items = count(lo);
  return r;
}

// Calls fn with the frames' item table.
template <class Fn>
cudaError_t with_items(const NormItems& n, const int32_t* spans, int n_frames, int64_t span, Fn fn) {
  if (!spans) return fn(UniformItems{span, (int)((span + n.chunk - 1) / n.chunk)});
  RaggedItems it;
  it.n = n_frames;
  it.row[0] = it.item[0] = 0;
  for (int f = 0; f < n_frames; ++f) {
    it.row[f + 1] = it.row[f] + spans[f];
    it.item[f + 1] = it.item[f] + (int32_t)((spans[f] + n.chunk - 1) / n.chunk);
  }
  return fn(it);
}

}  // namespace

cudaError_t launch_residual_norm(NormArgs a, const int32_t* spans, int n_frames, int64_t span, int sms,
                                 cudaStream_t st) {
  const Shape s = shape_of(a.width);
  const NormItems n = split(a.rows, s, spans, n_frames, span, sms, kFwdPerSm);
  a.warps = s.W;
  a.lanes = s.L;
  a.groups = s.G;
  a.items = n.items;
  a.sms = sms;
  return with_items(n, spans, n_frames, span, [&](const auto& it) { return fwd_all(a, it, s, st); });
}

NormItems residual_norm_items(int64_t rows, int width, const int32_t* spans, int n_frames, int64_t span, int sms) {
  NormItems r = split(rows, shape_of(width), spans, n_frames, span, sms, kBwdPerSm);
  r.bytes = 2 * align256(r.items * width * 4);
  return r;
}

cudaError_t launch_residual_norm_backward(NormArgs a, const NormItems& n, const int32_t* spans, int n_frames,
                                          int64_t span, int sms, void* workspace, cudaStream_t st) {
  const Shape s = shape_of(a.width);
  a.sms = sms;
  a.warps = s.W;
  a.lanes = s.L;
  a.groups = s.G;
  a.items = n.items;
  a.z_part = static_cast<float*>(workspace);
  a.d_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256(n.items * a.width * 4));
  return with_items(n, spans, n_frames, span, [&](const auto& it) { return bwd_all(a, it, n_frames, s, st); });
}

}  // namespace fas
