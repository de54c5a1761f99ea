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
// vectors a thread, so a row's values stay in registers from its arrival to
// its stores, and a row sum is a warp shuffle and one exchange through shared
// memory: of the CTA, or, for rows of more warps than a CTA takes, of the CTAs
// of a cluster.  A group works through its item's rows; gamma and gate stay
// with it, and the next rows are on their way into a ring in shared memory.
// Each thread copies just the bytes it will read itself (cp.async), so the
// ring needs no barrier.  (One vector a thread and rows prefetched into
// registers: twice the instructions a row, 57 us forward and 80 backward at
// 14,960 x 2048.)
//
// Bound by HBM: forward 42 us at 14,960 x 2048 bf16 (5.8 TB/s, 0.86 of the
// measured copy rate), backward 59 us (6.2 TB/s, 0.91) and 7 for its sums;
// 291 us (0.82) from 8-bit checkpoints at 79,200 x 2048, where decoding takes
// issue slots; device time of captured calls.  Narrow and wide rows: see Row.
//
// Backward: a group's rows never cross frames, so it adds its columns of Z
// and of dgamma_pre in registers and writes one partial row of each at its
// end; a second kernel adds the partials frame by frame and then frame after
// frame, in a fixed order (no atomics: results are bit-reproducible).

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "checkpoint.cuh"
#include "kernels.h"
#include "vec8.cuh"

namespace fas {
namespace {

constexpr int kMaxGroups = 4;  // row groups per CTA (named barriers 1 .. 4), and warps of a CTA unless a row needs more
constexpr int kMaxCtas = 8;    // CTAs of a cluster that share a row
// CTAs of four warps per SM: what the registers allow without spilling (16
// warps of 128, 12 of 168).  On 14,960 x 2048: forward 41.5 us with 4, 43 with
// 3, 44 with 5; backward 65 with 3, 74 with 2, 173 with 4, which spills.
constexpr int kFwdPerSm = 4, kBwdPerSm = 3;

// Who shares a row: 4, 8 or 16 lanes of a warp (up to 128 columns), one to
// four warps of a CTA, a CTA of more (kWide), or a cluster of CTAs of up to
// four warps.  A CTA that has a row to itself stands still while its row sums
// are exchanged, and the few such CTAs an SM holds hide less of it than three
// or four whose sums cross the cluster.  % of the copy rate, CTA against
// cluster (30 M elements): forward at 2,560 columns 84 against 60, 4,096 84 /
// 79, 5,120 (ten warps) 60 / 78, 16,384 (whose rows spilled in one CTA) 50 /
// 71; backward 76 / 64, 67 / 75, 64 / 71, 24 / 61; from 8 bits 63 / 44, 56 /
// 59, 38 / 55, 17 / 47.  Narrow rows: 64 columns 84, 61 and 53.
enum Row { kLanes, kWarps, kWide, kCluster };
constexpr int kWideFwd = 8, kWideBwd = 6;  // most warps of a kWide CTA

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

// Sums over the row's lanes and the W warps of its group.  `slot` alternates,
// so that one barrier a call is enough (a slot is written again two calls
// later); `phase` counts a slot's uses.
template <Row kRow, int N>
struct Exchange {
  static constexpr int kSlots = kRow == kWide ? 8 : 4, kGroups = kRow == kWide ? 1 : kMaxGroups;
  float v[kGroups][2][N][kSlots];
  __device__ __forceinline__ void start() {  // zero where no warp writes
    float* p = &v[0][0][0][0];
    for (int i = threadIdx.x; i < (int)(sizeof(v) / 4); i += blockDim.x) p[i] = 0.f;
    __syncthreads();
  }
  // v's sums over the warps.
  __device__ __forceinline__ void sum(float (&x)[N], int slot, int, const NormArgs& a, int w, int lane, int group,
                                      bool&) {
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) v[group][slot][i][w] = x[i];
    group_sync(group, a.warps * 32);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4* p = reinterpret_cast<const float4*>(v[group][slot][i]);
      x[i] = (p[0].x + p[0].y) + (p[0].z + p[0].w);
      if (kRow == kWide) x[i] += (p[1].x + p[1].y) + (p[1].z + p[1].w);
    }
  }
  __device__ __forceinline__ void finish() {}
};

// Set where a cluster's wait was given up.
__device__ unsigned int g_gave_up;
std::atomic<bool> g_clusters{false};  // a cluster was launched

// In a cluster each warp sends its sums to every CTA of the row (st.async) and
// each CTA waits on its own mbarrier for all warps' bytes: one trip between
// SMs, where storing and a barrier of the cluster take several (4,096 columns:
// 79% of the copy rate against 54 forward, 76 against 59 backward).  A slot is
// free again as in one CTA: who sends for call n + 2 has all of call n + 1,
// which each warp sent after reading call n.
//
// All CTAs of a cluster run together, so the waits end.  Should one not, its
// thread is `lost`: it sets the CTA's and the module's word and from then on
// neither waits, arrives nor sends, and its sums are NaN.  A phase ends only
// with every warp's bytes, and a lane that is lost sends none, so no other
// thread ever takes a sum that lacks some: it has the whole sum, or its own
// wait runs out too.
constexpr uint64_t kSettleNs = 1000000;  // for sums in flight to a CTA that has stopped waiting for them
template <int N>
struct Exchange<kCluster, N> {
  static constexpr int kPart = N == 1 ? 1 : 4;  // floats a warp sends: one, or three and a pad
  float part[2][kMaxCtas * kMaxGroups][kPart];
  uint64_t bar[2];
  int given_up;
  __device__ __forceinline__ void start() {
    for (int i = threadIdx.x; i < 2 * kMaxCtas * kMaxGroups * kPart; i += blockDim.x) (&part[0][0][0])[i] = 0.f;
    if (threadIdx.x == 0) {
      given_up = 0;
      ptx::mbar_init(ptx::smem_addr(&bar[0]), 1);
      ptx::mbar_init(ptx::smem_addr(&bar[1]), 1);
      ptx::fence_mbar_init();
    }
    __syncwarp();
    ptx::cluster_sync();
  }
  __device__ __forceinline__ bool wait(uint32_t b, int phase, uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
      if (ptx::mbar_try_wait_cluster(b, phase & 1)) return true;
      if ((it & 7u) != 0u) continue;
      if (*reinterpret_cast<volatile int*>(&given_up)) return false;
      const uint64_t now = ptx::global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) {
        *reinterpret_cast<volatile int*>(&given_up) = 1;
        atomicOr(&g_gave_up, 1u);
        return false;
      }
    }
  }
  __device__ __forceinline__ void sum(float (&x)[N], int slot, int phase, const NormArgs& a, int w, int lane, int,
                                      bool& lost) {
    const uint32_t b = ptx::smem_addr(&bar[slot]);
    if (threadIdx.x == 0 && !lost) ptx::mbar_arrive_expect_tx(b, a.warps * kPart * 4);
    if (lane < a.ctas && !lost) ptx::store_async_cluster(ptx::smem_addr(part[slot][w]), b, lane, x);
    // The state is touched after a first look at the barrier: in front of it, it cost the backward 2 to 5 points of
    // the copy rate.
    if (!ptx::mbar_try_wait_cluster(b, phase & 1) || lost) lost = lost || !wait(b, phase, a.limit_ns);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lost ? __int_as_float(0x7fffffff) : 0.f;
#pragma unroll 4
    for (int k = 0; k < a.warps; k += 4 / kPart) {  // the row's tail is zero
      const float4 p = *reinterpret_cast<const float4*>(part[slot][k]);
      if constexpr (N == 1) {
        x[0] += (p.x + p.y) + (p.z + p.w);
      } else {
        x[0] += p.x;
        x[1] += p.y;
        x[2] += p.z;
      }
    }
  }
  // No CTA leaves while another may still send to it.  The barrier has no
  // limit of its own and needs none: every wait before it has one.  A CTA that
  // is not lost has waited for all that was sent to it; one that is gives what
  // the others sent last the time to land.
  __device__ __forceinline__ void finish() {
    __syncwarp();
    ptx::cluster_sync();
    if (*reinterpret_cast<volatile int*>(&given_up)) {
      const uint64_t t0 = ptx::global_timer_ns();
      while (ptx::global_timer_ns() - t0 < kSettleNs) {
      }
    }
  }
};
template <Row kRow, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], Exchange<kRow, N>& ex, int slot, int phase, const NormArgs& a,
                                         int w, int lane, int group, bool& lost) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (kRow != kLanes || o < a.lanes)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (kRow == kLanes || (kRow == kWarps && a.warps == 1)) return;
  ex.sum(v, slot, phase, a, w, lane, group, lost);
}

// Stages of a row ring: two (forward) or three (backward; two for fp32) cover
// HBM's latency with the CTAs that fit.
constexpr int kRingFwd = 2;
template <bool kF32>
constexpr int kRingBwd = kF32 ? 2 : 3;

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

// A load that leaves x as it was unless `on`.  kInPlace: without a copy of x,
// which would wait for an earlier load, and without a branch.  (In clusters 61
// instead of 56% of the copy rate from 8 bits at 4,096 columns.  Elsewhere the
// compiler makes no copies, and this costs registers, to spilling.)
template <bool kInPlace>
__device__ __forceinline__ void load_if(bool on, float& x, const float* p) {
  if constexpr (kInPlace)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.f32 %0, [%1];\n\t}"
                 : "+f"(x)
                 : "l"(p), "r"((uint32_t)on));
  else if (on)
    x = *p;
}
template <bool kInPlace>
__device__ __forceinline__ void load_if(bool on, uint32_t& x, const uint8_t* p) {
  if constexpr (kInPlace)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.u8 %0, [%1];\n\t}"
                 : "+r"(x)
                 : "l"(p), "r"((uint32_t)on));
  else if (on)
    x = *p;
}

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

// Where a thread works: its row group's item.  A row has W warps, or (kLanes:
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
template <Row kRow, class Items>
__device__ __forceinline__ Place place(const NormArgs& a, const Items& items) {
  Place p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, lanes = kRow == kLanes ? a.lanes : 32;
  // (kWide's is 0, but with barriers of a constant number its backward ran at
  // 70 instead of 76% of the copy rate at 2,560 columns.)
  p.group = kRow == kCluster ? 0 : warp / a.warps;
  p.w = kRow == kCluster ? (int)(ptx::cluster_ctarank() * (blockDim.x / 32)) + warp : warp % a.warps;
  p.lane = lane % lanes;
  const int64_t item = kRow == kCluster ? (int64_t)(blockIdx.x / a.ctas)
                                        : (int64_t)blockIdx.x * a.groups + p.group * (32 / lanes) + lane / lanes;
  p.on = item < a.items;
  p.item = p.on ? item : 0;
  p.f = items.frame(p.item);
  p.stride = items.count(p.f);
  const int first = (int)(p.item - items.first(p.f));
  p.r0 = items.start(p.f) + first;
  p.n = p.on ? (int)((items.rows(p.f) - first + p.stride - 1) / p.stride) : 0;
  p.turns = kRow == kLanes ? (int)__reduce_max_sync(0xffffffffu, (unsigned)p.n) : p.n;
  return p;
}

template <class R, int V, bool kCkpt, Row kRow, class Items>
__global__ void __launch_bounds__(kRow == kWide ? 32 * kWideFwd : 128, kRow == kWide ? 2 : kFwdPerSm)
    residual_norm_fwd(const NormArgs a, const __grid_constant__ Items items) {
  using namespace vec;
  __shared__ __align__(16) Exchange<kRow, 1> ex;
  ex.start();
  const Place at = place<kRow>(a, items);
  const int W = a.warps, group = at.group, w = at.w, lane = at.lane, C = a.width, n = at.n;
  const int64_t r0 = at.r0, row_step = (int64_t)at.stride * C;  // elements between the item's rows
  const float inv_c = 1.0f / (float)C;
  extern __shared__ uint4 ring[];
  constexpr int S = kRingFwd, kX = sizeof(R) / 16, kVec = 1 + kX, kElem = sizeof(R) / 8;
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
  bool lost = false;
  for (int i = 0; i < at.turns; ++i) {
    const bool live = kRow != kLanes || i < n;
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
    row_sums(s, ex, 0, i, a, w, lane, group, lost);
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
    row_sums(s, ex, 1, i, a, w, lane, group, lost);
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
  ex.finish();
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

// Both row means come from one exchange: with t = dx' + r_x a (g = t - r_x xh
// m1), sum(b yh) = sum(coef yh t) - r_x m1 sum(coef yh xh), coef = alpha gate
// gamma_post, so the three sums of a xh, coef yh t and coef yh xh give both.
template <class R, int V, bool k8, Row kRow, class Items>
__global__ void __launch_bounds__(kRow == kWide ? 32 * kWideBwd : 128, kRow == kWide ? 2 : kBwdPerSm)
    residual_norm_bwd(const NormArgs a, const __grid_constant__ Items items) {
  using namespace vec;
  __shared__ __align__(16) Exchange<kRow, 3> ex;
  ex.start();
  ptx::grid_launch_next();
  const Place at = place<kRow>(a, items);
  const int W = a.warps, group = at.group, w = at.w, lane = at.lane, C = a.width, n = at.n, stride = at.stride;
  const int64_t r0 = at.r0, row_step = (int64_t)stride * C;  // elements between the item's rows
  const float inv_c = 1.0f / (float)C;
  extern __shared__ uint4 ring[];
  using H = Held<R, k8>;
  constexpr int kG = sizeof(R) / 16, kVec = kG + 1 + H::kPieces, kElem = sizeof(R) / 8;
  constexpr int S = kRingBwd<sizeof(R) == 32>;
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
    const bool on = i < n;
    if (kRow != kCluster && !on) return;
    const float* p = pr + (int64_t)i * stride;
    load_if<kRow == kCluster>(on, s.ry, p);
    load_if<kRow == kCluster>(on, s.rx, p + a.rows);
    if (k8)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t o = i * (row_step / ckpt::kBlock) + v * (vstep / ckpt::kBlock);
        load_if<kRow == kCluster>(on && in[v], s.by[v], sy + o);
        load_if<kRow == kCluster>(on && in[v], s.bx[v], sx + o);
      }
  };
  Small small[2] = {};
  load_small(0, small[0]);
  load_small(1, small[1]);
  const P2 zero = both(0.f);
  Params<V> params;
  params.at = base + S * V * kVec * step;
  params.step = step;
  P2 zs[V][4], ds[V][4];  // sums of the thread's columns of Z and dgamma_pre
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) zs[v][e] = ds[v][e] = zero;
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
  bool lost = false;
  auto row = [&](int i, Small& sm, int slot) {
    P2 y[V][4], x[V][4], t[V][4];
    const bool live = kRow != kLanes || i < n;
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
#pragma unroll
      for (int e = 0; e < 4; ++e) ds[v][e] = fma2(h[e], x[v][e], ds[v][e]);
    }
    rd.next();
    load();
    load_small(i + 2, sm);
    float s[3] = {sum(sa), sum(sb), sum(sc)};
    row_sums(s, ex, slot, i >> 1, a, w, lane, group, lost);
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
#pragma unroll
      for (int e = 0; e < 4; ++e) zs[v][e] = fma2(y[v][e], t[v][e], zs[v][e]);
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
      o.set(zs[v]);
      o.store(a.z_part, at.item * C + col[v]);
      o.set(ds[v]);
      o.store(a.d_part, at.item * C + col[v]);
    }
  ex.finish();
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
  int V, W, L, G, N;  // vectors a thread, warps and lanes a row, rows a CTA works on, CTAs a row
  Row row;
  int warps() const { return N > 1 ? W / N : W * std::max(1, kMaxGroups / W); }  // of a CTA
  int threads() const { return 32 * warps(); }
  int64_t ctas(int64_t items) const { return (items + G - 1) / G * N; }
};
// One vector a thread up to 256 columns, else two (half the instructions a row
// that one takes).  Clusters: the CTAs of two to four warps that leave the
// fewest idle, and the largest of those.
Shape shape_of(int width, int wide) {
  const int vecs = width / 8, V = vecs <= 32 ? 1 : 2, W = (vecs + 32 * V - 1) / (32 * V);
  if (W <= kMaxGroups) {
    const int L = vecs <= 4 ? 4 : vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32;
    return {V, W, L, kMaxGroups / W * (32 / L), 1, L < 32 ? kLanes : kWarps};
  }
  if (W <= wide) return {V, W, 32, 1, 1, kWide};
  int ctas = 0, warps = 0;
  for (int w = kMaxGroups; w >= 2; --w) {
    const int n = (W + w - 1) / w;
    if (n <= kMaxCtas && (!ctas || n * w < ctas * warps)) ctas = n, warps = w;
  }
  return {V, ctas * warps, 32, 1, ctas, kCluster};
}

// A kernel's ring: its opt-in shared memory, and, for more CTAs than SMs, the
// SM's whole share for it (by itself the driver leaves room for fewer CTAs
// than fit).  Set on every launch, as it belongs to the device's context, and
// always to the same value, the ring of the kernel's largest CTA: another
// thread may be about to launch the kernel with more threads than this call's.
template <class K>
cudaError_t allow_ring(K kern, size_t most, bool many) {
  cudaError_t e = cudaSuccess;
  if (most > 40 * 1024)  // up to 48 KB with the static part goes without
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess && many)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  return e;
}

// A kernel's launch with Shape s, for `items` items.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(const Shape& s, int64_t items, size_t smem, cudaStream_t st) {
    cfg.gridDim = dim3((unsigned)s.ctas(items));
    cfg.blockDim = dim3(s.threads());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s.N;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.N > 1 ? 1 : 0;
  }
  Launch(const Launch&) = delete;
};
// thread_bytes: the ring's share of one thread.
template <class K, class Items>
cudaError_t launch(K kern, const NormArgs& a, const Items& it, const Shape& s, int most_threads, size_t thread_bytes,
                   cudaStream_t st) {
  const cudaError_t e = allow_ring(kern, most_threads * thread_bytes, s.ctas(a.items) > a.sms);
  if (e != cudaSuccess) return e;
  if (s.N > 1) g_clusters = true;
  Launch l(s, a.items, s.threads() * thread_bytes, st);
  return cudaLaunchKernelEx(&l.cfg, kern, a, it);
}

// Threads of the largest CTA of a kind of row.
template <Row kRow, bool kBwd>
constexpr int kMostThreads = 32 * (kRow != kWide ? kMaxGroups : kBwd ? kWideBwd : kWideFwd);

template <class R, int V>
constexpr size_t kThreadFwd = kRingFwd * V * (16 + sizeof(R));
template <class R, int V, bool k8>
constexpr size_t kThreadBwd =
    V * 16 * (kRingBwd<sizeof(R) == 32> * (sizeof(R) / 16 + 1 + Held<R, k8>::kPieces) + Params<V>::kPieces);

// Clusters of Shape s that the device runs at once, by the variant that needs
// most: which SMs a cluster may share is the device's, so it is asked once.
template <bool kBwd>
int clusters_at_once(const Shape& s) {
  static std::atomic<int> known[64][kMaxCtas + 1][kMaxGroups + 1];
  int dev = -1, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  std::atomic<int>& k = known[dev][s.N][s.warps()];
  if ((n = k.load()) > 0) return n;
  using vec::F32;
  auto ask = [&](auto kern, size_t thread_bytes) {
    const cudaError_t e = allow_ring(kern, kMostThreads<kCluster, kBwd> * thread_bytes, true);
    Launch l(s, 1, s.threads() * thread_bytes, nullptr);
    return e == cudaSuccess ? cudaOccupancyMaxActiveClusters(&n, kern, &l.cfg) : e;
  };
  const cudaError_t e = kBwd ? ask(residual_norm_bwd<F32, 2, false, kCluster, UniformItems>, kThreadBwd<F32, 2, false>)
                             : ask(residual_norm_fwd<F32, 2, true, kCluster, UniformItems>, kThreadFwd<F32, 2>);
  if (e != cudaSuccess || n < 1) return 1;
  k.store(n);
  return n;
}

// A row of four warps in two CTAs: one exchange that all take part in, then
// some that the second CTA never joins.  Sets bit 0 of `result` for a sum that
// is not as it should be and bit 1 for one that was given up.
__global__ void __launch_bounds__(64) row_wait_selftest(const NormArgs a, unsigned int* result) {
  __shared__ __align__(16) Exchange<kCluster, 3> ex;
  ex.start();
  const int rank = (int)ptx::cluster_ctarank(), lane = threadIdx.x % 32, w = rank * 2 + threadIdx.x / 32;
  bool lost = false;
  for (int n = 0; n < (rank == 0 ? 6 : 1); ++n) {
    float s[3] = {w + 1.f, 10.f * (w + 1), 1.f};
    ex.sum(s, n & 1, n >> 1, a, w, lane, 0, lost);
    const bool right = s[0] == 10.f && s[1] == 100.f && s[2] == 4.f;
    const bool nan = s[0] != s[0] && s[1] != s[1] && s[2] != s[2];
    atomicOr(result, (n == 0 ? right && !lost : nan && lost) ? (n == 0 ? 0u : 2u) : 1u);
  }
  ex.finish();
}

// Calls fn with the type of the stream, the vectors a thread and who shares a row.
template <class Fn>
cudaError_t with_shape(const Shape& s, bool f32, Fn fn) {
  using std::integral_constant;
  auto rows = [&](auto r) {
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    if (s.row == kLanes) return fn(r, one, integral_constant<Row, kLanes>());
    if (s.row == kWide) return fn(r, two, integral_constant<Row, kWide>());
    if (s.row == kCluster) return fn(r, two, integral_constant<Row, kCluster>());
    return s.V == 1 ? fn(r, one, integral_constant<Row, kWarps>()) : fn(r, two, integral_constant<Row, kWarps>());
  };
  return f32 ? rows(vec::F32()) : rows(vec::Bf16());
}

template <class Items>
cudaError_t fwd_all(const NormArgs& a, const Items& it, const Shape& s, cudaStream_t st) {
  return with_shape(s, a.f32, [&](auto r, auto v, auto row) {
    using R = decltype(r);
    constexpr int V = decltype(v)::value;
    constexpr Row kRow = decltype(row)::value;
    constexpr int most = kMostThreads<kRow, false>;
    return a.y8 ? launch(residual_norm_fwd<R, V, true, kRow, Items>, a, it, s, most, kThreadFwd<R, V>, st)
                : launch(residual_norm_fwd<R, V, false, kRow, Items>, a, it, s, most, kThreadFwd<R, V>, st);
  });
}

template <class Items>
cudaError_t bwd_all(const NormArgs& a, const Items& it, int n_frames, const Shape& s, cudaStream_t st) {
  const cudaError_t e = with_shape(s, a.f32, [&](auto r, auto v, auto row) {
    using R = decltype(r);
    constexpr int V = decltype(v)::value;
    constexpr Row kRow = decltype(row)::value;
    auto go = [&](auto eight) {
      constexpr bool k8 = decltype(eight)::value;
      return launch(residual_norm_bwd<R, V, k8, kRow, Items>, a, it, s, kMostThreads<kRow, true>, kThreadBwd<R, V, k8>, st);
    };
    return a.y8 ? go(std::true_type()) : go(std::false_type());
  });
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
template <bool kBwd>
NormItems split(int64_t rows, const Shape& s, const int32_t* spans, int n_frames, int64_t span, int sms) {
  // In CTAs of four warps (which fix the registers a thread).
  constexpr int per_sm = kBwd ? kBwdPerSm : kFwdPerSm;
  const int ctas = std::max(1, per_sm * kMaxGroups / s.warps());
  const int64_t want = std::max<int64_t>(n_frames, s.N > 1 ? clusters_at_once<kBwd>(s) : (int64_t)ctas * sms * s.G);
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
  const Shape s = shape_of(a.width, kWideFwd);
  const NormItems n = split<false>(a.rows, s, spans, n_frames, span, sms);
  a.warps = s.W;
  a.lanes = s.L;
  a.groups = s.G;
  a.ctas = s.N;
  a.items = n.items;
  a.sms = sms;
  return with_items(n, spans, n_frames, span, [&](const auto& it) { return fwd_all(a, it, s, st); });
}

cudaError_t residual_norm_gave_up(bool* gave_up) {
  *gave_up = false;
  if (!g_clusters) return cudaSuccess;
  unsigned int e = 0;
  const cudaError_t rc = cudaMemcpyFromSymbol(&e, g_gave_up, sizeof(e));
  if (rc != cudaSuccess || !e) return rc;
  *gave_up = true;
  e = 0;
  return cudaMemcpyToSymbol(g_gave_up, &e, sizeof(e));
}

cudaError_t launch_row_wait_selftest(unsigned int* result, uint64_t limit_ns, cudaStream_t st) {
  const Shape s = {2, 4, 32, 1, 2, kCluster};
  NormArgs a;
  a.warps = s.W;
  a.ctas = s.N;
  a.limit_ns = limit_ns;
  g_clusters = true;
  Launch l(s, 1, 0, st);
  return cudaLaunchKernelEx(&l.cfg, row_wait_selftest, a, result);
}

NormItems residual_norm_items(int64_t rows, int width, const int32_t* spans, int n_frames, int64_t span, int sms) {
  NormItems r = split<true>(rows, shape_of(width, kWideBwd), spans, n_frames, span, sms);
  r.bytes = 2 * align256(r.items * width * 4);
  return r;
}

cudaError_t launch_residual_norm_backward(NormArgs a, const NormItems& n, const int32_t* spans, int n_frames,
                                          int64_t span, int sms, void* workspace, cudaStream_t st) {
  const Shape s = shape_of(a.width, kWideBwd);
  a.sms = sms;
  a.warps = s.W;
  a.lanes = s.L;
  a.groups = s.G;
  a.ctas = s.N;
  a.items = n.items;
  a.z_part = static_cast<float*>(workspace);
  a.d_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256(n.items * a.width * 4));
  return with_items(n, spans, n_frames, span, [&](const auto& it) { return bwd_all(a, it, n_frames, s, st); });
}

}  // namespace fas
