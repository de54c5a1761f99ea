// The gated feed-forward block and its backward pass:
//   g = x Wg^T   u = x Wu^T   h = act(g) u   y = h Wo^T
//   dh = dy Wo   dg = dh u act'(g)   du = dh act(g)
//   dx = dg Wg + du Wu   dWg = dg^T x   dWu = du^T x   dWo = dy^T h
// act(g) = g sigmoid(z): z = g (silu), or z = 2 sqrt(2/pi) (g + 0.044715 g^3)
// (gelu in its tanh form: (1 + tanh(z / 2)) / 2 is the sigmoid of z).
//
// One kernel does all six products, D[m, n] = sum_k A[m, k] B[n, k], on the
// tensor cores.  An operand's matrix is row-major in memory and is read as it
// lies, whichever of its axes is summed over: blocks of 64 x 64 elements come
// in by TMA (128-byte swizzle), and the descriptors say whether a block's rows
// run along k ("K-major") or along m or n.  Nothing is transposed in memory.
// What differs is the epilogue:
//   kGateUp  a tile holds the gate and the up columns of the same inner
//            features side by side, so both projections, the activation and
//            the product are one kernel and g and u only leave it if the
//            backward pass wants them;
//   kInner   the tile is dh; the kernel reads g and u and writes dg, du and h;
//   kPlain   the tile itself, rounded once, or its fp32 part of a product whose
//            k axis is split over several CTAs.
//
// Accumulators are fp32.  Rounded to bf16 on the way: h and (dg, du), which the
// next product's operands are, each one rounding of the size of the results'
// own; and g and u, where the caller keeps them.  The backward pass that
// computes g and u again for itself holds them in 16 + 8 bits (see Low): with
// bf16 alone the gradients were off by 3.5e-3 of their norm against 64 bits,
// so by 2.3e-3, for 2% of the time.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fas.h"
#include "feed_forward_plan.h"
#include "kernels.h"
#include "ptx.cuh"

namespace fas {
namespace {

using namespace feed_forward;

constexpr uint32_t kBlockBytes = kBlock * kBlock * 2;
constexpr int kEpilogueWarps = 8, kGroups = kEpilogueWarps / 4;  // four warps a group, a group its share of the columns

// TMA producer, MMA issuer, epilogue, and kInner's mover.
__host__ __device__ constexpr int threads(Epilogue e) { return 64 + 32 * kEpilogueWarps + (e == kInner ? 32 : 0); }

// One product's D [m, n] and its tiles.  A launch does one, or two with the
// same k and operand layouts (the gradients of both weights).
struct Problem {
  int64_t m = 0, n = 0;    // kGateUp, kInner: n = inner features
  int mt = 0, nt = 0;      // tiles
  void* out = nullptr;     // kPlain: bf16 [m, n]; kGateUp: h [m, n] (may be null)
};

struct GemmParams {
  Problem d[2];
  int tiles = 0;           // of both
  int whole = 0;           // the first so many tiles are done whole, ...
  int splits = 1;          // ... the others by so many CTAs (or pairs) each, along k (kPlain)
  int ksteps = 0;          // of 64
  float* parts = nullptr;  // their fp32 parts, a tile each
  void* gu = nullptr;      // kGateUp: g and u [m, 2n] (may be null)
  uint16_t* low = nullptr; // their low parts [m, n] (may be null), written by kGateUp, read by kInner through Maps::low
  int silu = 1;
  uint64_t limit_ns = 0;
};

// What a launch reads and writes by TMA: each problem's operands, ...
template <bool kStaged>
struct Maps {
  CUtensorMap a[2], b[2];
};
// ... and kInner's matrices [m, n].
template <>
struct Maps<true> {
  CUtensorMap a[2], b[2], g, u, low, dg, du, h;
};

// kInner's g and u come in, and dg, du and h go out, through two sets of three
// 128 x 64 tiles in shared memory.  Loads and stores by threads, each of its
// own row, reach 32 different lines an instruction; where the sum over the
// width is short they bounded the kernel (40,000 x 1024 x 2048: 262 us, this
// way 199; at a width of 2048, where it costs two operand stages, 293 and 302).
constexpr uint32_t kTileBytes = 2 * kBlockBytes, kSetBytes = 3 * kTileBytes;

// Set where a wait was given up.
__device__ unsigned int g_gave_up;
std::atomic<bool> g_launched{false};

constexpr int kMostStages = 6;
// Operand stages of 64 elements of k that fit shared memory.
__host__ __device__ constexpr int stages(Epilogue e, int G, int BN) { return e != kInner && BN / G == 128 ? 6 : 4; }
__host__ __device__ constexpr uint32_t stage_bytes(int G, int BN) { return (128 + BN / G) / kBlock * kBlockBytes; }
constexpr size_t smem_bytes(Epilogue e, int G, int BN) {
  return 1024 + (size_t)stages(e, G, BN) * stage_bytes(G, BN) + (e == kInner ? 2 * kSetBytes : 0);
}
struct Bars {
  uint64_t full[kMostStages];
  uint64_t empty[kMostStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t ready[2];  // kInner: g and u are in a set; what was there before is out
  uint64_t done[2];   // the epilogue's warps have written a set
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// A wait that ends: false where the CTA has given up, or gives up now.  No
// global word is read, so one call's lost wait says nothing about the next.
// kPair: for what the other CTA of the pair did.  Whoever waits sleeps: at the
// power cap the warps' polling costs the products' clock (together with the
// operands' L2 policy 2% of 14,960 x 2048 x 5504 in long runs).
template <bool kPair>
__device__ __forceinline__ bool wait(uint64_t* barrier, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  const uint32_t bar = ptx::smem_addr(barrier);
  if (kPair ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (kPair ? ptx::mbar_try_wait_cluster_sleep(bar, parity, 20000u) : ptx::mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if ((it & 7u) != 0u) continue;
    if (*abort) return false;
    const uint64_t now = ptx::global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit_ns) {
      *abort = 1;
      atomicOr(&g_gave_up, 1u);
      return false;
    }
  }
}

// Time for what no barrier counts any more, once a CTA or its partner has given up.
constexpr uint64_t kLostNs = 1000000;

// The same for what is under way to this CTA: it has to have come before the
// CTA ends, given up or not.
template <bool kPair>
__device__ __forceinline__ void settle(uint64_t* barrier, uint32_t parity, uint64_t limit_ns) {
  const uint32_t bar = ptx::smem_addr(barrier);
  const uint64_t t0 = ptx::global_timer_ns();
  while (!(kPair ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)))
    if (ptx::global_timer_ns() - t0 > max(limit_ns, kLostNs)) {
      atomicOr(&g_gave_up, 1u);
      return;
    }
}

__host__ __device__ constexpr uint32_t idesc(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
  return ptx::idesc_bf16_f32(m, n, b_mn) | ((a_mn ? 1u : 0u) << 15);
}

// A tile's operand in shared memory: blocks of 8 KB along m or n.  K-major, a
// block's rows are m or n and the blocks follow one another like rows of one
// matrix; otherwise its rows are k and the blocks are the descriptor's leading
// stride apart.  16 k elements on: 32 bytes, or 16 rows.
__device__ __forceinline__ uint64_t operand(uint32_t at) { return ptx::smem_desc_sw128(at, kBlockBytes, 1024); }
template <bool kMn>
__device__ __forceinline__ constexpr uint64_t k_step(int k) { return (uint64_t)((kMn ? k * 2048 : k * 32) >> 4); }

// Work item t: a tile, or a part of one of the last tiles.  (32-bit numbers:
// the divisions here lie between one tile's loads and the next's.)
struct Tile {
  int which;      // problem
  int m, n;
  int k0, k1;     // steps
  int part;       // number of the part, or -1: whole
};
// Tiles in runs of kRun along m, so that those in flight share rows of A and of B in L2 (8: 1% more).
constexpr int kRun = 16;
__device__ __forceinline__ int work_items(const GemmParams& p) { return p.whole + (p.tiles - p.whole) * p.splits; }
__device__ __forceinline__ void locate(const GemmParams& p, int t, Tile& r) {
  const int first = p.d[0].mt * p.d[0].nt;
  r.which = t >= first;
  if (r.which) t -= first;
  const Problem& d = p.d[r.which];
  const int per = kRun * d.nt, g = t / per, i = t - g * per;
  const int rows = min(kRun, d.mt - g * kRun);
  r.n = rows == kRun ? i / kRun : i / rows;
  r.m = g * kRun + i - r.n * rows;
}
__device__ __forceinline__ Tile tile_at(const GemmParams& p, int t) {
  Tile r;
  r.k0 = 0;
  r.k1 = p.ksteps;
  r.part = -1;
  if (t >= p.whole) {
    const int per = (p.ksteps + p.splits - 1) / p.splits, tail = (t - p.whole) / p.splits;
    r.part = t - p.whole;
    r.k0 = (r.part - tail * p.splits) * per;
    r.k1 = min(p.ksteps, r.k0 + per);
    t = p.whole + tail;
  }
  locate(p, t, r);
  return r;
}

// The operand stages in turn; `parity` of the use at hand.
template <int kStages>
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++s == kStages) {
      s = 0;
      parity ^= 1u;
    }
  }
};

// z with act(g) = g sigmoid(z), and dz / dg.  Beyond 30 the gelu's sigmoid is 0 or 1.
__device__ __forceinline__ void gate_arg(float g, bool silu, float& z, float& gc, float& dz) {
  if (silu) {
    z = gc = g;
    dz = 1.f;
  } else {
    constexpr float kC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(gc) : "f"(g), "f"(-30.f));  // NaN stays
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(gc) : "f"(gc), "f"(30.f));
    const float q = 0.044715f * gc * gc;
    z = kC * gc * (1.f + q);
    dz = kC * (1.f + 3.f * q);
  }
}
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + ptx::ex2(-1.4426950408889634f * z)); }
__device__ __forceinline__ float activation(float g, bool silu) {
  float z, gc, dz;
  gate_arg(g, silu, z, gc, dz);
  return g * sigmoid(z);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 16 bf16 of a row, of which the first `valid` (0, 8 or 16) exist.  A whole
// 32-byte sector in one access where the address allows it.
__device__ __forceinline__ void store16(uint16_t* p, const uint32_t (&w)[8], int valid) {
  if (valid >= 16 && (reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
    return;
  }
  if (valid >= 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  if (valid >= 16) *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}
// What bf16 leaves of a value in [2^E, 2^(E+1)), at most 2^(E-8), in 128ths of
// that (127 at most): an error of up to 2^-8 becomes one of 2^-16, at a tie
// 2^-15.  The parts of g and u share 16 bits.  E is kept within -96 and 111:
// what lies below is not worth its bits, what lies above keeps those of a
// smaller E.
struct Low {
  static __device__ __forceinline__ uint32_t power(uint32_t bits) {  // of 2^E
    return min(max(bits & 0x7F800000u, 0x0F800000u), 0x77000000u);
  }
  static __device__ __forceinline__ uint32_t of(float left, uint32_t bits) {  // a signed byte
    int q;
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(q) : "f"(left * __uint_as_float(0x7F000000u + (15u << 23) - power(bits))));
    return (uint32_t)q;
  }
  static __device__ __forceinline__ float add(int byte, float hi) {
    return fmaf((float)byte, __uint_as_float(power(__float_as_uint(hi)) - (15u << 23)), hi);
  }
  static __device__ __forceinline__ uint32_t both(float g, float u) {
    const uint32_t hi = ptx::pack_bf16x2(g, u), gb = hi << 16, ub = hi & 0xFFFF0000u;
    return __byte_perm(of(g - __uint_as_float(gb), gb), of(u - __uint_as_float(ub), ub), 0x5540) & 0xFFFFu;
  }
};

__device__ __forceinline__ void pack16(const float (&v)[16], uint32_t (&w)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = ptx::pack_bf16x2(v[2 * e], v[2 * e + 1]);
}

// 16 bf16 as two 16-byte pieces of a swizzled row in shared memory.
__device__ __forceinline__ void put16(uint8_t* row, int piece, int swizzle, const float (&v)[16]) {
  uint32_t w[8];
  pack16(v, w);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    *reinterpret_cast<uint4*>(row + (((piece + k) ^ swizzle) << 4)) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
}
__device__ __forceinline__ void get16(const uint8_t* row, int piece, int swizzle, float (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + (((piece + k) ^ swizzle) << 4));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[8 * k + 2 * e] = bf16_lo(u[e]), v[8 * k + 2 * e + 1] = bf16_hi(u[e]);
  }
}

// kInner's 64 columns of a set: this thread's row, its group's half of them.
// Tiles of g, u and their low parts (where there are any); dg, du and h take
// their place.
__device__ __forceinline__ void write_inner(uint32_t acc, uint8_t* set, int row, int group, bool silu, bool low) {
  uint8_t* at = set + row * 128;  // two blocks of 64 rows of 128 bytes follow one another
  const int swizzle = row & 7;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = group * 32 + i * 16, piece = c / 8;
    uint32_t a[16];
    ptx::tmem_ld16(acc + c, a);
    float g[16], u[16], h[16];
    get16(at, piece, swizzle, g);
    get16(at + kTileBytes, piece, swizzle, u);
    if (low) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 w = *reinterpret_cast<const uint4*>(at + 2 * kTileBytes + (((piece + k) ^ swizzle) << 4));
        const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t v = b[e / 2] >> (16 * (e & 1));
          g[8 * k + e] = Low::add((int8_t)v, g[8 * k + e]);
          u[8 * k + e] = Low::add((int8_t)(v >> 8), u[8 * k + e]);
        }
      }
    }
    ptx::tmem_ld_wait(a);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float dh = __uint_as_float(a[e]), ue = u[e];
      float z, gc, dz;
      gate_arg(g[e], silu, z, gc, dz);
      const float s = sigmoid(z), act = g[e] * s;
      h[e] = act * ue;
      u[e] = dh * act;
      g[e] = dh * ue * (s * fmaf(gc * (1.f - s), dz, 1.f));
    }
    put16(at, piece, swizzle, g);
    put16(at + kTileBytes, piece, swizzle, u);
    put16(at + 2 * kTileBytes, piece, swizzle, h);
  }
}

template <int kRows, int kSubs>
struct Size {};

// A thread's row of an accumulator of BN columns: its group's output columns, kCols from c0 on.
template <int BN, Epilogue kE>
struct Output {
  static constexpr int kTileCols = kE == kGateUp ? BN / 2 : BN, kCols = kTileCols / kGroups, kChunks = kCols / 16;
  const GemmParams& p;
  const Problem& d;
  int64_t row, col;
  int c0;
  float* part;  // this row's place among a tile's fp32 parts, or null

  // tile_row: of the kRows rows of the tile; sub: which of its accumulators.
  template <int kRows, int kSubs>
  __device__ __forceinline__ Output(const GemmParams& p_, const Tile& t, Size<kRows, kSubs>, int tile_row, int sub, int group)
      : p(p_), d(p_.d[kE == kPlain ? t.which : 0]), row((int64_t)t.m * kRows + tile_row),
        col((int64_t)(t.n * kSubs + sub) * kTileCols + group * kCols), c0(group * kCols), part(nullptr) {
    if constexpr (kE == kPlain)
      if (t.part >= 0) part = p.parts + (((int64_t)t.part * kRows + tile_row) * kSubs + sub) * BN + c0;
  }
  // How many of chunk i's columns exist.
  __device__ __forceinline__ int valid(int i) const {
    return row < d.m ? (int)max((int64_t)0, min((int64_t)16, d.n - (col + i * 16))) : 0;
  }
  __device__ __forceinline__ void put(void* to, int64_t width, int64_t shift, int i, const float (&v)[16]) {
    uint32_t w[8];
    pack16(v, w);
    store16(static_cast<uint16_t*>(to) + row * width + shift + col + i * 16, w, valid(i));
  }

  __device__ __forceinline__ void plain(int i, const uint32_t (&a)[16]) {
    if (part) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        reinterpret_cast<uint4*>(part + i * 16)[e] = make_uint4(a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3]);
    } else {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(a[e]);
      put(d.out, d.n, 0, i, v);
    }
  }

  __device__ __forceinline__ void gate_up(int i, const uint32_t (&a)[16], const uint32_t (&b)[16]) {
    float g[16], u[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) g[e] = __uint_as_float(a[e]), u[e] = __uint_as_float(b[e]);
    if (p.gu) {
      put(p.gu, 2 * d.n, 0, i, g);
      put(p.gu, 2 * d.n, d.n, i, u);
    }
    if (p.low) {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = Low::both(g[2 * e], u[2 * e]) | Low::both(g[2 * e + 1], u[2 * e + 1]) << 16;
      store16(p.low + row * d.n + col + i * 16, w, valid(i));
    }
    if (d.out) {
#pragma unroll
      for (int e = 0; e < 16; ++e) g[e] = activation(g[e], p.silu) * u[e];
      put(d.out, d.n, 0, i, g);
    }
  }

  // Out of the accumulator at `acc`, which `release` gives back.
  template <class Release>
  __device__ __forceinline__ void write(uint32_t acc, const Release& release) {
#pragma unroll 1
    for (int i = 0; i < kChunks; ++i) {
      uint32_t a[16];
      ptx::tmem_ld16(acc + c0 + i * 16, a);
      if constexpr (kE == kPlain) {
        ptx::tmem_ld_wait(a);
        plain(i, a);
      } else {
        uint32_t b[16];
        ptx::tmem_ld16(acc + kTileCols + c0 + i * 16, b);
        ptx::tmem_ld_wait(a);
        ptx::tmem_ld_wait(b);
        gate_up(i, a, b);
      }
    }
    release();
  }
  // The same where the next tile waits for the accumulator: all of it into
  // registers first.
  template <class Release>
  __device__ __forceinline__ void write_behind(uint32_t acc, const Release& release) {
    static_assert(kE == kPlain);
    uint32_t a[kChunks][16];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) ptx::tmem_ld16(acc + c0 + i * 16, a[i]);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) ptx::tmem_ld_wait(a[i]);
    release();
#pragma unroll
    for (int i = 0; i < kChunks; ++i) plain(i, a[i]);
  }
};

// Tiles of 128 G x BN by one CTA (G = 1) or a pair of CTAs (G = 2), persistent.
// In a pair each CTA holds its 128 rows of A and of the accumulator and half of
// B's tile; the leader's MMAs read both halves, so a byte of B is fetched once
// for 256 rows.  Up to 256 columns TMEM holds two accumulators, so that a
// tile's epilogue runs beside the next one's products.  Tiles of 512 columns
// fill it with one, in two halves: the next tile's first steps go into the left
// half while the right one is still read out.  What that costs (about 2 us a
// tile) long sums win back: the bytes that the SMs fetch from L2, which bound
// these products (without A's, a run of the 256-column tiles takes 22% less), go
// down by a quarter.
template <int G, int BN, bool kAMn, bool kBMn, Epilogue kE>
__global__ void __launch_bounds__(threads(kE), 1)
    feed_forward_gemm(const __grid_constant__ Maps<kE == kInner> maps, const __grid_constant__ GemmParams p) {
  constexpr bool kPair = G == 2;
  constexpr int kRows = 128, BM = kRows * G, kBBlocks = BN / G / kBlock;
  constexpr int kSubs = BN > 256 ? 2 : 1, SN = BN / kSubs, kSubBlocks = kBBlocks / kSubs;  // an MMA's columns
  constexpr int kAccs = kSubs > 1 ? 1 : 2, kStages = stages(kE, G, BN);
  constexpr uint32_t kABytes = kRows / kBlock * kBlockBytes, kStageBytes = stage_bytes(G, BN);
  constexpr uint32_t kIdesc = idesc(BM, SN, kAMn, kBMn), kTmemCols = kAccs * BN;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  const uint32_t ring = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u, sets = ring + kStages * kStageBytes;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = kPair ? ptx::cluster_ctarank() : 0u;
  volatile int* abort = &bars.abort;
  const int first = blockIdx.x / G, step = gridDim.x / G, work = work_items(p);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&bars.full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_addr(&bars.acc_full[b]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars.acc_empty[b]), kEpilogueWarps * G);
      ptx::mbar_init(ptx::smem_addr(&bars.ready[b]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars.done[b]), kEpilogueWarps);
    }
    ptx::mbar_init(ptx::smem_addr(&bars.drain), 1);
    bars.abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    if constexpr (kPair) {
      ptx::tmem_alloc_pair(ptx::smem_addr(&bars.tmem_base), kTmemCols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(ptx::smem_addr(&bars.tmem_base), kTmemCols);
      ptx::tmem_relinquish();
    }
  }
  __syncwarp();
  ptx::tc_fence_before_sync();
  __syncthreads();
  if constexpr (kPair) ptx::cluster_sync();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = bars.tmem_base;
  ptx::grid_wait_previous();  // what came before is in memory

  if (warp == 0) {
    if (lane == 0) {
      // Operands stay in L2 ahead of what is written (kInner at 79,200 x 2048 x 5504: 1.65 -> 1.62 ms).
      const uint64_t keep = ptx::policy_evict_last();
      Ring<kStages> ring_at;
      int64_t fill = 0;
      bool ok = true;
      for (int t = first; ok && t < work; t += step) {
        const Tile tile = tile_at(p, t);
        const CUtensorMap *map_a = &maps.a[0], *map_b = &maps.b[0];
        if (kE == kPlain && tile.which) map_a = &maps.a[1], map_b = &maps.b[1];
        for (int kk = tile.k0; kk < tile.k1; ++kk, ++fill, ring_at.next()) {
          const int s = ring_at.s;
          ok = wait<kPair>(&bars.empty[s], ring_at.parity ^ 1u, abort, p.limit_ns);  // (the first uses wait for nothing)
          if (!ok) break;
          // Both CTAs' bytes count on the leader's barrier, which its MMAs wait for.
          const uint32_t dst = ring + s * kStageBytes;
          uint32_t bar = ptx::smem_addr(&bars.full[s]);
          if (rank == 0) ptx::mbar_arrive_expect_tx(bar, G * kStageBytes);
          if constexpr (kPair) bar = ptx::cluster_addr(bar, 0);
          auto load = [&](uint32_t to, const CUtensorMap* map, bool mn, int at) {
            const int c0 = mn ? at : kk * kBlock, c1 = mn ? kk * kBlock : at;
            if constexpr (kPair) ptx::tma_load_2d_pair_hint(to, map, bar, c0, c1, keep);
            else ptx::tma_load_2d_hint(to, map, bar, c0, c1, keep);
          };
#pragma unroll
          for (int i = 0; i < kRows / kBlock; ++i)
            load(dst + i * kBlockBytes, map_a, kAMn, tile.m * BM + (int)rank * kRows + i * kBlock);
#pragma unroll
          for (int i = 0; i < kBBlocks; ++i) {
            const int j = (int)rank * kSubBlocks + i % kSubBlocks;  // of the MMA's columns
            int at = tile.n * BN + (i / kSubBlocks) * SN + j * kBlock;
            if constexpr (kE == kGateUp) {  // half an MMA's columns are gate rows, the others up rows
              constexpr int kHalf = SN / kBlock / 2;
              at = (tile.n * kSubs + i / kSubBlocks) * (SN / 2) + (j % kHalf) * kBlock + (j >= kHalf ? (int)p.d[0].n : 0);
            }
            load(dst + kABytes + i * kBlockBytes, map_b, kBMn, at);
          }
        }
      }
      // The last stages' arrivals, from MMAs of the leader, come before the CTA
      // ends; where it has given up, its copies in flight.
      for (int64_t f = max((int64_t)0, fill - kStages); f < fill; ++f) {
        const int s = (int)(f % kStages);
        const uint32_t parity = (uint32_t)(f / kStages) & 1u;
        if (ok) ok = wait<kPair>(&bars.empty[s], parity, abort, p.limit_ns);
        if (!ok && rank == 0) settle<false>(&bars.full[s], parity, p.limit_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && ptx::elect_one()) {
      auto commit = [](uint64_t* bar) {  // to the barrier of both CTAs of a pair
        if constexpr (kPair) {
          ptx::mma_commit_pair(ptx::cluster_addr(ptx::smem_addr(bar), 0));
          ptx::mma_commit_pair(ptx::cluster_addr(ptx::smem_addr(bar), 1));
        } else {
          ptx::mma_commit(ptx::smem_addr(bar));
        }
      };
      Ring<kStages> at;
      int it = 0;
      bool ok = true;
      for (int t = first; ok && t < work; t += step, ++it) {
        const Tile tile = tile_at(p, t);
        const int span = tile.k1 - tile.k0;
        auto arrived = [&](const Ring<kStages>& r) {
          ok = wait<kPair>(&bars.full[r.s], r.parity, abort, p.limit_ns);
          ptx::tc_fence_after_sync();
          return ok;
        };
        auto multiply = [&](int stage, uint32_t acc, int sub, bool add) {
          const uint32_t from = ring + (uint32_t)stage * kStageBytes;
          const uint64_t a = operand(from), b = operand(from + kABytes + sub * kSubBlocks * kBlockBytes);
#pragma unroll
          for (int k = 0; k < kBlock / 16; ++k) {
            if constexpr (kPair) ptx::mma_ss_pair(acc + sub * SN, a + k_step<kAMn>(k), b + k_step<kBMn>(k), kIdesc, add || k > 0);
            else ptx::mma_ss(acc + sub * SN, a + k_step<kAMn>(k), b + k_step<kBMn>(k), kIdesc, add || k > 0);
          }
        };
        if constexpr (kSubs == 1) {
          const int b = it & 1;
          ok = wait<kPair>(&bars.acc_empty[b], (uint32_t)(it >> 1 & 1) ^ 1u, abort, p.limit_ns);
          ptx::tc_fence_after_sync();
          for (int i = 0; ok && i < span; ++i, at.next()) {
            if (!arrived(at)) break;
            multiply(at.s, tmem + b * BN, 0, i > 0);
            commit(&bars.empty[at.s]);
          }
          if (ok) commit(&bars.acc_full[b]);
        } else {
          const int lead = min(span, kStages);
          const uint32_t parity = (uint32_t)(it & 1) ^ 1u;
          ok = wait<kPair>(&bars.acc_empty[0], parity, abort, p.limit_ns);
          ptx::tc_fence_after_sync();
          Ring<kStages> ahead = at;
          for (int i = 0; ok && i < lead; ++i, ahead.next())
            if (arrived(ahead)) multiply(ahead.s, tmem, 0, i > 0);
          if (ok) ok = wait<kPair>(&bars.acc_empty[1], parity, abort, p.limit_ns);
          ptx::tc_fence_after_sync();
          for (int i = 0; ok && i < span; ++i, at.next()) {
            if (i >= lead) {
              if (!arrived(at)) break;
              multiply(at.s, tmem, 0, true);
            }
            multiply(at.s, tmem, 1, i > 0);
            commit(&bars.empty[at.s]);
          }
          if (ok) commit(&bars.acc_full[0]);
        }
      }
      commit(&bars.drain);
      settle<kPair>(&bars.drain, 0, p.limit_ns);
    }
    __syncwarp();
  } else if (warp == 2 + kEpilogueWarps) {
    if constexpr (kE == kInner) {
      if (lane == 0) {
        // The mover: chunk q, 64 columns of a tile, passes through set q % 2.
        // What the epilogue has written goes out, and once it is read the g
        // and u of chunk q + 2 come in.
        constexpr int kChunks = BN / kBlock;
        const int64_t chunks = first < work ? (int64_t)((work - first + step - 1) / step) * kChunks : 0;
        auto origin = [&](int64_t q, int64_t& row, int64_t& col) {
          const Tile tile = tile_at(p, first + (int)(q / kChunks) * step);
          row = (int64_t)tile.m * BM + rank * kRows;
          col = (int64_t)tile.n * BN + (q % kChunks) * kBlock;
        };
        auto fetch = [&](int64_t q) {
          const uint32_t bar = ptx::smem_addr(&bars.ready[q & 1]), set = sets + (uint32_t)(q & 1) * kSetBytes;
          int64_t row, col;
          origin(q, row, col);
          ptx::mbar_arrive_expect_tx(bar, (p.low ? 3 : 2) * kTileBytes);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (p.low) ptx::tma_load_2d(set + 2 * kTileBytes + i * kBlockBytes, &maps.low, bar, (int)col, (int)row + i * kBlock);
            ptx::tma_load_2d(set + i * kBlockBytes, &maps.g, bar, (int)col, (int)row + i * kBlock);
            ptx::tma_load_2d(set + kTileBytes + i * kBlockBytes, &maps.u, bar, (int)col, (int)row + i * kBlock);
          }
        };
        int64_t fetched = min((int64_t)2, chunks);
        for (int64_t q = 0; q < fetched; ++q) fetch(q);
        bool ok = true;
        for (int64_t q = 0; q < chunks; ++q) {
          ok = wait<false>(&bars.done[q & 1], (uint32_t)(q >> 1) & 1u, abort, p.limit_ns);
          if (!ok) break;
          const uint32_t set = sets + (uint32_t)(q & 1) * kSetBytes;
          int64_t row, col;
          origin(q, row, col);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int64_t r = row + i * kBlock;
            if (r >= p.d[0].m || col >= p.d[0].n) continue;  // nothing of the block exists
            ptx::tma_store_2d(&maps.dg, set + i * kBlockBytes, (int)col, (int)r);
            ptx::tma_store_2d(&maps.du, set + kTileBytes + i * kBlockBytes, (int)col, (int)r);
            ptx::tma_store_2d(&maps.h, set + 2 * kTileBytes + i * kBlockBytes, (int)col, (int)r);
          }
          ptx::bulk_commit();
          if (fetched < chunks) {
            ptx::bulk_wait_read();
            fetch(fetched++);
          }
        }
        if (!ok) {  // copies in flight land before the CTA ends (a bounded wait)
          for (int64_t q = max((int64_t)0, fetched - 2); q < fetched; ++q)
            settle<false>(&bars.ready[q & 1], (uint32_t)(q >> 1) & 1u, p.limit_ns);
        }
        ptx::bulk_wait();
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp % 4, group = (warp - 2) / 4;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const int row = quarter * 32 + lane;
    auto release = [&](int b) {
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        const uint32_t bar = ptx::smem_addr(&bars.acc_empty[b]);
        if constexpr (kPair) ptx::mbar_arrive_cluster(ptx::cluster_addr(bar, 0));
        else ptx::mbar_arrive(bar);
      }
    };
    int it = 0;
    int64_t q = 0;
    bool ok = true;
    for (int t = first; ok && t < work; t += step, ++it) {
      const int b = kSubs == 1 ? it & 1 : 0, round = kSubs == 1 ? it >> 1 : it;  // the accumulator, and which use of it
      ok = __all_sync(0xffffffffu, wait<kPair>(&bars.acc_full[b], (uint32_t)round & 1u, abort, p.limit_ns));
      if (!ok) break;
      ptx::tc_fence_after_sync();
      const uint32_t acc = tmem + b * BN + lanes;
      if constexpr (kE == kInner) {
#pragma unroll 1
        for (int c = 0; c < BN; c += kBlock, ++q) {
          ok = __all_sync(0xffffffffu, wait<false>(&bars.ready[q & 1], (uint32_t)(q >> 1) & 1u, abort, p.limit_ns));
          if (!ok) break;
          write_inner(acc + c, smem_raw + (sets - ptx::smem_addr(smem_raw)) + (q & 1) * kSetBytes, row, group, p.silu, p.low != nullptr);
          ptx::fence_proxy_async_smem();  // this before the mover's stores and loads
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&bars.done[q & 1]));
        }
        release(b);
      } else {
        const Tile tile = tile_at(p, t);
#pragma unroll 1
        for (int sub = 0; sub < kSubs; ++sub) {
          Output<SN, kE> out(p, tile, Size<BM, kSubs>(), rank * kRows + row, sub, group);
          if constexpr (kSubs > 1) out.write_behind(acc + sub * SN, [&] { release(b + sub); });
          else out.write(acc, [&] { release(b); });
        }
      }
    }
    __syncwarp();
  }

  // Neither CTA of a pair ends, or frees its TMEM, while the other may still
  // signal it or read its operands.  The MMAs' arrivals come from the tensor
  // pipe, which no barrier of the threads orders: the producers have waited for
  // those on the stages, the epilogues for the accumulators', and the last one,
  // which follows all MMAs, both CTAs wait for here (the leader has).
  ptx::tc_fence_before_sync();
  __syncthreads();
  if constexpr (kPair) {
    if (warp == 1) {
      if (lane == 0) settle<true>(&bars.drain, 0, p.limit_ns);
      __syncwarp();
    }
    if (threadIdx.x == 0 && *abort) ptx::store_cluster(ptx::cluster_addr(ptx::smem_addr(&bars.abort), rank ^ 1u), 1u);
    __syncwarp();
    ptx::cluster_sync();
  }
  if (*abort) {
    const uint64_t t0 = ptx::global_timer_ns();
    while (ptx::global_timer_ns() - t0 < kLostNs) {
    }
    __syncwarp();
  }
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    if constexpr (kPair) ptx::tmem_dealloc_pair(tmem, kTmemCols);
    else ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// Few tokens: the weights' bytes bound it, and a tile of 128 rows of A would
// be mostly empty (few_gate_up and few_out say up to how many).
// Out[f, n] = sum_k W[f, k] X[n, k] by mma.sync with 16 rows of W as its m and
// 8 tokens as its n, fed from memory without staging: which elements of k an
// instruction takes together is free as long as both operands agree, so a lane
// loads 16 consecutive bytes of its row of W and of X and four lanes cover 64
// bytes of a row.  The warps of a CTA share the rows and split k; their fp32
// parts meet in shared memory and are added in order.
// Warps of a CTA: the product onto the width has few rows, each long.
constexpr int few_warps(bool gate) { return gate ? 8 : 16; }

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kGate: rows f and rows + f of w are gate and up of inner feature f, and out
// is act(g) u, gu both and low their low parts (each null: not stored); else
// out is the product.
template <int kTiles, bool kGate>
__global__ void __launch_bounds__(kGate ? 256 : 512, kGate ? 3 : 2)
    feed_forward_few(const uint16_t* x, const uint16_t* w, uint16_t* out, uint16_t* gu, uint16_t* low, int tokens, int64_t rows,
                     int64_t k, int silu) {
  constexpr int kMats = kGate ? 2 : 1, kN = kTiles * 8, kFewWarps = kGate ? 8 : 16;
  constexpr int kFewUnroll = kGate && kTiles > 1 ? 2 : 4;  // steps of 32 elements whose loads are in flight
  __shared__ float part[kFewWarps][kMats][16][kN + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const int64_t row0 = (int64_t)blockIdx.x * 16;
  float c[kMats][kTiles][4] = {};
  const uint16_t *pw[kMats][2], *px[kTiles];  // rows beyond the last read the last; their results are not stored
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) pw[m][r] = w + (m * rows + min(row0 + g + 8 * r, rows - 1)) * k + q * 8;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) px[t] = x + min(t * 8 + g, tokens - 1) * k + q * 8;
  const int64_t steps = (k + 31) / 32, per = (steps + kFewWarps - 1) / kFewWarps;
  const int64_t s0 = warp * per, s1 = min(steps, s0 + per);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load = [&](const uint16_t* p, int64_t s) {
    return s < s1 && s * 32 + q * 8 < k ? *reinterpret_cast<const uint4*>(p + s * 32) : zero;
  };
  uint4 a[kFewUnroll][kMats][2], b[kFewUnroll][kTiles];
  ptx::grid_wait_previous();
  for (int64_t s = s0; s < s1; s += kFewUnroll) {
#pragma unroll
    for (int u = 0; u < kFewUnroll; ++u) {
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) a[u][m][r] = load(pw[m][r], s + u);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) b[u][t] = load(px[t], s + u);
    }
#pragma unroll
    for (int u = 0; u < kFewUnroll; ++u)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
          mma_16x8x16(c[m][t], a[u][m][0].x, a[u][m][1].x, a[u][m][0].y, a[u][m][1].y, b[u][t].x, b[u][t].y);
          mma_16x8x16(c[m][t], a[u][m][0].z, a[u][m][1].z, a[u][m][0].w, a[u][m][1].w, b[u][t].z, b[u][t].w);
        }
  }
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[warp][m][g + (e / 2) * 8][t * 8 + q * 2 + (e & 1)] = c[m][t][e];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * kN; i += kFewWarps * 32) {
    const int r = i % 16, n = i / 16;
    const int64_t f = row0 + r;
    if (f >= rows || n >= tokens) continue;
    float v[kMats] = {};
#pragma unroll
    for (int p = 0; p < kFewWarps; ++p)
#pragma unroll
      for (int m = 0; m < kMats; ++m) v[m] += part[p][m][r][n];
    auto store = [](uint16_t* p, float y) { *p = (uint16_t)ptx::pack_bf16x2(y, 0.f); };
    if constexpr (kGate) {
      if (gu) {
        store(gu + n * 2 * rows + f, v[0]);
        store(gu + n * 2 * rows + rows + f, v[1]);
      }
      if (low) low[n * rows + f] = (uint16_t)Low::both(v[0], v[1]);
      if (out) store(out + n * rows + f, activation(v[0], silu) * v[1]);
    } else {
      store(out + n * rows + f, v[0]);
    }
  }
}

// The parts of the tiles that were split along k, added in order.  A CTA takes
// 2048 elements of a tile, a thread eight.
template <int BM, int BN>
__global__ void __launch_bounds__(256) feed_forward_join(const __grid_constant__ GemmParams p) {
  constexpr int kPer = BM * BN / 2048;
  ptx::grid_wait_previous();
  const int tail = (int)(blockIdx.x / kPer);
  const int at = (int)(blockIdx.x % kPer) * 2048 + threadIdx.x * 8;
  Tile t;
  locate(p, p.whole + tail, t);
  const Problem& d = p.d[t.which];
  const int64_t row = (int64_t)t.m * BM + at / BN, col = (int64_t)t.n * BN + at % BN;
  if (row >= d.m || col >= d.n) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const float* part = p.parts + (int64_t)tail * p.splits * (BM * BN) + at;
#pragma unroll 4
  for (int k = 0; k < p.splits; ++k, part += BM * BN) {
    const float4 x = reinterpret_cast<const float4*>(part)[0], y = reinterpret_cast<const float4*>(part)[1];
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
  }
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = ptx::pack_bf16x2(v[2 * e], v[2 * e + 1]);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(d.out) + row * d.n + col) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A row-major bf16 matrix (columns of a wider one where `row` is given) in blocks of 64 x 64.
int matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t row = 0) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(row ? row : cols) * 2};
  const cuuint32_t box[2] = {kBlock, kBlock};
  return bf16_tensor_map(map, base, 2, dims, strides, box);
}
// The two halves of a [rows, 2 inner] matrix, each bounded by itself: a block
// across the first one's edge must not touch the second.
int both_maps(CUtensorMap* first, CUtensorMap* second, const void* both, int64_t rows, int64_t inner) {
  const int rc = matrix_map(first, both, rows, inner, 2 * inner);
  return rc != FAS_OK ? rc : matrix_map(second, static_cast<const uint16_t*>(both) + inner, rows, inner, 2 * inner);
}

struct Matrix {
  const void* at;
  int64_t rows, cols;
};

// out[m, n] = A B^T summed over k.
struct Product {
  int64_t m, n;
  Matrix a, b;
  void* out;
};

struct Launcher {
  Machine machine;
  uint64_t limit_ns;
  cudaStream_t st;
  int launches = 0;

  // Starts while the kernel before it ends: every kernel here waits for that
  // one's results before it touches memory.
  template <class K, class... Args>
  int start(K kern, int64_t grid, int threads, size_t smem, int cluster, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    ++launches;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? FAS_OK : FAS_ERR_CUDA;
  }

  template <int kForm, bool kAMn, bool kBMn, Epilogue kE, int kN>
  int go(GemmParams p, const Product (&products)[kN], int64_t k, const Spread& s, Maps<kE == kInner> maps) {
    constexpr int G = kForms[kForm].G, kBm = 128 * G, kBn = kForms[kForm].cols, kOut = kE == kGateUp ? kBn / 2 : kBn;
    int64_t tiles = 0;
    for (int i = 0; i < kN; ++i) {
      const Product& d = products[i];
      if (matrix_map(&maps.a[i], d.a.at, d.a.rows, d.a.cols) != FAS_OK || matrix_map(&maps.b[i], d.b.at, d.b.rows, d.b.cols) != FAS_OK)
        return FAS_ERR_CUDA;
      p.d[i] = {d.m, d.n, (int)((d.m + kBm - 1) / kBm), (int)((d.n + kOut - 1) / kOut), d.out};
      tiles += (int64_t)p.d[i].mt * p.d[i].nt;
    }
    if (tiles > INT32_MAX / 2) return FAS_ERR_UNSUPPORTED;  // and a step of the grid on still counts in 32 bits
    p.tiles = (int)tiles;
    p.whole = s.parts ? (int)s.whole : p.tiles;
    p.splits = s.splits;
    p.ksteps = (int)((k + kBlock - 1) / kBlock);
    p.limit_ns = limit_ns;
    auto kern = feed_forward_gemm<G, kBn, kAMn, kBMn, kE>;
    const size_t smem = smem_bytes(kE, G, kBn);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return FAS_ERR_CUDA;
    g_launched = true;
    const int rc = start(kern, std::min<int64_t>(p.whole + s.parts, machine.units(G)) * G, threads(kE), smem, G, maps, p);
    if (rc != FAS_OK || s.parts == 0) return rc;
    return start(feed_forward_join<kBm, kBn>, (int64_t)(p.tiles - p.whole) * (kBm * kBn / 2048), 256, 0, 1, p);
  }

  // out[n, f] = sum_k x[n, k] w[f, k] for a few tokens (kGate: see feed_forward_few).
  template <bool kGate>
  int few(const void* x, const void* w, void* out, void* gu, uint16_t* low, int64_t tokens, int64_t rows, int64_t k, bool silu) {
    auto go = [&](auto tiles) {
      return start(feed_forward_few<decltype(tiles)::value, kGate>, (rows + 15) / 16, few_warps(kGate) * 32, 0, 1,
                   static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), static_cast<uint16_t*>(out),
                   static_cast<uint16_t*>(gu), low, (int)tokens, rows, k, (int)silu);
    };
    if (tokens <= 8) return go(std::integral_constant<int, 1>());
    if (tokens <= 16) return go(std::integral_constant<int, 2>());
    return go(std::integral_constant<int, 4>());
  }

  template <bool kAMn, bool kBMn, Epilogue kE, int kN>
  int run(const GemmParams& p, const Product (&products)[kN], int64_t k, const Spread& s, const Maps<kE == kInner>& maps = {}) {
    if constexpr (kE == kPlain)
      if (s.form == 2) return go<2, kAMn, kBMn, kE>(p, products, k, s, maps);
    return s.form == 1 ? go<1, kAMn, kBMn, kE>(p, products, k, s, maps) : go<0, kAMn, kBMn, kE>(p, products, k, s, maps);
  }
};

// h, g and u, and the low parts of g and u from x, those that are given.
int project(Launcher& l, const FeedForwardArgs& a, void* h, void* gu, uint16_t* low) {
  const int64_t N = a.tokens, C = a.width, F = a.inner;
  if (few_gate_up(N, F)) return l.few<true>(a.x, a.w_in, h, gu, low, N, F, C, a.activation == FAS_ACT_SILU);
  GemmParams p;
  p.gu = gu;
  p.low = low;
  p.silu = a.activation == FAS_ACT_SILU;
  const Product d[1] = {{N, F, {a.x, N, C}, {a.w_in, 2 * F, C}, h}};
  return l.run<false, false, kGateUp>(p, d, C, spread(kGateUp, N, 2 * F, C, l.machine));
}

}  // namespace

// Of pairs of CTAs, as many run at once as the device takes of the kernel that
// it takes fewest of: the plan, the workspace and every launch go by that.
int feed_forward_pairs(int sms, int* pairs) {
  static std::atomic<int> known[64];  // + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FAS_ERR_CUDA;
  *pairs = known[dev] - 1;
  if (*pairs >= 0) return FAS_OK;
  int most = sms / 2;
  auto of = [&](auto kern, Epilogue e, int cols) {
    const size_t smem = smem_bytes(e, 2, cols);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max(2, sms / 2 * 2));
    cfg.blockDim = dim3(threads(e));
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return false;
    most = std::min(most, n);
    return true;
  };
  if (!of(feed_forward_gemm<2, 256, false, false, kGateUp>, kGateUp, 256) ||
      !of(feed_forward_gemm<2, 256, false, true, kInner>, kInner, 256) ||
      !of(feed_forward_gemm<2, 256, false, false, kPlain>, kPlain, 256) ||
      !of(feed_forward_gemm<2, 256, false, true, kPlain>, kPlain, 256) ||
      !of(feed_forward_gemm<2, 256, true, true, kPlain>, kPlain, 256) ||
      !of(feed_forward_gemm<2, 512, false, false, kPlain>, kPlain, 512) ||
      !of(feed_forward_gemm<2, 512, false, true, kPlain>, kPlain, 512) ||
      !of(feed_forward_gemm<2, 512, true, true, kPlain>, kPlain, 512))
    return FAS_ERR_CUDA;
  known[dev] = most + 1;
  *pairs = most;
  return FAS_OK;
}

int64_t feed_forward_workspace(int64_t tokens, int width, int inner, bool backward, bool kept, int sms, int pairs) {
  return Workspace(tokens, width, inner, backward, kept, {sms, pairs}).bytes;
}

int launch_feed_forward(const FeedForwardArgs& a, void* workspace, int* launches, cudaStream_t stream) {
  const int64_t N = a.tokens, C = a.width, F = a.inner;
  const Machine machine = {a.sms, a.pairs};
  const Workspace ws(N, a.width, a.inner, false, true, machine);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  Launcher l{machine, a.limit_ns, stream};
  int rc = project(l, a, w + ws.h, a.kept_out, nullptr);
  GemmParams p;
  p.parts = reinterpret_cast<float*>(w + ws.parts);
  const Product y[1] = {{N, C, {w + ws.h, N, F}, {a.w_out, C, F}, a.y}};
  if (rc == FAS_OK) {
    rc = few_out(N, C, F) ? l.few<false>(w + ws.h, a.w_out, a.y, nullptr, nullptr, N, C, F, false)
                          : l.run<false, false, kPlain>(p, y, F, spread(kPlain, N, C, F, machine));
  }
  *launches = l.launches;
  return rc;
}

int launch_feed_forward_backward(const FeedForwardArgs& a, void* workspace, int* launches, cudaStream_t stream) {
  const int64_t N = a.tokens, C = a.width, F = a.inner;
  const Machine machine = {a.sms, a.pairs};
  const Workspace ws(N, a.width, a.inner, true, a.kept != nullptr, machine);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  Launcher l{machine, a.limit_ns, stream};
  uint16_t* const low = a.kept ? nullptr : reinterpret_cast<uint16_t*>(w + ws.low);
  int rc = a.kept ? FAS_OK : project(l, a, nullptr, w + ws.gu, low);
  const Matrix x{a.x, N, C}, dy{a.dy, N, C}, w_in{a.w_in, 2 * F, C}, w_out{a.w_out, C, F}, h{w + ws.h, N, F},
      dgu{w + ws.dgu, N, 2 * F};
  GemmParams p;
  p.silu = a.activation == FAS_ACT_SILU;
  Maps<true> maps;
  if (rc == FAS_OK) rc = both_maps(&maps.g, &maps.u, a.kept ? a.kept : w + ws.gu, N, F);
  if (rc == FAS_OK) rc = both_maps(&maps.dg, &maps.du, dgu.at, N, F);
  if (rc == FAS_OK) rc = matrix_map(&maps.h, h.at, N, F);
  p.low = low;
  if (rc == FAS_OK && low) rc = matrix_map(&maps.low, low, N, F);
  const Product dh[1] = {{N, F, dy, w_out, nullptr}};
  if (rc == FAS_OK) rc = l.run<false, true, kInner>(p, dh, C, spread(kInner, N, F, C, machine), maps);
  GemmParams q;
  q.parts = reinterpret_cast<float*>(w + ws.parts);
  const Product dx[1] = {{N, C, dgu, w_in, a.dx}};
  if (rc == FAS_OK) rc = l.run<false, true, kPlain>(q, dx, 2 * F, spread(kPlain, N, C, 2 * F, machine));
  const Product dw[2] = {{2 * F, C, dgu, x, a.dw_in}, {C, F, dy, h, a.dw_out}};
  if (rc == FAS_OK) rc = l.run<true, true, kPlain>(q, dw, N, spread_weights(N, C, F, machine));
  *launches = l.launches;
  return rc;
}

// One tile whose sum takes longer than the limit (2^24 terms, at least 20 ms):
// its epilogues give up, while the loads and products go on to their end.
int launch_product_wait_selftest(unsigned int* result, uint64_t limit_ns, int sms, int pairs, cudaStream_t st) {
  constexpr int64_t kTerms = 1 << 24, kSide = 8;
  uint8_t* memory = nullptr;
  constexpr int64_t kOperand = kTerms * kSide * 2, kMatrix = 256;  // a small matrix [8, 8]; both: [8, 16]
  if (cudaMalloc(&memory, kOperand + 4 * kMatrix) != cudaSuccess) return FAS_ERR_CUDA;
  uint8_t *out = memory + kOperand, *gu = out + kMatrix, *dgu = gu + kMatrix, *h = dgu + kMatrix;
  const Matrix rows{memory, kSide, kTerms}, cols{memory, kTerms, kSide};
  Launcher l{{sms, pairs}, limit_ns, st};
  GemmParams p;
  Maps<true> inner;
  Spread one;
  int rc = cudaMemsetAsync(memory, 0, kOperand + 4 * kMatrix, st) == cudaSuccess ? FAS_OK : FAS_ERR_CUDA;
  if (rc == FAS_OK) rc = both_maps(&inner.g, &inner.u, gu, kSide, kSide);
  if (rc == FAS_OK) rc = both_maps(&inner.dg, &inner.du, dgu, kSide, kSide);
  if (rc == FAS_OK) rc = matrix_map(&inner.h, h, kSide, kSide);
  unsigned int gave_up = 0;
  auto next = [&](int launched) {  // the word is left set after the last
    if (rc == FAS_OK) rc = launched;
    if (rc != FAS_OK) return;
    bool lost = false;
    if (cudaStreamSynchronize(st) != cudaSuccess || feed_forward_gave_up(&lost) != cudaSuccess) rc = FAS_ERR_CUDA;
    gave_up += lost;
  };
  const Product plain[1] = {{kSide, kSide, rows, rows, out}}, wide[1] = {{kSide, kSide, cols, cols, out}};
  const Product gate[1] = {{kSide, kSide, rows, {memory, 2 * kSide, kTerms / 2}, out}}, dh[1] = {{kSide, kSide, rows, cols, nullptr}};
  for (one.form = 0; one.form < 3; ++one.form) {
    next(l.run<false, false, kPlain>(p, plain, kTerms, one));
    next(l.run<true, true, kPlain>(p, wide, kTerms, one));
    if (one.form < 2) next(l.run<false, false, kGateUp>(p, gate, kTerms / 2, one));
    if (one.form < 2) next(l.run<false, true, kInner>(p, dh, kTerms, one, inner));
  }
  const unsigned int right = 2, set = 1;
  if (rc == FAS_OK && gave_up == 10 &&
      (cudaMemcpyToSymbol(g_gave_up, &set, sizeof(set)) != cudaSuccess ||
       cudaMemcpy(result, &right, sizeof(right), cudaMemcpyHostToDevice) != cudaSuccess))
    rc = FAS_ERR_CUDA;
  return cudaFree(memory) == cudaSuccess ? rc : FAS_ERR_CUDA;
}

cudaError_t feed_forward_gave_up(bool* gave_up) {
  *gave_up = false;
  if (!g_launched) return cudaSuccess;
  unsigned int e = 0;
  const cudaError_t rc = cudaMemcpyFromSymbol(&e, g_gave_up, sizeof(e));
  if (rc != cudaSuccess || !e) return rc;
  *gave_up = true;
  e = 0;
  return cudaMemcpyToSymbol(g_gave_up, &e, sizeof(e));
}

}  // namespace fas
