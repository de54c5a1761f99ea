// Backward pass of the frame-aligned sparse attention for sm_103a.
//
// With s = 1/sqrt(d), for row i and the keys j its frame sees:
//   P_ij = exp(s q_i.k_j - lse_i)          (recomputed, lse from the forward)
//   delta_i = sum_c dout_ic out_ic         dS_ij = P_ij (dout_i.v_j - delta_i)
//   dq_i = s sum_j dS_ij k_j    dk_j = s sum_i dS_ij q_i    dv_j = sum_i P_ij dout_i
// Visibility is symmetric in the frames, so the queries that see a key frame
// are the same table ranges that the frame's own queries see, and both
// passes walk the plan's work list ("Deleting the Mask": the visible tokens
// are at most two contiguous ranges).
//
// Two kernels.  The query pass owns 128 query rows and accumulates dq over
// the visible keys; the key pass owns 128 key rows and accumulates dk and dv
// over the queries that see them.  Together they compute S and dP twice (7
// products for the 5 that the gradients need), but every gradient stays in
// TMEM until its one store: no fp32 gradient goes through memory, no atomics,
// bit-reproducible results.  One kernel for all five has not been built.  By
// count it would not lose: its operands take some 1660 clocks of shared-memory
// bandwidth a block of 64 queries (dS is stored there for two more operands),
// these two kernels' products 1790 of the tensor pipe.  It would add 64 KB of
// fp32 reductions to L2 a pair of tiles, whose order has to be fixed for
// results to stay bit-reproducible.
//
// At d = 128 bound by the tensor pipe and, on long runs, by power: 6 heads of
// 22 frames of 3600 take 11.8 to 12.1 ms (with the clock), 1.16 to 1.20
// PFLOP/s of the five products and 1.63 to 1.67 of the seven executed, 0.96 to
// 0.99 of the rate that the library's bf16 product sustains (1.70); 16 heads of
// 17 frames of 880, 1.54 ms (1.10).  At d = 64 the exponentials and their
// conversions bound it, which both kernels compute (0.79 PFLOP/s of five on
// the frames of 880, 0.88 on those of 3600).
//
// A visible range is walked in blocks; its last block is shortened to the
// tokens it has (a multiple of 16) through the MMA's N or its K steps, so no
// hidden token enters a product, whatever it holds, and no mask is needed.
//
// Precision: S, dP, the gradients, P and dS are fp32; P and dS are rounded to
// bf16 as operands of the products, as P is in the forward.  Since sum_j
// dS_ij = 0 up to out's rounding, a common component c of the keys cancels in
// dq, but the roundings of dS times c do not: the query pass sums what
// rounding added to each row and takes it out along c (the mean of the first
// 64 keys), which leaves the roundings times k - c.  (On keys with a common
// component of three times their spread, as the prepass's mean-centring is
// for, dq's error against 64 bits is 2.4e-3, dk's and dv's; 5.5e-3 without.)

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention_core.cuh"
#include "fas.h"
#include "internal.h"
#include "kernels.h"
#include "ptx.cuh"

namespace fas {
namespace {

using core::drain_wait;

constexpr int kRowsB = kQTile;  // rows of a work item (MMA M)
// Softmax warpgroups: all work on the same block, each on a third of its
// columns.  (Two, each on a half, run their exponentials in lockstep and leave
// the special-function unit idle under everything else: the mid geometry's
// query pass took 698 us instead of 652, the key pass 788 instead of 773.)
constexpr int kSoftGroups = 3;
constexpr int kSoftThreads = 128 * kSoftGroups;
constexpr int kWarpK = 4 * kSoftGroups, kWarpV = kWarpK + 1, kWarpMma = kWarpK + 2, kWarpMean = kWarpK + 3;
constexpr int kThreadsB = 32 * (kWarpMean + 1);
constexpr int kMaxStagesB = 6;
constexpr uint32_t kTmemAll = 512;

// Blocks of one item's two visible ranges.
struct Blocks {
  int4 r;
  int nb0, nb;
  int B;
  __device__ __forceinline__ Blocks(int4 rng, int b) : r(rng), nb0((rng.y + b - 1) / b), B(b) {
    nb = nb0 + (rng.w + b - 1) / b;
  }
  __device__ __forceinline__ int start(int j) const { return j < nb0 ? r.x + j * B : r.z + (j - nb0) * B; }
  __device__ __forceinline__ int count(int j) const {
    const int left = j < nb0 ? r.y - j * B : r.w - (j - nb0) * B;
    return left < B ? left : B;
  }
};

struct BarsB {
  uint64_t tile_full;
  uint64_t full[2][kMaxStagesB];   // [ring][stage]
  uint64_t empty[2][kMaxStagesB];
  uint64_t s_full, dp_full;
  uint64_t s_free, dp_free;        // query pass: S, dP read into registers
  uint64_t p_full[2], ds_full;     // P (in two parts) and dS stored as bf16
  uint64_t acc_done;               // query pass: dQ(j) has read dS(j)
  uint64_t acc_full, drain;
  uint32_t tmem_base;
  int abort, skip;
};

__device__ __forceinline__ void init_bars(BarsB& b) {
  auto one = [](uint64_t& x, int n) { ptx::mbar_init(ptx::smem_addr(&x), n); };
  one(b.tile_full, 1);
  for (int i = 0; i < 2; ++i) {
    for (int s = 0; s < kMaxStagesB; ++s) {
      one(b.full[i][s], 1);
      one(b.empty[i][s], 1);
    }
  }
  one(b.s_full, 1);
  one(b.dp_full, 1);
  one(b.s_free, kSoftThreads);
  one(b.dp_free, kSoftThreads);
  one(b.p_full[0], kSoftThreads);
  one(b.p_full[1], kSoftThreads);
  one(b.ds_full, kSoftThreads);
  one(b.acc_done, 1);
  one(b.acc_full, 1);
  one(b.drain, 1);
  b.abort = 0;
  ptx::fence_mbar_init();
  ptx::fence_proxy_async_smem();
}

// 1D bulk copy (16-byte aligned addresses, bytes a multiple of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// x as the sum of three bf16 values (24 bits: exact to fp32 rounding) in the
// first three elements of a 16-byte row, the others zero; infinities and NaN
// in the first alone.
__device__ __forceinline__ uint4 split3(float x) {
  const uint32_t a = ptx::pack_bf16x2(x, 0.f) & 0xFFFFu;
  if ((a & 0x7F80u) == 0x7F80u) return make_uint4(a, 0u, 0u, 0u);
  const float r1 = x - __uint_as_float(a << 16);
  const uint32_t b = ptx::pack_bf16x2(r1, 0.f) & 0xFFFFu;
  const float r2 = r1 - __uint_as_float(b << 16);
  return make_uint4(a | b << 16, ptx::pack_bf16x2(r2, 0.f) & 0xFFFFu, 0u, 0u);
}

// Descriptor of a K-major operand without swizzle: 8-row groups of 128 bytes
// (16 bytes a row) one after the other, the next 8 columns lbo_bytes on.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t lbo_bytes) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo_bytes >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)(128u >> 4) << 32) | (1ull << 46);
}

__device__ __forceinline__ void mul_f32x2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// Loads `kRows` tokens of a head from token `first` as a K-major tile of 64-
// column halves, in boxes of kBox tokens (one tensor map serves tiles and
// blocks of every size).  A tile's rows past the frame's end are the next
// frame's (or zeros past the last token): every row of a tile is computed by
// itself, and those are never stored.
template <int D>
constexpr int kBox = D == 64 ? 16 : 32;
template <int D, int kRows>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int first, int h) {
  static_assert(kRows % kBox<D> == 0, "");
#pragma unroll
  for (int half = 0; half < D / 64; ++half)
#pragma unroll
    for (int r = 0; r < kRows; r += kBox<D>)
      ptx::tma_load_3d(dst + half * (kRows * 128) + r * 128, tm, bar, half * 64, first + r, h);
}

// One ring's producer: block j into stage j % depth.  kStats: the tokens'
// softmax statistics (kStatBytes each, two arrays) travel with the block.
constexpr uint32_t kStatBytes = 16;
template <int D, int B, bool kStats>
__device__ __forceinline__ void produce(BarsB& bars, int ring, const CUtensorMap* tm, int depth, uint32_t s0, int h,
                                        const Blocks& blk, const BwdParams& p, uint32_t stat_s0) {
  constexpr uint32_t kBytes = B * D * 2;
  volatile int* abort_flag = &bars.abort;
  int j = 0;
  bool ok = true;
  for (; j < blk.nb; ++j) {
    const int st = j % depth, u = j / depth;
    if (j == depth) ptx::grid_wait_previous();  // a bounded wait must not count the previous kernel's time
    if (u >= 1)
      ok = ptx::mbar_wait<true>(ptx::smem_addr(&bars.empty[ring][st]), (u - 1) & 1, abort_flag, p.err,
                                kErrWaitProducer, p.limit_ns);
    if (!ok) break;
    const uint32_t fb = ptx::smem_addr(&bars.full[ring][st]);
    const uint32_t nb = kStats ? (uint32_t)blk.count(j) * kStatBytes : 0;
    ptx::mbar_arrive_expect_tx(fb, kBytes + 2 * nb);
    load_rows<D, B>(s0 + st * kBytes, tm, fb, blk.start(j), h);
    if (kStats) {
      const uint8_t* src = p.stats + ((int64_t)h * p.N + blk.start(j)) * kStatBytes;
      bulk_load(stat_s0 + st * (2 * B * kStatBytes), src, nb, fb);
      bulk_load(stat_s0 + st * (2 * B * kStatBytes) + B * kStatBytes, src + (int64_t)p.H * p.N * kStatBytes, nb, fb);
    }
  }
  if (!ok)  // let every copy this thread started land before the CTA exits
    for (int i = (j > depth ? j - depth : 0); i < j; ++i)
      drain_wait(ptx::smem_addr(&bars.full[ring][i % depth]), (i / depth) & 1, p.err, p.limit_ns);
}

// D[128 x n] = A[128 x D] . B^T, A in TMEM (bf16 pairs) or K-major shared
// memory, B the first n rows of a K-major block of kB rows.
template <int D, int kB, bool kATmem, bool kAdd = false>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a_tmem, uint64_t a_desc, uint64_t b_desc, int n) {
  const uint32_t idesc = ptx::idesc_bf16_f32(kRowsB, (uint32_t)n, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t b = b_desc + (((kk >> 2) * (kB * 128) + (kk & 3) * 32) >> 4);
    if (kATmem)
      ptx::mma_ts(d, a_tmem + kk * 8, b, idesc, kAdd || kk > 0 ? 1u : 0u);
    else
      ptx::mma_ss(d, a_desc + (((kk >> 2) * (kRowsB * 128) + (kk & 3) * 32) >> 4), b, idesc, kAdd || kk > 0 ? 1u : 0u);
  }
}

// D[128 x D] += A[128 x n] . B[n x D]: A's bf16 chunks of 16 columns in TMEM,
// kStride columns apart (8 each), B a block read along its rows.
// kPart 0, 1: the first or the last chunks of each warpgroup's share of the
// block (released in that order); 2: all.
template <int kB>
constexpr int kFirstChunks = (kB / 16 / kSoftGroups + 1) / 2;
template <int D, int kB, int kStride, int kPart>
__device__ __forceinline__ void mma_acc(uint32_t d, uint32_t a, uint64_t b_desc, int n, bool first) {
  constexpr uint32_t idesc = ptx::idesc_bf16_f32(kRowsB, D, true);
#pragma unroll
  for (int kk = 0; kk < kB / 16; ++kk)
    if ((kPart == 2 || (kk % (kB / 16 / kSoftGroups) < kFirstChunks<kB>) == (kPart == 0)) && (n == kB || kk * 16 < n))
      ptx::mma_ts(d, a + kk * kStride, b_desc + ((kk * 2048) >> 4), idesc, (!first || kk > 0) ? 1u : 0u);
}

// A 128-row K-major tile into TMEM as an A operand.
template <int D>
__device__ __forceinline__ void tile_to_tmem(uint32_t col, uint64_t desc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    ptx::tmem_cp_128x256b(col + kk * 8, desc + (((kk >> 2) * (kRowsB * 128) + (kk & 3) * 32) >> 4));
}

// Writes 16 columns of an fp32 accumulator row, scaled, as bf16.
__device__ __forceinline__ void store_acc(uint32_t taddr, uint16_t* dst, float scale, bool valid) {
  uint32_t o[16], pk[8];
  ptx::tmem_ld16(taddr, o);
  ptx::tmem_ld_wait(o);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    pk[e] = ptx::pack_bf16x2(__uint_as_float(o[2 * e]) * scale, __uint_as_float(o[2 * e + 1]) * scale);
  if (valid) {
    uint4* d4 = reinterpret_cast<uint4*>(dst);
    d4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    d4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
  }
}

// Common start of both kernels: error check, barriers, TMEM.
#define FAS_BWD_PROLOGUE()                                                                          \
  if (threadIdx.x == 0) bars.skip = *reinterpret_cast<volatile unsigned int*>(p.err) != 0u;          \
  __syncthreads();                                                                                   \
  if (bars.skip) {                                                                                   \
    ptx::grid_wait_previous(); /* what follows this kernel must also follow the one before */       \
    return;                                                                                          \
  }                                                                                                  \
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;                                        \
  const int4 item = p.work[blockIdx.x];                                                              \
  const int h = item.x, f = item.y, tile = item.z;                                                   \
  const int2 sp = p.spans[f];                                                                        \
  if (threadIdx.x == 0) init_bars(bars);                                                             \
  if (warp == kWarpMma) {                                                                            \
    ptx::tmem_alloc(ptx::smem_addr(&bars.tmem_base), kTmemAll);                                      \
    ptx::tmem_relinquish();                                                                          \
  }                                                                                                  \
  ptx::tc_fence_before_sync();                                                                       \
  __syncthreads();                                                                                   \
  ptx::tc_fence_after_sync();                                                                        \
  const uint32_t tmem = bars.tmem_base;                                                              \
  volatile int* abort_flag = &bars.abort

// ------------------------------------------------------------- query pass
//
// Q and dO of the tile sit in TMEM as A operands; K and V blocks of 96 keys
// (144 at d = 64) stream through two rings.  The warpgroups work on the same
// block, and dS has its own place in TMEM, so S(j+1) only needs S(j) to have
// been read into registers, dP(j+1) the same of dP(j), and the tensor pipe runs
// S(j+1), dP(j+1) while block j is exponentiated.  Tensor order: S(j+1),
// dP(j+1), dQ(j).
//
// 96 keys: S, dP (fp32) and dS (bf16) take 240 columns beside dq, Q and dO; at
// d = 64 there is room for 144, and the softmax warps, which bound it, pay
// their waits less often (8.8 -> 8.0 ms on 6 heads x 22 x 3600, both passes).
// Blocks of 128 with dS in dP's columns chain dS(j), dQ(j), dP(j+1) and left
// the pipe 57% busy; blocks of 64 in two buffers, 52% (an MMA of N = 64 takes
// 32 clocks, less than the issue of the next).
template <int D>
constexpr int kBk = D == 64 ? 144 : 96;  // keys per block

template <int D>
struct QLayout {
  static constexpr uint32_t kAcc = 0, kS = D, kDp = kS + kBk<D>, kDs = kDp + kBk<D>, kQ = kDs + kBk<D> / 2, kDo = kQ + D / 2;
  static_assert(kDo + D / 2 <= kTmemAll, "TMEM columns");
  static constexpr uint32_t kTile = kRowsB * D * 2, kBlock = kBk<D> * D * 2;
  static constexpr int kStages = 3;  // per ring
  static constexpr size_t kSmem = 1024 + 2 * kTile + 2 * kStages * kBlock;
};

template <int D>
__global__ void __launch_bounds__(kThreadsB, 1)
    attention_bwd_q(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const BwdParams p) {
  using L = QLayout<D>;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ BarsB bars;
  __shared__ float red[kSoftGroups][kRowsB];  // delta, then what rounding added to the rows by group
  __shared__ __align__(16) float centre[D];
  const uint32_t q_s = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u, do_s = q_s + L::kTile;
  const uint32_t k_s0 = do_s + L::kTile, v_s0 = k_s0 + S * L::kBlock;
  ptx::grid_launch_next();
  FAS_BWD_PROLOGUE();
  const Blocks blk(p.table[f], kBk<D>);

  if (warp == kWarpK || warp == kWarpV) {
    if (lane == 0) {
      if (warp == kWarpK) {
        const uint32_t tb = ptx::smem_addr(&bars.tile_full);
        ptx::mbar_arrive_expect_tx(tb, 2 * L::kTile);
        load_rows<D, kRowsB>(q_s, &tm_q, tb, sp.x + tile * kRowsB, h);
        load_rows<D, kRowsB>(do_s, &tm_do, tb, sp.x + tile * kRowsB, h);
        produce<D, kBk<D>, false>(bars, 0, &tm_k, S, k_s0, h, blk, p, 0);
        if (bars.abort) drain_wait(tb, 0, p.err, p.limit_ns);
      } else {
        produce<D, kBk<D>, false>(bars, 1, &tm_v, S, v_s0, h, blk, p, 0);
      }
    }
  } else if (warp == kWarpMma) {
    if (ptx::elect_one()) {
      auto wait = [&](uint64_t& b, int parity) {
        return ptx::mbar_wait<false>(ptx::smem_addr(&b), parity & 1, abort_flag, p.err, kErrWaitMma, p.limit_ns);
      };
      const uint64_t kd = ptx::smem_desc_sw128(k_s0, 16, 1024), vd = ptx::smem_desc_sw128(v_s0, 16, 1024);
      const uint64_t kmn = ptx::smem_desc_sw128(k_s0, kBk<D> * 128, 1024);
      constexpr uint64_t kStep = L::kBlock >> 4;
      int ks = 0, kph = 0, vs = 0, vph = 0, os = 0;  // ring positions: S's K, dP's V, dQ's K
      auto s_mma = [&](int n) {
        if (!wait(bars.full[0][ks], kph)) return false;
        mma_rows<D, kBk<D>, true>(tmem + L::kS, tmem + L::kQ, 0, kd + ks * kStep, n);
        ptx::mma_commit(ptx::smem_addr(&bars.s_full));
        if (++ks == S) {
          ks = 0;
          kph ^= 1;
        }
        return true;
      };
      auto dp_mma = [&](int n) {
        if (!wait(bars.full[1][vs], vph)) return false;
        mma_rows<D, kBk<D>, true>(tmem + L::kDp, tmem + L::kDo, 0, vd + vs * kStep, n);
        ptx::mma_commit(ptx::smem_addr(&bars.dp_full));
        ptx::mma_commit(ptx::smem_addr(&bars.empty[1][vs]));
        if (++vs == S) {
          vs = 0;
          vph ^= 1;
        }
        return true;
      };
      bool ok = wait(bars.tile_full, 0);
      int n = blk.count(0);
      if (ok) {
        tile_to_tmem<D>(tmem + L::kQ, ptx::smem_desc_sw128(q_s, 16, 1024));
        tile_to_tmem<D>(tmem + L::kDo, ptx::smem_desc_sw128(do_s, 16, 1024));
        ok = s_mma(n) && dp_mma(n);
      }
      for (int j = 0; ok && j < blk.nb; ++j) {
        const bool more = j + 1 < blk.nb;
        const int n1 = more ? blk.count(j + 1) : 0;
        if (more) {
          ok = wait(bars.s_free, j);
          ptx::tc_fence_after_sync();
          ok = ok && s_mma(n1) && wait(bars.dp_free, j);
          ptx::tc_fence_after_sync();
          ok = ok && dp_mma(n1);
        }
        ok = ok && wait(bars.ds_full, j);
        if (!ok) break;
        ptx::tc_fence_after_sync();
        mma_acc<D, kBk<D>, 8, 2>(tmem + L::kAcc, tmem + L::kDs, kmn + os * kStep, n, j == 0);
        ptx::mma_commit(ptx::smem_addr(&bars.acc_done));
        ptx::mma_commit(ptx::smem_addr(&bars.empty[0][os]));
        if (++os == S) os = 0;
        n = n1;
      }
      ptx::mma_commit(ptx::smem_addr(&bars.acc_full));
      ptx::mma_commit(ptx::smem_addr(&bars.drain));
      drain_wait(ptx::smem_addr(&bars.drain), 0, p.err, p.limit_ns);
      if (!ok) bars.abort = 1;
    }
    __syncwarp();
  } else if (warp == kWarpMean) {
    // The mean of the first keys the rows see (64 at most): the lane's D / 32
    // columns.  Needed by the epilogue alone.
    constexpr int E = D / 32;
    const int n = min(blk.r.y, 64);
    const uint16_t* src = p.k + (int64_t)h * p.head_stride + (int64_t)blk.r.x * p.row_stride + lane * E;
    float c[E] = {};
#pragma unroll 16
    for (int r = 0; r < n; ++r)  // n is a multiple of 16
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(src + r * p.row_stride)[e];
        c[2 * e] += __uint_as_float(w << 16);
        c[2 * e + 1] += __uint_as_float(w & 0xFFFF0000u);
      }
#pragma unroll
    for (int e = 0; e < E; ++e) centre[lane * E + e] = c[e] / (float)n;
    ptx::named_barrier_arrive(2, kSoftThreads + 32);
  } else {
    const int g = warp / 4, trow = (warp % 4) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
    const int row = tile * kRowsB + trow;
    const bool valid = row < sp.y;
    const int64_t token = (int64_t)sp.x + row, at = (int64_t)h * p.head_stride + token * p.row_stride;
    auto wait = [&](uint64_t& b, int parity) {
      const bool got = ptx::mbar_wait<false>(ptx::smem_addr(&b), parity & 1, abort_flag, p.err, kErrWaitSoftmax,
                                             p.limit_ns);
      return (bool)__all_sync(0xffffffffu, got);
    };
    const float lse = valid ? p.lse[(int64_t)h * p.N + token] : INFINITY;
    // delta: D / 8 lanes read a row of out and of dout, each of 8 warps 16 rows.
    if (warp < 8) {
      constexpr int kLanes = D / 8, kPer = 32 / kLanes;
      const int sub = lane / kLanes, c = lane % kLanes;
      uint4 a[16 / kPer], b[16 / kPer];
#pragma unroll
      for (int i = 0; i < 16 / kPer; ++i) {
        const int r = tile * kRowsB + warp * 16 + i * kPer + sub;
        a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < sp.y) {
          const int64_t o = (int64_t)h * p.head_stride + ((int64_t)sp.x + r) * p.row_stride + c * 8;
          a[i] = *reinterpret_cast<const uint4*>(p.out + o);
          b[i] = *reinterpret_cast<const uint4*>(p.dout + o);
        }
      }
#pragma unroll
      for (int i = 0; i < 16 / kPer; ++i) {
        const uint32_t aw[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, bw[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d = fmaf(__uint_as_float(aw[e] << 16), __uint_as_float(bw[e] << 16), d);
          d = fmaf(__uint_as_float(aw[e] & 0xFFFF0000u), __uint_as_float(bw[e] & 0xFFFF0000u), d);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (c == 0) red[0][warp * 16 + i * kPer + sub] = d;
      }
    }
    ptx::named_barrier_sync(1, kSoftThreads);
    // A row past the frame's end gets P = 0 and is never stored.  One of
    // infinite lse gets P = 0 too, and its out may hold anything.
    const float delta = lse == INFINITY ? 0.f : red[0][trow];
    const float nl = -lse * core::kLog2e;
    if (valid && g < 2) {  // group 0: -lse / s, group 1: -delta, as the key pass's MMA takes them
      uint8_t* st = p.stats + ((int64_t)g * p.H * p.N + (int64_t)h * p.N + token) * kStatBytes;
      *reinterpret_cast<uint4*>(st) = split3(g == 0 ? -lse / p.scale : -delta);
    }
    ptx::named_barrier_sync(1, kSoftThreads);  // red is written again
    bool ok = true;
    const uint64_t c2 = ptx::f32x2(p.scale * core::kLog2e, p.scale * core::kLog2e), nl2 = ptx::f32x2(nl, nl);
    const float nd = -delta;
    const uint64_t minus1 = ptx::f32x2(-1.f, -1.f);
    float e0 = 0.f, e1 = 0.f;  // what rounding dS to bf16 added to the row
    constexpr int kCh = kBk<D> / 16 / kSoftGroups;  // chunks of 16 columns per group
    const uint32_t sbase = tmem + lane_base + L::kS + g * kCh * 16, dbase = tmem + lane_base + L::kDp + g * kCh * 16;
    const uint32_t dst = tmem + lane_base + L::kDs + g * kCh * 8;
    for (int j = 0; ok && j < blk.nb; ++j) {
      const int nch = blk.count(j) / 16 - g * kCh;  // this group's chunks that hold keys
      ok = wait(bars.s_full, j);
      if (!ok) break;
      ptx::tc_fence_after_sync();
      uint32_t r[kCh][16];
      core::load_chunks<0, kCh>(sbase, r);
      ptx::tc_fence_before_sync();
      ptx::mbar_arrive(ptx::smem_addr(&bars.s_free));
      float pr[kCh][16];
#pragma unroll
      for (int u = 0; u < kCh; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x0, x1;
          ptx::fma_f32x2(x0, x1, __uint_as_float(r[u][2 * e]), __uint_as_float(r[u][2 * e + 1]), c2, nl2);
          pr[u][2 * e] = ptx::ex2(x0);
          pr[u][2 * e + 1] = ptx::ex2(x1);
        }
      ok = wait(bars.dp_full, j);
      if (!ok) break;
      ptx::tc_fence_after_sync();
      core::load_chunks<0, kCh>(dbase, r);
      ptx::tc_fence_before_sync();
      ptx::mbar_arrive(ptx::smem_addr(&bars.dp_free));
      if (j > 0) {  // dS(j-1) has been read (long ago, as a rule)
        ok = wait(bars.acc_done, j - 1);
        if (!ok) break;
        ptx::tc_fence_after_sync();
      }
      uint32_t pk[kCh][8];
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x0 = __uint_as_float(r[u][2 * e]), x1 = __uint_as_float(r[u][2 * e + 1]);
          ptx::add_f32x2(x0, x1, nd, nd);
          mul_f32x2(pr[u][2 * e], pr[u][2 * e + 1], x0, x1, pr[u][2 * e], pr[u][2 * e + 1]);  // dS
          pk[u][e] = ptx::pack_bf16x2(pr[u][2 * e], pr[u][2 * e + 1]);
        }
        ptx::tmem_st8(dst + u * 8, pk[u]);
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before_sync();
      ptx::mbar_arrive(ptx::smem_addr(&bars.ds_full));
      // Off the tensor pipe's path: what the roundings add up to.  Columns
      // past the range's end hold leftovers and do not count.
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float w0, w1;
          ptx::fma_f32x2(w0, w1, pr[u][2 * e], pr[u][2 * e + 1], minus1,
                         ptx::f32x2(__uint_as_float(pk[u][e] << 16), __uint_as_float(pk[u][e] & 0xFFFF0000u)));
          ptx::add_f32x2(a0, a1, w0, w1);
        }
        e0 += u < nch ? a0 : 0.f;
        e1 += u < nch ? a1 : 0.f;
      }
    }
    red[g][trow] = e0 + e1;
    ok = ok && wait(bars.acc_full, 0);
    ptx::named_barrier_sync(2, kSoftThreads + 32);  // and the mean
    if (ok && !bars.abort) {
      ptx::tc_fence_after_sync();
      float extra = 0.f;
#pragma unroll
      for (int i = 0; i < kSoftGroups; ++i) extra += red[i][trow];
#pragma unroll 1
      for (int c0 = g * 16; c0 < D; c0 += kSoftGroups * 16) {
        uint32_t o[16], w[8];
        ptx::tmem_ld16(tmem + lane_base + L::kAcc + c0, o);
        ptx::tmem_ld_wait(o);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = ptx::pack_bf16x2(fmaf(-extra, centre[c0 + 2 * e], __uint_as_float(o[2 * e])) * p.scale,
                                  fmaf(-extra, centre[c0 + 2 * e + 1], __uint_as_float(o[2 * e + 1])) * p.scale);
        if (valid) {
          uint4* d4 = reinterpret_cast<uint4*>(p.dq + at + c0);
          d4[0] = make_uint4(w[0], w[1], w[2], w[3]);
          d4[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    }
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, kTmemAll);
  }
}

// --------------------------------------------------------------- key pass
//
// Rows are keys, so S and dP are computed transposed: S^T = K.Q^T and dP^T =
// V.dO^T with the tile's K and V as A operands and blocks of Q and dO as B;
// P^T and dS^T then are the A operands of dv += P^T.dO and dk += dS^T.Q, whose
// B operands are the same Q and dO blocks read along their rows.  The two
// accumulators and one S^T and dP^T buffer each fill TMEM; the warpgroups work
// on the same block.  Tensor order: dV(j), S(j+1), dK(j), dP(j+1): P(j+1) is
// computed under dK(j) and dP(j+1), dS(j) under dV(j) and S(j+1).  P is
// released in two parts, so that dV(j) starts on the first.
//
// The softmax statistics differ by column here.  They enter through the MMA:
// one more K step of 16 whose A operand holds ones in three columns and whose
// B operand holds -lse / s (for S^T) or -delta (for dP^T) split into three
// bf16 values a query, so the accumulators come out as S^T - lse / s and dP^T
// - delta.  (Read from shared memory as vectors per column, they took 30% of
// its cycles, which the MMAs' operands need.)
//
// 96 queries: 144 at d = 64, as in the query pass; at d = 128, 64 with both
// tiles in TMEM and 128 with both in shared memory measured within 1%.
template <int D>
constexpr int kBq = D == 64 ? 144 : 96;  // queries per block

template <int D>
struct KLayout {
  // V's A operand is in TMEM; K's too where there is room (d = 64).
  static constexpr bool kKT = D == 64;
  static constexpr uint32_t kDk = 0, kDv = D, kS = 2 * D, kDp = kS + kBq<D>, kV = kDp + kBq<D>, kK = kV + D / 2;
  static_assert(kK + (kKT ? D / 2 : 0) <= kTmemAll, "TMEM columns");
  static constexpr uint32_t kTile = kRowsB * D * 2, kBlock = kBq<D> * D * 2;
  static constexpr uint32_t kStat = 2 * kBq<D> * kStatBytes;  // a stage's statistics
  // Ones for A's rows, then zeros for the rows of A and of B (columns 8 .. 15).
  static constexpr uint32_t kOneRows = kRowsB, kZeroRows = kBq<D> > kRowsB ? kBq<D> : kRowsB;
  static constexpr uint32_t kOnes = (kOneRows + kZeroRows) * 16;
  static constexpr int kFit = (int)((232448 - 1024 - 512 - kOnes - 2 * kTile) / (2 * kBlock + kStat));
  static constexpr int kStages = kFit < kMaxStagesB ? kFit : kMaxStagesB;
  static constexpr size_t kSmem = 1024 + kOnes + 2 * kTile + kStages * (2 * kBlock + kStat);
};

template <int D>
__global__ void __launch_bounds__(kThreadsB, 1)
    attention_bwd_k(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                    const BwdParams p) {
  using L = KLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ BarsB bars;
  const uint32_t k_s = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t v_s = k_s + L::kTile, q_s0 = v_s + L::kTile, do_s0 = q_s0 + L::kStages * L::kBlock;
  const uint32_t stat_s0 = do_s0 + L::kStages * L::kBlock, ones_s = stat_s0 + L::kStages * L::kStat;
  // The ones: rows of {1, 1, 1, 0, 0, 0, 0, 0}, then rows of zeros, which are
  // columns 8 .. 15 of both operands of the statistics' K step.
  for (uint32_t i = threadIdx.x; i < L::kOnes / 16; i += kThreadsB)
    *reinterpret_cast<uint4*>(smem_raw + (ones_s - ptx::smem_addr(smem_raw)) + i * 16) =
        i < L::kOneRows ? make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();
  FAS_BWD_PROLOGUE();
  const Blocks blk(p.table[f], kBq<D>);

  if (warp == kWarpK || warp == kWarpV) {
    if (lane == 0) {
      if (warp == kWarpK) {
        const uint32_t tb = ptx::smem_addr(&bars.tile_full);
        ptx::mbar_arrive_expect_tx(tb, 2 * L::kTile);
        load_rows<D, kRowsB>(k_s, &tm_k, tb, sp.x + tile * kRowsB, h);
        load_rows<D, kRowsB>(v_s, &tm_v, tb, sp.x + tile * kRowsB, h);
        // The statistics, and so everything this CTA writes, come after the
        // query pass.  (The other roles wait for its end too before their
        // first bounded wait that hangs on it.)
        ptx::grid_wait_previous();
        produce<D, kBq<D>, true>(bars, 0, &tm_q, L::kStages, q_s0, h, blk, p, stat_s0);
        if (bars.abort) drain_wait(tb, 0, p.err, p.limit_ns);
      } else {
        produce<D, kBq<D>, false>(bars, 1, &tm_do, L::kStages, do_s0, h, blk, p, 0);
      }
    }
  } else if (warp == kWarpMma) {
    if (ptx::elect_one()) {
      auto wait = [&](uint64_t& b, int parity) {
        return ptx::mbar_wait<false>(ptx::smem_addr(&b), parity & 1, abort_flag, p.err, kErrWaitMma, p.limit_ns);
      };
      const uint64_t kdesc = ptx::smem_desc_sw128(k_s, 16, 1024), vdesc = ptx::smem_desc_sw128(v_s, 16, 1024);
      const uint64_t qd = ptx::smem_desc_sw128(q_s0, 16, 1024), dod = ptx::smem_desc_sw128(do_s0, 16, 1024);
      const uint64_t qmn = ptx::smem_desc_sw128(q_s0, kBq<D> * 128, 1024), domn = ptx::smem_desc_sw128(do_s0, kBq<D> * 128, 1024);
      constexpr uint32_t kZeros = L::kOneRows * 16;
      const uint64_t ones = smem_desc_plain(ones_s, kZeros);
      constexpr uint64_t kStep = L::kBlock >> 4;
      auto stat = [&](int st, int which) {
        const uint32_t at = stat_s0 + st * L::kStat + which * (kBq<D> * kStatBytes);
        return smem_desc_plain(at, ones_s + kZeros - at);
      };
      int qs = 0, qph = 0, ds = 0, dph = 0;  // ring positions of S's Q and dP's dO
      auto s_mma = [&](int n) {
        if (!wait(bars.full[0][qs], qph)) return false;
        ptx::mma_ss(tmem + L::kS, ones, stat(qs, 0), ptx::idesc_bf16_f32(kRowsB, (uint32_t)n, false), 0u);
        mma_rows<D, kBq<D>, L::kKT, true>(tmem + L::kS, tmem + L::kK, kdesc, qd + qs * kStep, n);
        ptx::mma_commit(ptx::smem_addr(&bars.s_full));
        return true;
      };
      auto dp_mma = [&](int n) {  // the same block as the last s_mma
        if (!wait(bars.full[1][ds], dph)) return false;
        ptx::mma_ss(tmem + L::kDp, ones, stat(qs, 1), ptx::idesc_bf16_f32(kRowsB, (uint32_t)n, false), 0u);
        mma_rows<D, kBq<D>, true, true>(tmem + L::kDp, tmem + L::kV, 0, dod + ds * kStep, n);
        ptx::mma_commit(ptx::smem_addr(&bars.dp_full));
        return true;
      };
      auto next = [](int& st, int& ph) {
        if (++st == L::kStages) {
          st = 0;
          ph ^= 1;
        }
      };
      bool ok = wait(bars.tile_full, 0);
      int n = blk.count(0);
      if (ok) {
        tile_to_tmem<D>(tmem + L::kV, vdesc);
        if (L::kKT) tile_to_tmem<D>(tmem + L::kK, kdesc);
        ptx::grid_wait_previous();
        ok = s_mma(n) && dp_mma(n);
      }
      for (int j = 0; ok && j < blk.nb; ++j) {
        const bool more = j + 1 < blk.nb;
        const int n1 = more ? blk.count(j + 1) : 0, st = qs;  // st: block j's stage in both rings
        ok = wait(bars.p_full[0], j);
        if (!ok) break;
        ptx::tc_fence_after_sync();
        mma_acc<D, kBq<D>, 16, 0>(tmem + L::kDv, tmem + L::kS, domn + st * kStep, n, j == 0);
        ok = wait(bars.p_full[1], j);
        if (!ok) break;
        ptx::tc_fence_after_sync();
        mma_acc<D, kBq<D>, 16, 1>(tmem + L::kDv, tmem + L::kS, domn + st * kStep, n, false);
        ptx::mma_commit(ptx::smem_addr(&bars.empty[1][st]));
        next(qs, qph);
        next(ds, dph);
        if (more) ok = s_mma(n1);
        ok = ok && wait(bars.ds_full, j);
        if (!ok) break;
        ptx::tc_fence_after_sync();
        mma_acc<D, kBq<D>, 16, 2>(tmem + L::kDk, tmem + L::kDp, qmn + st * kStep, n, j == 0);
        ptx::mma_commit(ptx::smem_addr(&bars.empty[0][st]));
        if (more) ok = dp_mma(n1);
        n = n1;
      }
      ptx::mma_commit(ptx::smem_addr(&bars.acc_full));
      ptx::mma_commit(ptx::smem_addr(&bars.drain));
      drain_wait(ptx::smem_addr(&bars.drain), 0, p.err, p.limit_ns);
      if (!ok) bars.abort = 1;
    }
    __syncwarp();
  } else if (warp < kWarpK) {
    const int g = warp / 4, trow = (warp % 4) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
    auto wait = [&](uint64_t& b, int parity) {
      const bool got = ptx::mbar_wait<false>(ptx::smem_addr(&b), parity & 1, abort_flag, p.err, kErrWaitSoftmax,
                                             p.limit_ns);
      return (bool)__all_sync(0xffffffffu, got);
    };
    ptx::grid_wait_previous();
    const float c = p.scale * core::kLog2e;
    static_assert(kBq<D> % (16 * kSoftGroups) == 0, "");
    constexpr int kCh = kBq<D> / 16 / kSoftGroups;  // chunks of 16 columns per group
    const uint32_t sbase = tmem + lane_base + L::kS + g * kCh * 16, dbase = tmem + lane_base + L::kDp + g * kCh * 16;
    bool ok = true;
    for (int j = 0; ok && j < blk.nb; ++j) {
      ok = wait(bars.s_full, j);
      if (!ok) break;
      ptx::tc_fence_after_sync();
      uint32_t r[kCh][16];
      core::load_chunks<0, kCh>(sbase, r);
      float pr[kCh][16];
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x0, x1;
          mul_f32x2(x0, x1, __uint_as_float(r[u][2 * e]), __uint_as_float(r[u][2 * e + 1]), c, c);
          pr[u][2 * e] = ptx::ex2(x0);
          pr[u][2 * e + 1] = ptx::ex2(x1);
          pk[e] = ptx::pack_bf16x2(pr[u][2 * e], pr[u][2 * e + 1]);
        }
        ptx::tmem_st8(sbase + u * 16, pk);
        if (u == kFirstChunks<kBq<D>> - 1 || u == kCh - 1) {
          ptx::tmem_st_wait();
          ptx::tc_fence_before_sync();
          ptx::mbar_arrive(ptx::smem_addr(&bars.p_full[u == kCh - 1]));
        }
      }
      ok = wait(bars.dp_full, j);
      if (!ok) break;
      ptx::tc_fence_after_sync();
      core::load_chunks<0, kCh>(dbase, r);
#pragma unroll
      for (int u = 0; u < kCh; ++u) {
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x0, x1;
          mul_f32x2(x0, x1, __uint_as_float(r[u][2 * e]), __uint_as_float(r[u][2 * e + 1]), pr[u][2 * e],
                    pr[u][2 * e + 1]);
          pk[e] = ptx::pack_bf16x2(x0, x1);
        }
        ptx::tmem_st8(dbase + u * 16, pk);
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before_sync();
      ptx::mbar_arrive(ptx::smem_addr(&bars.ds_full));
    }
    ok = ok && wait(bars.acc_full, 0);
    if (ok && !bars.abort) {
      ptx::tc_fence_after_sync();
      const int row = tile * kRowsB + trow;
      const int64_t at = (int64_t)h * p.head_stride + ((int64_t)sp.x + row) * p.row_stride;
#pragma unroll 1
      for (int u = g; u < D / 8; u += kSoftGroups) {  // dk's chunks of 16 columns, then dv's
        const bool k = u < D / 16;
        const int c0 = (k ? u : u - D / 16) * 16;
        store_acc(tmem + lane_base + (k ? L::kDk : L::kDv) + c0, (k ? p.dk : p.dv) + at + c0, k ? p.scale : 1.f,
                  row < sp.y);
      }
    }
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, kTmemAll);
  }
}

#undef FAS_BWD_PROLOGUE

// Tensor map {d, N, H} with boxes of kBox tokens.
int token_map(CUtensorMap* m, const void* base, int d, const BwdParams& p) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)p.N, (cuuint64_t)p.H};
  const cuuint64_t strides[2] = {(cuuint64_t)p.row_stride * 2, (cuuint64_t)p.head_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(d == 64 ? kBox<64> : kBox<128>), 1};
  return bf16_tensor_map(m, base, 3, dims, strides, box);
}

template <int D>
int launch(const BwdParams& p, int grid, cudaStream_t st) {
  using LQ = QLayout<D>;
  using LK = KLayout<D>;
  CUtensorMap tq, tdo, tk, tv;
  if (token_map(&tq, p.q, D, p) != FAS_OK || token_map(&tdo, p.dout, D, p) != FAS_OK ||
      token_map(&tk, p.k, D, p) != FAS_OK || token_map(&tv, p.v, D, p) != FAS_OK)
    return -1;
  auto kq = attention_bwd_q<D>;
  auto kk = attention_bwd_k<D>;
  if (cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LQ::kSmem) != cudaSuccess ||
      cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LK::kSmem) != cudaSuccess)
    return -1;
  kq<<<grid, kThreadsB, LQ::kSmem, st>>>(tq, tdo, tk, tv, p);
  if (cudaGetLastError() != cudaSuccess) return -1;
  // The key pass starts in the query pass's tail and waits there for its
  // statistics.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreadsB);
  cfg.dynamicSmemBytes = LK::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kk, tk, tv, tq, tdo, p) == cudaSuccess ? 2 : -1;
}

}  // namespace

int launch_attention_backward(int d, const BwdParams& p, int grid, cudaStream_t stream) {
  if (d == 128) return launch<128>(p, grid, stream);
  if (d == 64) return launch<64>(p, grid, stream);
  return -1;
}

}  // namespace fas
