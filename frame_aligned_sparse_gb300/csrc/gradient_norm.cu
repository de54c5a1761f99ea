// The norm of all gradients together, and clipping by it:
//   norm = sqrt(sum over all tensors of g^2),  g' = g min(1, max_norm / (norm + eps)).
//
// Two kernels.  The first adds squares: fp32 within a thread's share of a
// piece of 8192 elements (32 or fewer terms a sum), 64 bits from there on,
// in an order that the sizes fix, so the norm is bit-reproducible.  Where a
// thread's fp32 sum overflowed or came out so small that squares may have
// been lost below fp32's range, the thread reads its share again and adds it
// in 64 bits (not for a share of zeros: gradients of rows that no token took
// are ordinary, and 300 M of them in 16 bits took 1.13 ms so, 0.09 now).  The
// second kernel adds the first one's sums (every CTA for itself: a few KB from
// L2, and nothing waits on another CTA) and scales, by a factor in fp32 where
// that holds it with all its bits and in 64 bits where the norm is so large
// that it does not.  It goes through the pieces backwards, so that what the
// first kernel read last is still in L2.  Tensor addresses travel in the
// launch's parameters: nothing is copied to the device, and a captured graph
// holds them.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

#include "kernels.h"
#include "ptx.cuh"

namespace fas {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 8192;  // elements of a tensor that a CTA takes at a time

template <int kMost>
struct Table {
  const void* in[kMost];
  void* out[kMost];
  int64_t n[kMost];
  int64_t first[kMost];  // pieces before the tensor
  uint8_t f32[kMost];
  int tensors;
  int64_t pieces, keep_from;  // pieces from keep_from on: the last kKeepBytes
};
constexpr int64_t kKeepBytes = 96 << 20;  // of L2's 129 MB

// What is added below may have lost squares under fp32's smallest, or passed its largest.
constexpr float kSafe = 0x1p-90f;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int kMost>
__device__ __forceinline__ int tensor_of(const Table<kMost>& t, int64_t piece) {
  int lo = 0, hi = t.tensors - 1;  // the last tensor with first <= piece (empty ones share the next one's first)
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= piece) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <bool kF32>
__device__ __forceinline__ float element(const void* base, int64_t i) {
  if constexpr (kF32) return static_cast<const float*>(base)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[i] << 16);
}

// A piece's elements: `head` up to the first 16-byte boundary, whole vectors, and the rest.
template <bool kF32>
struct Span {
  static constexpr int kVec = kF32 ? 4 : 8;
  int64_t from;
  int head, vecs, count;
  __device__ __forceinline__ Span(const void* base, int64_t from_, int64_t n) : from(from_) {
    count = (int)min((int64_t)kPiece, n - from);
    const uintptr_t at = reinterpret_cast<uintptr_t>(base) + (uintptr_t)from * (kF32 ? 4 : 2);
    head = min(count, (int)(((16 - (at & 15)) & 15) / (kF32 ? 4 : 2)));
    vecs = (count - head) / kVec;
  }
  __device__ __forceinline__ int loose() const { return count - vecs * kVec; }
  __device__ __forceinline__ int64_t loose_at(int i) const { return from + (i < head ? i : i + vecs * kVec); }
  __device__ __forceinline__ int64_t vec_at(int v) const { return from + head + (int64_t)v * kVec; }
};

__device__ __forceinline__ uint4 load_hint(const void* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}

template <bool kF32>
__device__ __forceinline__ double piece_squares(const void* base, int64_t from, int64_t n, uint64_t policy) {
  const Span<kF32> sp(base, from, n);
  constexpr int kVec = Span<kF32>::kVec;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t bits = 0;  // of all values
  auto add = [&](uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bits |= w[e];
      if constexpr (kF32) {
        s[e] = fmaf(__uint_as_float(w[e]), __uint_as_float(w[e]), s[e]);
      } else {
        s[e] = fmaf(bf16_lo(w[e]), bf16_lo(w[e]), s[e]);
        s[e] = fmaf(bf16_hi(w[e]), bf16_hi(w[e]), s[e]);
      }
    }
  };
  auto at = [&](int v) {
    return load_hint(static_cast<const uint8_t*>(base) + sp.vec_at(v) * (kF32 ? 4 : 2), policy);
  };
  constexpr int kSteps = kPiece / kVec / kThreads;
  if (sp.vecs == kSteps * kThreads) {
    uint4 v[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) v[k] = at(threadIdx.x + k * kThreads);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) add(v[k]);
  } else {
    for (int v = threadIdx.x; v < sp.vecs; v += kThreads) add(at(v));
  }
  for (int i = threadIdx.x; i < sp.loose(); i += kThreads) {
    const float x = element<kF32>(base, sp.loose_at(i));
    s[0] = fmaf(x, x, s[0]);
    bits |= __float_as_uint(x);
  }
  const float all = (s[0] + s[1]) + (s[2] + s[3]);
  if (all >= kSafe && all < INFINITY) return (double)all;
  if ((bits & (kF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0) return 0.0;
  double d = 0.0;
  auto add64 = [&](float x) {
    if (x != 0.f) d = fma((double)x, (double)x, d);
  };
  for (int v = threadIdx.x; v < sp.vecs; v += kThreads) {
    const uint4 x = at(v);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (kF32) {
        add64(__uint_as_float(w[e]));
      } else {
        add64(bf16_lo(w[e]));
        add64(bf16_hi(w[e]));
      }
    }
  }
  for (int i = threadIdx.x; i < sp.loose(); i += kThreads) add64(element<kF32>(base, sp.loose_at(i)));
  return d;
}

// The sum over the CTA's threads, in thread 0.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
  __syncthreads();
  double sum = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreads / 32; ++w) sum += part[w];
  return sum;
}

template <int kMost>
__global__ void __launch_bounds__(kThreads) gradient_squares(const __grid_constant__ Table<kMost> t, double* partial) {
  double sum = 0.0;
  // What gradient_scale reads first stays in L2, the rest goes through.
  const uint64_t keep = ptx::policy_evict_last(), pass = ptx::policy_evict_first();
  for (int64_t p = blockIdx.x; p < t.pieces; p += gridDim.x) {
    const int i = tensor_of(t, p);
    const int64_t from = (p - t.first[i]) * kPiece;
    const uint64_t policy = p >= t.keep_from ? keep : pass;
    sum += t.f32[i] ? piece_squares<true>(t.in[i], from, t.n[i], policy) : piece_squares<false>(t.in[i], from, t.n[i], policy);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// sqrt of the partial sums' total, in thread 0.
__device__ __forceinline__ double norm_of(const double* partial, int count) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) sum += partial[i];
  return sqrt(block_sum(sum));
}

__global__ void __launch_bounds__(kThreads) gradient_total(const double* partial, int count, float* norm) {
  ptx::grid_wait_previous();
  const double total = norm_of(partial, count);
  if (threadIdx.x == 0) *norm = (float)total;
}

// F: float, or double for factors below fp32's normal numbers.
template <bool kF32, class F>
__device__ __forceinline__ void piece_scale(const void* in, void* out, int64_t from, int64_t n, F f, uint64_t policy) {
  constexpr int kElem = kF32 ? 4 : 2;
  const Span<kF32> sp(in, from, n);
  const uint8_t* src = static_cast<const uint8_t*>(in);
  uint8_t* dst = static_cast<uint8_t*>(out);
  auto one = [&](int64_t i) {
    const float x = (float)(element<kF32>(in, i) * f);
    if constexpr (kF32) static_cast<float*>(out)[i] = x;
    else static_cast<uint16_t*>(out)[i] = (uint16_t)ptx::pack_bf16x2(x, 0.f);
  };
  auto scaled = [&](uint4 v) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = kF32 ? __float_as_uint((float)(__uint_as_float(w[e]) * f))
                  : ptx::pack_bf16x2((float)(bf16_lo(w[e]) * f), (float)(bf16_hi(w[e]) * f));
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
    for (int i = threadIdx.x; i < sp.count; i += kThreads) one(sp.from + i);
    return;
  }
  constexpr int kSteps = kPiece / Span<kF32>::kVec / kThreads;
  if (sp.vecs == kSteps * kThreads) {
    uint4 v[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
      v[k] = load_hint(src + sp.vec_at(threadIdx.x + k * kThreads) * kElem, policy);
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
      ptx::st_global_hint(dst + sp.vec_at(threadIdx.x + k * kThreads) * kElem, scaled(v[k]), policy);
  } else {
    for (int v = threadIdx.x; v < sp.vecs; v += kThreads)
      ptx::st_global_hint(dst + sp.vec_at(v) * kElem, scaled(load_hint(src + sp.vec_at(v) * kElem, policy)), policy);
  }
  for (int i = threadIdx.x; i < sp.loose(); i += kThreads) one(sp.loose_at(i));
}

template <int kMost>
__global__ void __launch_bounds__(kThreads)
    gradient_scale(const __grid_constant__ Table<kMost> t, const double* partial, int count, float max_norm, float eps,
                   float* norm) {
  __shared__ double factor;
  ptx::grid_wait_previous();
  const double total = norm_of(partial, count);
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0 && norm) *norm = (float)total;
    const double limit = total + (double)eps;
    factor = limit <= (double)max_norm ? 1.0 : (double)max_norm / limit;  // NaN stays NaN
  }
  __syncthreads();
  const float f = (float)factor;
  const bool small = factor > 0.0 && factor < 0x1p-126;
  const uint64_t pass = ptx::policy_evict_first();
  for (int64_t q = blockIdx.x; q < t.pieces; q += gridDim.x) {
    const int64_t p = t.pieces - 1 - q;
    const int i = tensor_of(t, p);
    if (f == 1.f && t.in[i] == t.out[i]) continue;
    const int64_t from = (p - t.first[i]) * kPiece;
    if (small) {
      if (t.f32[i]) piece_scale<true>(t.in[i], t.out[i], from, t.n[i], factor, pass);
      else piece_scale<false>(t.in[i], t.out[i], from, t.n[i], factor, pass);
    } else {
      if (t.f32[i]) piece_scale<true>(t.in[i], t.out[i], from, t.n[i], f, pass);
      else piece_scale<false>(t.in[i], t.out[i], from, t.n[i], f, pass);
    }
  }
}

template <int kMost>
void fill(Table<kMost>& t, const GradientList& g, int from, int count) {
  t.tensors = count;
  t.pieces = 0;
  for (int i = 0; i < count; ++i) {
    t.in[i] = g.in[from + i];
    t.out[i] = g.out ? g.out[from + i] : nullptr;
    t.n[i] = g.elements[from + i];
    t.first[i] = t.pieces;
    t.f32[i] = (uint8_t)(g.dtypes[from + i] != 0);
    t.pieces += (t.n[i] + kPiece - 1) / kPiece;
  }
  t.keep_from = t.pieces;
  int64_t room = g.out ? kKeepBytes : 0;
  for (int i = count - 1; i >= 0 && room > 0; --i) {
    const int64_t piece = kPiece * (t.f32[i] ? 4 : 2), pieces = t.keep_from - t.first[i];
    const int64_t kept = std::min(pieces, room / piece);
    t.keep_from -= kept;
    room = kept < pieces ? 0 : room - kept * piece;
  }
}

// CTAs an SM.  More of the reading kernel's are better up to six (354 M
// gradients: 112 us; three 129, eight 117); reading and writing at once, few
// at a time keep closer together in memory (three 213 us, six 222).
constexpr int kReading = 6, kScaling = 3;
int grid_for(int64_t pieces, int sms, int per_sm) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(pieces, std::min(sms * per_sm, kGradientSlots)));
}

// Starts while the kernel before it ends, and waits for its results.
template <class... Params, class... Args>
cudaError_t start_after(void (*kern)(Params...), int grid, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, Params(args)...);
}

template <int kMost>
cudaError_t run(const GradientList& g, float* norm, const float* clip, double* partial, int sms, int* launches,
                cudaStream_t st) {
  const std::unique_ptr<Table<kMost>> t(new (std::nothrow) Table<kMost>);
  if (!t) return cudaErrorMemoryAllocation;
  int slots = 0;
  *launches = 0;
  for (int from = 0; from == 0 || from < g.n; from += kMost) {
    fill(*t, g, from, std::min(kMost, g.n - from));
    const int grid = grid_for(t->pieces, sms, kReading);
    gradient_squares<kMost><<<grid, kThreads, 0, st>>>(*t, partial + slots);
    slots += grid;
    ++*launches;
  }
  if (!clip) {
    const cudaError_t e = start_after(gradient_total, 1, st, partial, slots, norm);
    if (e != cudaSuccess) return e;
    ++*launches;
  } else {
    for (int from = 0; from == 0 || from < g.n; from += kMost) {
      if (g.n > kMost) fill(*t, g, from, std::min(kMost, g.n - from));
      const cudaError_t e = start_after(gradient_scale<kMost>, grid_for(t->pieces, sms, kScaling), st, *t, partial, slots, clip[0], clip[1],
                                        from == 0 ? norm : nullptr);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gradient_norm(const GradientList& g, float* norm, const float* clip, double* partial, int sms,
                                 int* launches, cudaStream_t stream) {
  if (g.n <= kGradientsFew) return run<kGradientsFew>(g, norm, clip, partial, sms, launches, stream);
  return run<kGradientsMost>(g, norm, clip, partial, sms, launches, stream);
}

}  // namespace fas
