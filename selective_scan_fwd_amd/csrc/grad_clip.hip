// The Euclidean norm over many tensors and their scaling to a largest norm.
//
//   norm = sqrt(sum over all tensors of x^2),  y = x min(1, max_norm / (norm + 1e-6))
//
// Two passes over the gradients, bound by memory: the first sums squares, the
// second scales.  A pass handles up to 120 tensors in one launch: the table of
// pointers and sizes travels in the kernel's arguments (3.6 KB), so nothing is
// copied to the device first.  Tensors are cut into chunks of 2048 elements and
// a block takes runs of up to 8 of them, as many runs as all others, so small
// and large tensors load the card alike and no block is left with a last round
// of its own (310 MB of bf16: sums 55 us; with chunks of 16384 dealt out one by
// one 85 us).  Longer lists take a launch for every 120, each over the whole card,
// block b adding to partial sum b, so there are no more of them than of one
// launch's (6000 tensors of 4 MB: sums 1.3 ms; with the partial sums divided
// over the launches, 20 blocks each, 20.8).  The second pass goes back from the
// last run, which is nearest still, to the first: 97 us, forwards 105 us.  Its
// loads and stores are past their last use here and marked so; without that the
// next pass over other memory waits for the written lines to leave the cache
// (sums 85 us).
#include <hip/hip_runtime.h>

#include "mixer_internal.h"
#include "vm_internal.h"

namespace vmk {
namespace {

constexpr int kThreads = 512;
constexpr int kAhead = 4;    // loads of 16 bytes that a thread has in flight
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The tensor of chunk c: the last one whose first chunk is <= c.
__device__ __forceinline__ int tensor_of(const ClipTable &t, uint32_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double x, double *red) {
  for (int o = 32; o > 0; o >>= 1) x += __shfl_down(x, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0;
  for (int w = 0; w < kThreads / 64; ++w) x += red[w];
  __syncthreads();
  return x;
}

__device__ __forceinline__ bool aligned16(const void *p) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// Squares are exact in fp64 and their sums carry 53 bits, so no gradient
// overflows the norm and the order of the sums costs nothing in fp32.
template <typename T>
__device__ __forceinline__ double run_squares(const T *x, int64_t n) {
  constexpr int kVec = 16 / sizeof(T);
  double a = 0, b = 0;
  int64_t done = 0;
  if (aligned16(x)) {
    const int64_t vecs = n / kVec;
    const u32x4 *from = reinterpret_cast<const u32x4 *>(x);
    const auto add = [&](u32x4 raw) {
      const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        const double p = to_f32(e[j]), q = to_f32(e[j + 1]);
        a = __builtin_fma(p, p, a);
        b = __builtin_fma(q, q, b);
      }
    };
    int64_t i = threadIdx.x;
    for (; i + (kAhead - 1) * kThreads < vecs; i += kAhead * kThreads) {
      u32x4 raw[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) raw[j] = from[i + j * kThreads];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) add(raw[j]);
    }
    for (; i < vecs; i += kThreads) add(from[i]);
    done = vecs * kVec;
  }
  for (int64_t i = done + threadIdx.x; i < n; i += kThreads) {
    const double p = to_f32(x[i]);
    a = __builtin_fma(p, p, a);
  }
  return a + b;
}

template <typename T>
__device__ __forceinline__ void run_scale(const T *x, T *y, int64_t n, float f) {
  constexpr int kVec = 16 / sizeof(T);
  int64_t done = 0;
  if (aligned16(x) && aligned16(y)) {
    const int64_t vecs = n / kVec;
    const u32x4 *from = reinterpret_cast<const u32x4 *>(x) + (vecs - 1);
    u32x4 *to = reinterpret_cast<u32x4 *>(y) + (vecs - 1);
    const auto scaled = [f](u32x4 raw) {
      T *e = reinterpret_cast<T *>(&raw);
#pragma unroll
      for (int j = 0; j < kVec; ++j) e[j] = from_f32<T>(to_f32(e[j]) * f);
      return raw;
    };
    int64_t i = threadIdx.x;
    for (; i + (kAhead - 1) * kThreads < vecs; i += kAhead * kThreads) {
      u32x4 raw[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) raw[j] = __builtin_nontemporal_load(from - (i + j * kThreads));
#pragma unroll
      for (int j = 0; j < kAhead; ++j) __builtin_nontemporal_store(scaled(raw[j]), to - (i + j * kThreads));
    }
    for (; i < vecs; i += kThreads) __builtin_nontemporal_store(scaled(from[-i]), to - i);
    done = vecs * kVec;
  }
  for (int64_t i = done + threadIdx.x; i < n; i += kThreads) y[i] = from_f32<T>(to_f32(x[i]) * f);
}

// The elements [at, at + n) of tensor i that chunks [from, to) of its own hold.
struct Run {
  int64_t at, n;
};
__device__ __forceinline__ Run run_of(const ClipTable &t, int i, uint32_t from, uint32_t to) {
  const int64_t at = static_cast<int64_t>(from - t.first[i]) * kClipChunk;
  const int64_t end = static_cast<int64_t>(to - t.first[i]) * kClipChunk;
  return Run{at, (end < t.elems[i] ? end : t.elems[i]) - at};
}
// Block b takes runs b, b + grid, ... of `len` chunks.
struct Runs {
  uint32_t chunks, len, rounds;
};
__device__ __forceinline__ Runs runs_of(const ClipTable &t) {
  Runs r;
  r.chunks = t.first[t.n];
  r.rounds = (r.chunks + gridDim.x * kClipRun - 1) / (gridDim.x * kClipRun);
  r.len = (r.chunks + gridDim.x * r.rounds - 1) / (gridDim.x * r.rounds);
  return r;
}

__global__ __launch_bounds__(kThreads) void clip_sums_kernel(ClipTable t, double *partial, int have) {
  __shared__ double red[kThreads / 64];
  const Runs all = runs_of(t);
  double sum = 0;
  for (uint32_t y = 0; y < all.rounds; ++y) {
    uint32_t c = (y * gridDim.x + blockIdx.x) * all.len;
    const uint32_t end = c + all.len < all.chunks ? c + all.len : all.chunks;
    for (int i = c < end ? tensor_of(t, c) : 0; c < end; ++i) {
      const uint32_t to = t.first[i + 1] < end ? t.first[i + 1] : end;
      const Run r = run_of(t, i, c, to);
      sum += t.bf16[i] ? run_squares(static_cast<const bf16_t *>(t.in[i]) + r.at, r.n)
                       : run_squares(static_cast<const float *>(t.in[i]) + r.at, r.n);
      c = to;
    }
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = static_cast<int>(blockIdx.x) < have ? partial[blockIdx.x] + sum : sum;
}

// Every block adds the partial sums itself (at most a few KB from the caches,
// in the same order everywhere), which saves a launch between the passes.
__device__ __forceinline__ float total_norm(const double *partial, int partials, double *red) {
  double sum = 0;
  for (int i = threadIdx.x; i < partials; i += kThreads) sum += partial[i];
  return static_cast<float>(sqrt(block_sum(sum, red)));
}

__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipTable t, const double *partial,
                                                              int partials, float max_norm, float *norm) {
  __shared__ double red[kThreads / 64];
  const float total = total_norm(partial, partials, red);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  float f = max_norm / (total + 1e-6f);
  f = f > 1.0f ? 1.0f : f;              // (NaN stays NaN)
  const Runs all = runs_of(t);
  for (uint32_t y = all.rounds; y-- > 0;) {
    const uint32_t begin = (y * gridDim.x + blockIdx.x) * all.len;
    uint32_t c = begin + all.len < all.chunks ? begin + all.len : all.chunks;
    for (int i = begin < c ? tensor_of(t, c - 1) : 0; begin < c; --i) {
      const uint32_t from = t.first[i] > begin ? t.first[i] : begin;
      const Run r = run_of(t, i, from, c);
      c = from;
      if (t.out[i] == nullptr || (f == 1.0f && t.out[i] == t.in[i])) continue;
      if (t.bf16[i])
        run_scale(static_cast<const bf16_t *>(t.in[i]) + r.at, static_cast<bf16_t *>(t.out[i]) + r.at, r.n, f);
      else
        run_scale(static_cast<const float *>(t.in[i]) + r.at, static_cast<float *>(t.out[i]) + r.at, r.n, f);
    }
  }
}

__global__ __launch_bounds__(kThreads) void clip_norm_kernel(const double *partial, int partials,
                                                             float *norm) {
  __shared__ double red[kThreads / 64];
  const float total = total_norm(partial, partials, red);
  if (threadIdx.x == 0) *norm = total;
}

}  // namespace

hipError_t launch_clip_sums(const ClipTable &t, double *partial, int have, int blocks, hipStream_t s) {
  hipLaunchKernelGGL(clip_sums_kernel, dim3(blocks), dim3(kThreads), 0, s, t, partial, have);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipTable &t, const double *partial, int partials, float max_norm,
                             float *norm, int blocks, hipStream_t s) {
  hipLaunchKernelGGL(clip_scale_kernel, dim3(blocks), dim3(kThreads), 0, s, t, partial, partials, max_norm,
                     norm);
  return hipGetLastError();
}

hipError_t launch_clip_norm_only(const double *partial, int partials, float *norm, hipStream_t s) {
  hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(kThreads), 0, s, partial, partials, norm);
  return hipGetLastError();
}

}  // namespace vmk
