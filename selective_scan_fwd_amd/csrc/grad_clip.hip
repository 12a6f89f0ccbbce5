// The Euclidean norm over many tensors and their scaling to a largest norm.
//
//   norm = sqrt(sum over all tensors of x^2),  y = x min(1, max_norm / (norm + 1e-6))
//
// Two passes over the gradients, bound by memory: the first sums squares, the
// second scales.  A pass handles up to 120 tensors in one launch: the table of
// pointers and sizes travels in the kernel's arguments (3.6 KB), so nothing is
// copied to the device first.  Tensors are cut into chunks of 16384 elements
// and a block takes every grid-th chunk, so small and large tensors load the
// card alike.
#include <hip/hip_runtime.h>

#include "mixer_internal.h"
#include "vm_internal.h"

namespace vmk {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;    // loads of 16 bytes that a thread has in flight
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
__device__ __forceinline__ double chunk_squares(const T *x, int n) {
  constexpr int kVec = 16 / sizeof(T);
  double a = 0, b = 0;
  int done = 0;
  if (aligned16(x)) {
    const int vecs = n / kVec;
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
    int i = threadIdx.x;
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
  for (int i = done + threadIdx.x; i < n; i += kThreads) {
    const double p = to_f32(x[i]);
    a = __builtin_fma(p, p, a);
  }
  return a + b;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *x, T *y, int n, float f) {
  constexpr int kVec = 16 / sizeof(T);
  int done = 0;
  if (aligned16(x) && aligned16(y)) {
    const int vecs = n / kVec;
    const u32x4 *from = reinterpret_cast<const u32x4 *>(x);
    u32x4 *to = reinterpret_cast<u32x4 *>(y);
    const auto scaled = [f](u32x4 raw) {
      T *e = reinterpret_cast<T *>(&raw);
#pragma unroll
      for (int j = 0; j < kVec; ++j) e[j] = from_f32<T>(to_f32(e[j]) * f);
      return raw;
    };
    int i = threadIdx.x;
    for (; i + (kAhead - 1) * kThreads < vecs; i += kAhead * kThreads) {
      u32x4 raw[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) raw[j] = from[i + j * kThreads];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) to[i + j * kThreads] = scaled(raw[j]);
    }
    for (; i < vecs; i += kThreads) to[i] = scaled(from[i]);
    done = vecs * kVec;
  }
  for (int i = done + threadIdx.x; i < n; i += kThreads) y[i] = from_f32<T>(to_f32(x[i]) * f);
}

__device__ __forceinline__ int chunk_len(int64_t elems, int64_t at) {
  const int64_t left = elems - at;
  return static_cast<int>(left < kClipChunk ? left : kClipChunk);
}

__global__ __launch_bounds__(kThreads) void clip_sums_kernel(ClipTable t, double *partial) {
  __shared__ double red[kThreads / 64];
  const uint32_t chunks = t.first[t.n];
  double sum = 0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = static_cast<int64_t>(c - t.first[i]) * kClipChunk;
    const int n = chunk_len(t.elems[i], at);
    sum += t.bf16[i] ? chunk_squares(static_cast<const bf16_t *>(t.in[i]) + at, n)
                     : chunk_squares(static_cast<const float *>(t.in[i]) + at, n);
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
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
  const uint32_t chunks = t.first[t.n];
  for (uint32_t b = blockIdx.x; b < chunks; b += gridDim.x) {
    const uint32_t c = chunks - 1 - b;  // what the sums read last is nearest still
    const int i = tensor_of(t, c);
    if (t.out[i] == nullptr || (f == 1.0f && t.out[i] == t.in[i])) continue;
    const int64_t at = static_cast<int64_t>(c - t.first[i]) * kClipChunk;
    const int n = chunk_len(t.elems[i], at);
    if (t.bf16[i])
      chunk_scale(static_cast<const bf16_t *>(t.in[i]) + at, static_cast<bf16_t *>(t.out[i]) + at, n, f);
    else
      chunk_scale(static_cast<const float *>(t.in[i]) + at, static_cast<float *>(t.out[i]) + at, n, f);
  }
}

__global__ __launch_bounds__(kThreads) void clip_norm_kernel(const double *partial, int partials,
                                                             float *norm) {
  __shared__ double red[kThreads / 64];
  const float total = total_norm(partial, partials, red);
  if (threadIdx.x == 0) *norm = total;
}

}  // namespace

hipError_t launch_clip_sums(const ClipTable &t, double *partial, int blocks, hipStream_t s) {
  hipLaunchKernelGGL(clip_sums_kernel, dim3(blocks), dim3(kThreads), 0, s, t, partial);
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
