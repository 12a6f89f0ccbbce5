// One token of the selective scan on kept states:
//   h <- exp(dt A) h + dt B u;  y = C h + D u;  out = y SiLU(z)
//
// Bound by memory: a state (n fp32 a channel) is read once and written once.  Four
// lanes share a channel, 4 states each, so that a wave's states are one run of
// memory; each of the four forms the channel's step for itself.  128 sequences of 4096
// channels with 16 states (64 MB): 15 us, 4.3 TB/s.
#include <hip/hip_runtime.h>

#include "prompt_device.h"

namespace vmk {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 2;                 // channels to each four lanes
constexpr int kChannels = kThreads / 4 * kEach;

// Sum over each four neighbouring lanes.
__device__ __forceinline__ float sum4(float x) {
  x += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0xb1, 0xf, 0xf, true));     // lane ^ 1
  return x + __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x4e, 0xf, 0xf, true));   // lane ^ 2
}

// VEC: n is a multiple of 4 and states and A are whole pieces of 16 bytes.
template <bool VEC>
__device__ __forceinline__ f32x4 load_states(const float *p, int first, int n) {
  f32x4 x = {0, 0, 0, 0};
  if (VEC) {
    if (first < n) x = *reinterpret_cast<const f32x4 *>(p + first);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (first + i < n) x[i] = p[first + i];
  }
  return x;
}

// Two channels to each four lanes, every load under way before the first use: an idle
// row reads the first state and stores none.
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void token_scan_kernel(TokenScanArgs a, int wide) {
  const int row = blockIdx.x / wide, q = threadIdx.x % 4;
  const int64_t slot = a.where != nullptr ? a.where[row] : row;
  const bool idle = slot < 0 || slot >= a.kept;
  f32x4 B = {0, 0, 0, 0}, C = B, h[kEach], A[kEach];
  float u[kEach], d[kEach], z[kEach], D[kEach];
  float *state[kEach];
  int c[kEach];
  bool live[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int ch = (blockIdx.x % wide) * kChannels + k * (kThreads / 4) + threadIdx.x / 4;
    live[k] = ch < a.dim;
    c[k] = live[k] ? ch : 0;                   // (lanes past the channels go along with the first)
    A[k] = load_states<VEC>(a.A + static_cast<int64_t>(c[k]) * a.n, 4 * q, a.n);
    u[k] = to_f32(static_cast<const T *>(a.u)[row * a.us + c[k]]);
    d[k] = to_f32(static_cast<const T *>(a.delta)[row * a.ds + c[k]]) + (a.bias != nullptr ? a.bias[c[k]] : 0.0f);
    z[k] = a.z != nullptr ? to_f32(static_cast<const T *>(a.z)[row * a.zs + c[k]]) : 0.0f;
    D[k] = a.D != nullptr ? a.D[c[k]] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * q + i < a.n) {
      B[i] = to_f32(static_cast<const T *>(a.B)[row * a.bs + 4 * q + i]);
      C[i] = to_f32(static_cast<const T *>(a.C)[row * a.cs + 4 * q + i]);
    }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    state[k] = a.state + ((idle ? 0 : slot) * a.dim + c[k]) * a.n;
    h[k] = load_states<VEC>(state[k], 4 * q, a.n);
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const float dt = a.softplus ? softplus_f(d[k]) : d[k], du = dt * u[k];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[k][i] = __builtin_fmaf(hw_exp2(dt * rate2(A[k][i])), h[k][i], du * B[i]);
      // (a place without a state has 0 times an infinite dt or dt u, which is no number)
      sum = 4 * q + i < a.n ? __builtin_fmaf(C[i], h[k][i], sum) : sum;
    }
    if (live[k] && !idle) {
      if (VEC) {
        if (4 * q < a.n) *reinterpret_cast<f32x4 *>(state[k] + 4 * q) = h[k];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * q + i < a.n) state[k][4 * q + i] = h[k][i];
      }
    }
    float y = __builtin_fmaf(D[k], u[k], sum4(sum));
    if (a.z != nullptr) y *= silu_f(z[k]);
    if (live[k] && q == 0) static_cast<T *>(a.out)[static_cast<int64_t>(row) * a.dim + c[k]] = from_f32<T>(idle ? 0.0f : y);
  }
}

}  // namespace

hipError_t launch_token_scan(const TokenScanArgs &a, bool bf16, hipStream_t s) {
  const int wide = (a.dim + kChannels - 1) / kChannels;
  const uint32_t grid = static_cast<uint32_t>(static_cast<int64_t>(wide) * a.batch);
  const bool vec = a.n % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0 && (reinterpret_cast<uintptr_t>(a.A) & 15) == 0;
  if (bf16) {
    if (vec)
      token_scan_kernel<bf16_t, true><<<grid, kThreads, 0, s>>>(a, wide);
    else
      token_scan_kernel<bf16_t, false><<<grid, kThreads, 0, s>>>(a, wide);
  } else {
    if (vec)
      token_scan_kernel<float, true><<<grid, kThreads, 0, s>>>(a, wide);
    else
      token_scan_kernel<float, false><<<grid, kThreads, 0, s>>>(a, wide);
  }
  return hipGetLastError();
}

}  // namespace vmk
