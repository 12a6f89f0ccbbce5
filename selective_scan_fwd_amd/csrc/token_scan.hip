// One token of the selective scan on kept states:
//   h <- exp(dt A) h + dt B u;  y = C h + D u;  out = y SiLU(z)
//
// Bound by memory: a state (n fp32 a channel) is read once and written once.  Four
// lanes share a channel, 4 states each, so that a wave's states are one run of
// memory; each of the four forms the channel's step for itself.
#include <hip/hip_runtime.h>

#include "prompt_device.h"

namespace vmk {
namespace {

constexpr int kThreads = 256;
constexpr int kChannels = kThreads / 4;

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

template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void token_scan_kernel(TokenScanArgs a, int wide) {
  const int row = blockIdx.x / wide, ch = (blockIdx.x % wide) * kChannels + threadIdx.x / 4, q = threadIdx.x % 4;
  const bool live = ch < a.dim;
  const int c = live ? ch : 0;                 // (lanes past the channels go along with the first)
  const int64_t slot = a.where != nullptr ? a.where[row] : row;
  float y = 0.0f;
  if (slot >= 0 && slot < a.kept) {
    float *state = a.state + (slot * a.dim + c) * a.n;
    f32x4 h = load_states<VEC>(state, 4 * q, a.n);
    const f32x4 A = load_states<VEC>(a.A + static_cast<int64_t>(c) * a.n, 4 * q, a.n);
    const float u = to_f32(static_cast<const T *>(a.u)[row * a.us + c]);
    float dt = to_f32(static_cast<const T *>(a.delta)[row * a.ds + c]) + (a.bias != nullptr ? a.bias[c] : 0.0f);
    const float z = a.z != nullptr ? to_f32(static_cast<const T *>(a.z)[row * a.zs + c]) : 0.0f;
    const float D = a.D != nullptr ? a.D[c] : 0.0f;
    f32x4 B = {0, 0, 0, 0}, C = B;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * q + i < a.n) {
        B[i] = to_f32(static_cast<const T *>(a.B)[row * a.bs + 4 * q + i]);
        C[i] = to_f32(static_cast<const T *>(a.C)[row * a.cs + 4 * q + i]);
      }
    if (a.softplus) dt = softplus_f(dt);
    const float du = dt * u;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = __builtin_fmaf(hw_exp2(dt * rate2(A[i])), h[i], du * B[i]);
      sum = __builtin_fmaf(C[i], h[i], sum);
    }
    if (live) {
      if (VEC) {
        if (4 * q < a.n) *reinterpret_cast<f32x4 *>(state + 4 * q) = h;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * q + i < a.n) state[4 * q + i] = h[i];
      }
    }
    y = __builtin_fmaf(D, u, sum4(sum));
    if (a.z != nullptr) y *= silu_f(z);
  }
  if (live && q == 0) static_cast<T *>(a.out)[static_cast<int64_t>(row) * a.dim + c] = from_f32<T>(y);
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
