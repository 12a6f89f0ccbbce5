// One token of the gated delta rule on stored states:
//   S' = exp(g) S,  e = beta (v - S'^T k),  S <- S' + k e^T,
//   out = scale S^T q = scale (S'^T q + (q.k) e)
//
// Bound by memory: each state (dk dv fp32) is read once and written once.  A
// wave takes 32 columns of one head: 8 lanes hold 4 columns each of 8 groups of
// rows, all loads are issued before the first use, and the one reduction over
// the row groups carries both products, since out follows from S' alone.
// 128 sequences of 32 heads, 128 x 128 (480 MB): 102 us, 4.7 TB/s, where a copy
// of 4 GB runs at 4.9.  One sequence of 16 heads: 4.5 us, in a call of 10.
#include <hip/hip_runtime.h>

#include "delta_device.h"

namespace vmk {
namespace {

constexpr int kCols = 32;

template <typename T, int DK, bool VEC>
__global__ __launch_bounds__(64) void delta_step_kernel(StepArgs A) {
  constexpr int kRows = DK / 8;           // rows of one lane: rg, rg + 8, ...
  __shared__ float sk[DK], sq[DK];
  const int lane = threadIdx.x, rg = lane / 8;
  const int colblocks = (A.dv + kCols - 1) / kCols;
  const int cb = blockIdx.x % colblocks;
  const int64_t bh = blockIdx.x / colblocks;
  const int b = static_cast<int>(bh / A.hv), h = static_cast<int>(bh % A.hv), kh = h / (A.hv / A.hk);
  const int col = cb * kCols + (lane % 8) * 4;
  const int64_t slot = uniform(A.slots != nullptr ? A.slots[b] : b);
  const Rsrc out = buffer(static_cast<T *>(A.out) + bh * A.dv, A.dv * sizeof(T));
  const auto store_out = [&](f32x4 y) {
    if (rg == 0)
#pragma unroll
      for (int e = 0; e < 4; ++e) bstore(out, (col + e) * sizeof(T), from_f32<T>(y[e]));
  };
  if (slot < 0 || slot >= A.n_slots) {
    store_out(f32x4{0, 0, 0, 0});
    return;
  }
  // rows past dk lie past the resource's end, columns past dv go nowhere
  const Rsrc S = buffer(A.state + (slot * A.hv + h) * A.dk * A.dv, A.dk * A.dv * 4);
  uint32_t at[4];                           // of row rg, this lane's columns
#pragma unroll
  for (int e = 0; e < 4; ++e) at[e] = col + e < A.dv ? (rg * A.dv + col + e) * 4 : kNowhere;
  const uint32_t step = 8 * A.dv * 4;
  f32x4 x[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (VEC)
      x[i] = __builtin_bit_cast(f32x4, bload16(S, at[0] + i * step));
    else
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = bload<float>(S, at[e] + i * step);
  }
  const int64_t key = (static_cast<int64_t>(b) * A.hk + kh) * A.dk;
  for (int i = lane; i < DK; i += 64) {
    sk[i] = i < A.dk ? to_f32(static_cast<const T *>(A.k)[key + i]) : 0.0f;
    sq[i] = i < A.dk ? to_f32(static_cast<const T *>(A.q)[key + i]) : 0.0f;
  }
  const float a = hw_exp2(A.g[bh] * kLog2e), beta = A.beta[bh];
  const Rsrc values = buffer(static_cast<const T *>(A.v) + bh * A.dv, A.dv * sizeof(T));
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = to_f32(bload<T>(values, (col + e) * sizeof(T)));
  __syncthreads();
  f32x4 pk = {0, 0, 0, 0}, pq = {0, 0, 0, 0};
  float qk = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float kv = sk[rg + 8 * i], qv = sq[rg + 8 * i];
    x[i] *= a;
    pk += x[i] * kv;
    pq += x[i] * qv;
    qk = __builtin_fmaf(qv, kv, qk);
  }
#pragma unroll
  for (int o = 8; o < 64; o *= 2) {
    qk += __shfl_xor(qk, o);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      pk[e] += __shfl_xor(pk[e], o);
      pq[e] += __shfl_xor(pq[e], o);
    }
  }
  const f32x4 err = (v - pk) * beta;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const f32x4 y = x[i] + err * sk[rg + 8 * i];
    if (VEC)
      bstore16(S, at[0] + i * step, __builtin_bit_cast(u32x4, y));
    else
#pragma unroll
      for (int e = 0; e < 4; ++e) bstore(S, at[e] + i * step, y[e]);
  }
  store_out((pq + err * qk) * A.scale);
}

template <typename T, int DK>
hipError_t launch(const StepArgs &a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(a.batch) * a.hv * ((a.dv + kCols - 1) / kCols)));
  const bool vec = a.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
  if (vec)
    hipLaunchKernelGGL((delta_step_kernel<T, DK, true>), grid, dim3(64), 0, s, a);
  else
    hipLaunchKernelGGL((delta_step_kernel<T, DK, false>), grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_step(const StepArgs &a, bool bf16, hipStream_t s) {
  if (a.dk <= 64) return bf16 ? launch<bf16_t, 64>(a, s) : launch<float, 64>(a, s);
  return bf16 ? launch<bf16_t, 128>(a, s) : launch<float, 128>(a, s);
}

}  // namespace vmk
