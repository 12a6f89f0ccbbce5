// Gated delta rule, the pass over the chunks of a sequence that carries the
// state, forward and backward.
//
// With S the state before a chunk, G its running log decay and w = exp(G_C - G):
//   R = beta (v - e^G (K S)),  V = T R
//   out = scale e^G (Q S) + P V,  S <- e^{G_C} S + K^T (w V)
// and backward, with dS the gradient of the state after the chunk:
//   dV = P^T dout + w (K dS),  dR = T^T dV,  dv = beta dR
//   dS <- e^{G_C} dS + Q^T (scale e^G dout) - K^T (e^G beta dR)
#include <hip/hip_runtime.h>

#include "delta_device.h"

namespace vmk {
namespace {

// A wave owns 16 columns of the state: every product of the chunk stays within
// those columns, so a wave's chain of products passes from registers to
// registers and waves share only the chunk's operands in LDS.
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

template <typename T>
__device__ __forceinline__ float load_value(const T *p, bool ok) { return ok ? to_f32(*p) : 0.0f; }

// A[64][64] or its transpose from LDS as A operand: rows 16 rt.., inner 16 kt..
__device__ __forceinline__ f32x4 tile_a(const float *m, int rt, int kt, int li, int lg) {
  return load4(m + (16 * rt + li) * kPitchC + 16 * kt + 4 * lg);
}
template <int PITCH>
__device__ __forceinline__ f32x4 tile_at(const float *m, int rt, int kt, int li, int lg) {
  const float *p = m + (16 * kt + 4 * lg) * PITCH + 16 * rt + li;
  return f32x4{p[0], p[PITCH], p[2 * PITCH], p[3 * PITCH]};
}

__device__ __forceinline__ void stage_tile(float *dst, const float *src) {
  for (int i = threadIdx.x; i < kC * kC / 4; i += kThreads) {
    const int row = i / (kC / 4), c = (i % (kC / 4)) * 4;
    if (c / 16 <= row / 16)               // (blocks above the diagonal are never read)
      *reinterpret_cast<f32x4 *>(dst + row * kPitchC + c) = load4(src + row * kC + c);
  }
}

// Forward.  KEEP: S and V are stored for the backward pass, out and state not.
template <typename T, int DK, bool KEEP>
__global__ __launch_bounds__(kThreads) void delta_scan_kernel(DeltaArgs A) {
  constexpr int kPitch = DK + 4, kDt = DK / 16;
  __shared__ float sk[kC * kPitch];
  __shared__ float sq[KEEP ? 4 : kC * kPitch];
  __shared__ float st[kC * kPitchC];
  __shared__ float sp[KEEP ? 4 : kC * kPitchC];
  __shared__ float seg[kC], sw[kC], sbeta[kC];
  const int s = blockIdx.x, h = blockIdx.y, kh = h / (A.hv / A.hk);
  const Seq q = sequence(A, s);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16, lg = lane / 16;
  const int col = (blockIdx.z * kWaves + wave) * 16 + li;
  const bool mine = col < A.dv;
  const int64_t state_at = (static_cast<int64_t>(s) * A.hv + h) * A.dk * A.dv;
  f32x4 S[kDt];
#pragma unroll
  for (int d = 0; d < kDt; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * d + 4 * lg + r;
      S[d][r] = A.h0 != nullptr && mine && row < A.dk ? A.h0[state_at + static_cast<int64_t>(row) * A.dv + col] : 0.0f;
    }
  const bool vec_k = can_vec4(A.k, A.ks, A.dk, sizeof(T)), vec_q = can_vec4(A.q, A.qs, A.dk, sizeof(T));
  const int64_t dt = A.reverse ? -1 : 1;
  for (int64_t c0 = 0; c0 < q.len; c0 += kC) {
    const int n = q.len - c0 < kC ? static_cast<int>(q.len - c0) : kC;
    const int64_t at = (q.slot0 + c0 / kC) * A.hv + h;
    const int64_t t0 = token_of(A, q, c0, 0);
    __syncthreads();
    stage_rows<DK, kPitch, kThreads>(sk, static_cast<const T *>(A.k) + t0 * A.ks + static_cast<int64_t>(kh) * A.dk,
                                     dt * A.ks, n, A.dk, vec_k);
    stage_tile(st, A.T + at * kC * kC);
    if (!KEEP) {
      stage_rows<DK, kPitch, kThreads>(sq, static_cast<const T *>(A.q) + t0 * A.qs + static_cast<int64_t>(kh) * A.dk,
                                       dt * A.qs, n, A.dk, vec_q);
      stage_tile(sp, A.P + at * kC * kC);
    }
    if (threadIdx.x < kC) {
      const int i = threadIdx.x;
      const double gi = A.gam[at * kC + i], gl = A.gam[at * kC + kC - 1];
      seg[i] = hw_exp2(static_cast<float>(gi) * kLog2e);
      sw[i] = hw_exp2(static_cast<float>(gl - gi) * kLog2e);
      sbeta[i] = i < n ? A.beta[token_of(A, q, c0, i) * A.hv + h] : 0.0f;
    }
    f32x4 v[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * rt + 4 * lg + r;
        v[rt][r] = load_value(static_cast<const T *>(A.v) + (t0 + dt * i) * A.vs + static_cast<int64_t>(h) * A.dv + col,
                              mine && i < n);
      }
    __syncthreads();
    if (KEEP && mine)
#pragma unroll
      for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * d + 4 * lg + r;
          if (row < A.dk) A.S[at * A.dk * A.dv + static_cast<int64_t>(row) * A.dv + col] = S[d][r];
        }
    f32x4 R[4], V[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < kDt; ++d) x = mfma16(load4(sk + (16 * rt + li) * kPitch + 16 * d + 4 * lg), S[d], x);
      const f32x4 eg = load4(seg + 16 * rt + 4 * lg), b = load4(sbeta + 16 * rt + 4 * lg);
      R[rt] = b * (v[rt] - eg * x);
    }
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int kt = 0; kt <= rt; ++kt) x = mfma16(tile_a(st, rt, kt, li, lg), R[kt], x);
      V[rt] = x;
    }
    if (!KEEP) {
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        f32x4 x = {0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < kDt; ++d) x = mfma16(load4(sq + (16 * rt + li) * kPitch + 16 * d + 4 * lg), S[d], x);
        x = x * load4(seg + 16 * rt + 4 * lg) * A.scale;
#pragma unroll
        for (int kt = 0; kt <= rt; ++kt) x = mfma16(tile_a(sp, rt, kt, li, lg), V[kt], x);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * rt + 4 * lg + r;
          if (mine && i < n)
            static_cast<T *>(A.out)[((t0 + dt * i) * A.hv + h) * A.dv + col] = from_f32<T>(x[r]);
        }
      }
    } else if (mine) {
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int r = 0; r < 4; ++r) A.V[at * kC * A.dv + static_cast<int64_t>(16 * rt + 4 * lg + r) * A.dv + col] = V[rt][r];
    }
    const float last = seg[kC - 1];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) V[rt] = V[rt] * load4(sw + 16 * rt + 4 * lg);
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
      f32x4 x = S[d] * last;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) x = mfma16(tile_at<kPitch>(sk, d, kt, li, lg), V[kt], x);
      S[d] = x;
    }
  }
  if (!KEEP && A.state != nullptr && mine)
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * d + 4 * lg + r;
        if (row < A.dk) A.state[state_at + static_cast<int64_t>(row) * A.dv + col] = S[d][r];
      }
}

template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void delta_scan_bwd_kernel(DeltaArgs A) {
  constexpr int kPitch = DK + 4, kDt = DK / 16;
  __shared__ float sk[kC * kPitch];
  __shared__ float sq[kC * kPitch];
  __shared__ float st[kC * kPitchC];
  __shared__ float sp[kC * kPitchC];
  __shared__ float seg[kC], sw[kC], sbeta[kC];
  const int s = blockIdx.x, h = blockIdx.y, kh = h / (A.hv / A.hk);
  const Seq q = sequence(A, s);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16, lg = lane / 16;
  const int col = (blockIdx.z * kWaves + wave) * 16 + li;
  const bool mine = col < A.dv;
  const int64_t state_at = (static_cast<int64_t>(s) * A.hv + h) * A.dk * A.dv;
  f32x4 D[kDt];
#pragma unroll
  for (int d = 0; d < kDt; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * d + 4 * lg + r;
      D[d][r] = A.dstate != nullptr && mine && row < A.dk ? A.dstate[state_at + static_cast<int64_t>(row) * A.dv + col]
                                                          : 0.0f;
    }
  const bool vec_k = can_vec4(A.k, A.ks, A.dk, sizeof(T)), vec_q = can_vec4(A.q, A.qs, A.dk, sizeof(T));
  const int64_t dt = A.reverse ? -1 : 1;
  const int64_t chunks = (q.len + kC - 1) / kC;
  for (int64_t c0 = (chunks - 1) * kC; c0 >= 0; c0 -= kC) {
    const int n = q.len - c0 < kC ? static_cast<int>(q.len - c0) : kC;
    const int64_t at = (q.slot0 + c0 / kC) * A.hv + h;
    const int64_t t0 = token_of(A, q, c0, 0);
    __syncthreads();
    stage_rows<DK, kPitch, kThreads>(sk, static_cast<const T *>(A.k) + t0 * A.ks + static_cast<int64_t>(kh) * A.dk,
                                     dt * A.ks, n, A.dk, vec_k);
    stage_rows<DK, kPitch, kThreads>(sq, static_cast<const T *>(A.q) + t0 * A.qs + static_cast<int64_t>(kh) * A.dk,
                                     dt * A.qs, n, A.dk, vec_q);
    stage_tile(st, A.T + at * kC * kC);
    stage_tile(sp, A.P + at * kC * kC);
    if (threadIdx.x < kC) {
      const int i = threadIdx.x;
      const double gi = A.gam[at * kC + i], gl = A.gam[at * kC + kC - 1];
      seg[i] = hw_exp2(static_cast<float>(gi) * kLog2e);
      sw[i] = hw_exp2(static_cast<float>(gl - gi) * kLog2e);
      sbeta[i] = i < n ? A.beta[token_of(A, q, c0, i) * A.hv + h] : 0.0f;
    }
    f32x4 o[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * rt + 4 * lg + r;
        o[rt][r] = load_value(static_cast<const T *>(A.dout) + ((t0 + dt * i) * A.hv + h) * A.dv + col, mine && i < n);
      }
    __syncthreads();
    if (mine)
#pragma unroll
      for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * d + 4 * lg + r;
          if (row < A.dk) A.dS[at * A.dk * A.dv + static_cast<int64_t>(row) * A.dv + col] = D[d][r];
        }
    f32x4 V[4], R[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < kDt; ++d) x = mfma16(load4(sk + (16 * rt + li) * kPitch + 16 * d + 4 * lg), D[d], x);
      x = x * load4(sw + 16 * rt + 4 * lg);
#pragma unroll
      for (int kt = rt; kt < 4; ++kt) x = mfma16(tile_at<kPitchC>(sp, rt, kt, li, lg), o[kt], x);
      V[rt] = x;
    }
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int kt = rt; kt < 4; ++kt) x = mfma16(tile_at<kPitchC>(st, rt, kt, li, lg), V[kt], x);
      R[rt] = x;
    }
    const float last = seg[kC - 1];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const f32x4 b = load4(sbeta + 16 * rt + 4 * lg), eg = load4(seg + 16 * rt + 4 * lg);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * rt + 4 * lg + r;
        if (mine) {
          A.dR[at * kC * A.dv + static_cast<int64_t>(i) * A.dv + col] = R[rt][r];
          if (i < n)
            static_cast<T *>(A.dval)[((t0 + dt * i) * A.hv + h) * A.dv + col] = from_f32<T>(b[r] * R[rt][r]);
        }
      }
      R[rt] = R[rt] * eg * b;
      o[rt] = o[rt] * eg * A.scale;
    }
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) x = mfma16(tile_at<kPitch>(sk, d, kt, li, lg), R[kt], x);
      x = D[d] * last - x;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) x = mfma16(tile_at<kPitch>(sq, d, kt, li, lg), o[kt], x);
      D[d] = x;
    }
  }
  if (A.dh0 != nullptr && mine)
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * d + 4 * lg + r;
        if (row < A.dk) A.dh0[state_at + static_cast<int64_t>(row) * A.dv + col] = D[d][r];
      }
}

template <typename T, int DK>
hipError_t launch_fwd(const DeltaArgs &a, bool keep, hipStream_t s) {
  const dim3 grid(a.nseq, a.hv, (a.dv + 16 * kWaves - 1) / (16 * kWaves));
  if (keep)
    hipLaunchKernelGGL((delta_scan_kernel<T, DK, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((delta_scan_kernel<T, DK, false>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}
template <typename T, int DK>
hipError_t launch_bwd(const DeltaArgs &a, hipStream_t s) {
  const dim3 grid(a.nseq, a.hv, (a.dv + 16 * kWaves - 1) / (16 * kWaves));
  hipLaunchKernelGGL((delta_scan_bwd_kernel<T, DK>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs &a, bool bf16, bool keep, hipStream_t s) {
  if (a.dk <= 64) return bf16 ? launch_fwd<bf16_t, 64>(a, keep, s) : launch_fwd<float, 64>(a, keep, s);
  return bf16 ? launch_fwd<bf16_t, 128>(a, keep, s) : launch_fwd<float, 128>(a, keep, s);
}

hipError_t launch_delta_scan_bwd(const DeltaArgs &a, bool bf16, hipStream_t s) {
  if (a.dk <= 64) return bf16 ? launch_bwd<bf16_t, 64>(a, s) : launch_bwd<float, 64>(a, s);
  return bf16 ? launch_bwd<bf16_t, 128>(a, s) : launch_bwd<float, 128>(a, s);
}

}  // namespace vmk
