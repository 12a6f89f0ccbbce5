// Gated delta rule, backward: the gradients of a chunk once the states before
// it (S), their gradients after it (dS), the corrected values (V) and the
// gradients dR of the triangular system's right side are known.
//
// With G the running log decay, D_ij = exp(G_i - G_j), w = exp(G_C - G):
//   M  = scale D (dout V^T)   (j <= i),   N = -D (dR V^T)   (j < i)
//   X  = dR S^T,  Y = N K
//   dq = scale e^G (dout S^T) + M K
//   Z1 = w (V dS^T) + M^T Q + (beta N)^T K,   Z2 = beta Y - beta e^G X
//   dk = Z1 + Z2
//   dbeta = rowsum(dR v) - e^G k.X + k.Y
//   dG = q.dq + k.(Z2 - Z1);  the chunk's last G also e^{G_C} <S, dS> + sum k.(w V dS^T)
//   dg_t = sum of dG over the steps >= t of the chunk
// (every decay factor of a product of i and j counts once for i and once
// against j, so the sums over its terms are dot products of what is there).
#include <hip/hip_runtime.h>

#include "delta_device.h"

namespace vmk {
namespace {

constexpr int kThreads = 512;
constexpr int kSlice = 32;              // value columns of one pass
constexpr int kPitchS = kSlice + 4;

template <int PITCH>
__device__ __forceinline__ f32x4 tile_a(const float *m, int rt, int kt, int li, int lg) {
  return load4(m + (16 * rt + li) * PITCH + 16 * kt + 4 * lg);
}
template <int PITCH>
__device__ __forceinline__ f32x4 tile_at(const float *m, int rt, int kt, int li, int lg) {
  const float *p = m + (16 * kt + 4 * lg) * PITCH + 16 * rt + li;
  return f32x4{p[0], p[PITCH], p[2 * PITCH], p[3 * PITCH]};
}

// Four values of a row at column c of [..][d], zero past the row's end.
template <typename T>
__device__ __forceinline__ f32x4 load_row4(const T *row, int c, int d, bool vec) {
  if (vec) return c < d ? load4(row + c) : f32x4{0, 0, 0, 0};
  f32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < d) v[e] = to_f32(row[c + e]);
  return v;
}

// One workgroup per (chunk slot, key head), the value heads of the key head in
// turn: dq and dk are summed over them in registers.  Wave w owns rows
// 16 (w % 4) .. and half w / 4 of the columns.
template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void delta_grad_kernel(DeltaArgs A) {
  constexpr int kPitch = DK + 4, kNt = DK / 32;
  __shared__ float sk[kC * kPitch];
  __shared__ float sq[kC * kPitch];
  __shared__ float slice[(2 * DK + 3 * kC) * kPitchS];
  __shared__ double sg[kC];
  __shared__ float seg[kC], sw[kC], sbeta[kC], srv[kC], swk[8], sdot[8];
  __shared__ float sgam[2][kC], sbet[2][kC];
  float *sS = slice, *sD = sS + DK * kPitchS, *sO = sD + DK * kPitchS, *sV = sO + kC * kPitchS,
        *sR = sV + kC * kPitchS;
  static_assert((2 * DK + 3 * kC) * kPitchS >= 2 * kC * kPitchC, "the masked products reuse the slices");
  float *sm = slice, *sn = slice + kC * kPitchC;
  const int64_t slot = blockIdx.x;
  const Seq q = sequence(A, sequence_of(A, slot));
  const int64_t c0 = (slot - q.slot0) * kC;
  if (c0 >= q.len || c0 < 0) return;
  const int n = q.len - c0 < kC ? static_cast<int>(q.len - c0) : kC;
  const int kh = blockIdx.y, group = A.hv / A.hk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16,
            lg = lane / 16;
  const int rt = wave % 4, half = wave / 4;
  const int64_t t0 = token_of(A, q, c0, 0), dt = A.reverse ? -1 : 1;
  stage_rows<DK, kPitch, kThreads>(sk, static_cast<const T *>(A.k) + t0 * A.ks + static_cast<int64_t>(kh) * A.dk,
                                   dt * A.ks, n, A.dk, can_vec4(A.k, A.ks, A.dk, sizeof(T)));
  stage_rows<DK, kPitch, kThreads>(sq, static_cast<const T *>(A.q) + t0 * A.qs + static_cast<int64_t>(kh) * A.dk,
                                   dt * A.qs, n, A.dk, can_vec4(A.q, A.qs, A.dk, sizeof(T)));
  const bool vec_s = (A.dv & 3) == 0;
  const bool vec_o = can_vec4(A.dout, A.dv, A.dv, sizeof(T)), vec_v = can_vec4(A.v, A.vs, A.dv, sizeof(T));
  const f32x4 zero = {0, 0, 0, 0};
  f32x4 dq[kNt], dk[kNt];
#pragma unroll
  for (int c = 0; c < kNt; ++c) dq[c] = dk[c] = zero;
  for (int e = 0; e < group; ++e) {
    const int h = kh * group + e;
    const int64_t at = slot * A.hv + h;
    __syncthreads();
    if (threadIdx.x < kC) {
      const int i = threadIdx.x;
      const double gi = A.gam[at * kC + i], gl = A.gam[at * kC + kC - 1];
      sg[i] = gi;
      seg[i] = hw_exp2(static_cast<float>(gi) * kLog2e);
      sw[i] = hw_exp2(static_cast<float>(gl - gi) * kLog2e);
      sbeta[i] = i < n ? A.beta[token_of(A, q, c0, i) * A.hv + h] : 0.0f;
    }
    f32x4 aq[kNt], ak[kNt], ax[kNt], pm[2], pn[2];
#pragma unroll
    for (int c = 0; c < kNt; ++c) aq[c] = ak[c] = ax[c] = zero;
    pm[0] = pm[1] = pn[0] = pn[1] = zero;
    float dot = 0, rv = 0;
    const float *gS = A.S + at * A.dk * A.dv, *gD = A.dS + at * A.dk * A.dv;
    const float *gV = A.V + at * kC * A.dv, *gR = A.dR + at * kC * A.dv;
    for (int v0 = 0; v0 < A.dv; v0 += kSlice) {
      __syncthreads();
      for (int i = threadIdx.x; i < DK * (kSlice / 4); i += kThreads) {
        const int row = i / (kSlice / 4), c = (i % (kSlice / 4)) * 4;
        f32x4 x = zero, y = zero;
        if (row < A.dk) {
          x = load_row4(gS + static_cast<int64_t>(row) * A.dv, v0 + c, A.dv, vec_s);
          y = load_row4(gD + static_cast<int64_t>(row) * A.dv, v0 + c, A.dv, vec_s);
        }
        dot += x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
        *reinterpret_cast<f32x4 *>(sS + row * kPitchS + c) = x;
        *reinterpret_cast<f32x4 *>(sD + row * kPitchS + c) = y;
      }
      {
        static_assert(kC * (kSlice / 4) == kThreads, "one piece of a row to a thread");
        const int row = threadIdx.x / (kSlice / 4), c = (threadIdx.x % (kSlice / 4)) * 4;
        f32x4 o = zero, x = zero, r = zero, v = zero;
        if (row < n) {
          const int64_t t = t0 + dt * row;
          o = load_row4(static_cast<const T *>(A.dout) + (t * A.hv + h) * A.dv, v0 + c, A.dv, vec_o);
          v = load_row4(static_cast<const T *>(A.v) + t * A.vs + static_cast<int64_t>(h) * A.dv, v0 + c, A.dv, vec_v);
          x = load_row4(gV + static_cast<int64_t>(row) * A.dv, v0 + c, A.dv, vec_s);
          r = load_row4(gR + static_cast<int64_t>(row) * A.dv, v0 + c, A.dv, vec_s);
        }
        rv += r[0] * v[0] + r[1] * v[1] + r[2] * v[2] + r[3] * v[3];
        *reinterpret_cast<f32x4 *>(sO + row * kPitchS + c) = o;
        *reinterpret_cast<f32x4 *>(sV + row * kPitchS + c) = x;
        *reinterpret_cast<f32x4 *>(sR + row * kPitchS + c) = r;
      }
      __syncthreads();
#pragma unroll
      for (int kt = 0; kt < kSlice / 16; ++kt) {
        const f32x4 o = tile_a<kPitchS>(sO, rt, kt, li, lg), v = tile_a<kPitchS>(sV, rt, kt, li, lg),
                    r = tile_a<kPitchS>(sR, rt, kt, li, lg);
#pragma unroll
        for (int c = 0; c < kNt; ++c) {
          const f32x4 bs = tile_a<kPitchS>(sS, half * kNt + c, kt, li, lg),
                      bd = tile_a<kPitchS>(sD, half * kNt + c, kt, li, lg);
          aq[c] = mfma16(o, bs, aq[c]);
          ax[c] = mfma16(r, bs, ax[c]);
          ak[c] = mfma16(v, bd, ak[c]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (2 * half + c > rt) continue;
          const f32x4 b = tile_a<kPitchS>(sV, 2 * half + c, kt, li, lg);
          pm[c] = mfma16(o, b, pm[c]);
          pn[c] = mfma16(r, b, pn[c]);
        }
      }
    }
    __syncthreads();
    // masked products, and the sums that the staging threads hold
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * rt + 4 * lg + r, j = 16 * (2 * half + c) + li;
        const float d = i >= j ? hw_exp2(static_cast<float>(sg[i] - sg[j]) * kLog2e) : 0.0f;
        sm[i * kPitchC + j] = i >= j ? A.scale * d * pm[c][r] : 0.0f;
        sn[i * kPitchC + j] = i > j ? -d * pn[c][r] : 0.0f;
      }
#pragma unroll
    for (int o = 1; o < kSlice / 4; o *= 2) rv += __shfl_xor(rv, o);
    if (threadIdx.x % (kSlice / 4) == 0) srv[threadIdx.x / (kSlice / 4)] = rv;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) dot += __shfl_xor(dot, o);
    if (lane == 0) sdot[wave] = dot;
    __syncthreads();
    const f32x4 eg = load4(seg + 16 * rt + 4 * lg), w = load4(sw + 16 * rt + 4 * lg),
                be = load4(sbeta + 16 * rt + 4 * lg);
    f32x4 sum_g = zero, sum_b = zero, sum_w = zero;     // over this wave's columns
#pragma unroll
    for (int c = 0; c < kNt; ++c) {
      const int ct = half * kNt + c;
      f32x4 xq = aq[c] * eg * A.scale, z1 = ak[c] * w, y = zero;
      const f32x4 kr = tile_at<kPitch>(sk, ct, rt, li, lg), qr = tile_at<kPitch>(sq, ct, rt, li, lg);
      sum_w += z1 * kr;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        const f32x4 bk = tile_at<kPitch>(sk, ct, kt, li, lg);
        if (kt <= rt) {
          xq = mfma16(tile_a<kPitchC>(sm, rt, kt, li, lg), bk, xq);
          y = mfma16(tile_a<kPitchC>(sn, rt, kt, li, lg), bk, y);
        }
        if (kt >= rt) {
          const f32x4 bq = tile_at<kPitch>(sq, ct, kt, li, lg);
          z1 = mfma16(tile_at<kPitchC>(sm, rt, kt, li, lg), bq, z1);
          z1 = mfma16(tile_at<kPitchC>(sn, rt, kt, li, lg) * load4(sbeta + 16 * kt + 4 * lg), bk, z1);
        }
      }
      const f32x4 x = ax[c] * eg, z2 = (y - x) * be;
      sum_b += kr * (y - x);
      sum_g += qr * xq + kr * (z2 - z1);
      dq[c] += xq;
      dk[c] += z1 + z2;
    }
#pragma unroll
    for (int o = 1; o < 16; o *= 2)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        sum_g[r] += __shfl_xor(sum_g[r], o);
        sum_b[r] += __shfl_xor(sum_b[r], o);
        sum_w[r] += __shfl_xor(sum_w[r], o);
      }
    float all_w = sum_w[0] + sum_w[1] + sum_w[2] + sum_w[3];
    all_w += __shfl_xor(all_w, 16);
    all_w += __shfl_xor(all_w, 32);
    if (lane == 0) swk[wave] = all_w;
    if (li == 0)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        sgam[half][16 * rt + 4 * lg + r] = sum_g[r];
        sbet[half][16 * rt + 4 * lg + r] = sum_b[r];
      }
    __syncthreads();
    if (wave == 0) {
      float ss = 0, sk_all = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss += sdot[i];
        sk_all += swk[i];
      }
      float x = sgam[0][lane] + sgam[1][lane];
      if (lane == 63) x += seg[kC - 1] * ss + sk_all;
      for (int o = 1; o < 64; o *= 2) {
        const float y = __shfl_down(x, o);
        if (lane + o < 64) x += y;
      }
      if (lane < n) {
        const int64_t i = token_of(A, q, c0, lane) * A.hv + h;
        A.dg[i] = A.g[i] < kMinLogDecay ? 0.0f : x;
        A.dbeta[i] = srv[lane] + sbet[0][lane] + sbet[1][lane];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kNt; ++c)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * rt + 4 * lg + r, col = 16 * (half * kNt + c) + li;
      if (i < n && col < A.dk) {
        const int64_t o = ((t0 + dt * i) * A.hk + kh) * A.dk + col;
        static_cast<T *>(A.dq)[o] = from_f32<T>(dq[c][r]);
        static_cast<T *>(A.dkey)[o] = from_f32<T>(dk[c][r]);
      }
    }
}

template <typename T, int DK>
hipError_t launch(const DeltaArgs &a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(a.slots), a.hk);
  hipLaunchKernelGGL((delta_grad_kernel<T, DK>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grad(const DeltaArgs &a, bool bf16, hipStream_t s) {
  if (a.dk <= 64) return bf16 ? launch<bf16_t, 64>(a, s) : launch<float, 64>(a, s);
  return bf16 ? launch<bf16_t, 128>(a, s) : launch<float, 128>(a, s);
}

}  // namespace vmk
