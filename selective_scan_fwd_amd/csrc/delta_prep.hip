// Gated delta rule, the part of a chunk that needs no state.
//
// For the chunk's steps i, j with running log decay G:
//   A_ij = beta_i exp(G_i - G_j) k_i.k_j   (j < i)
//   T    = (I + A)^-1
//   P_ij = scale exp(G_i - G_j) q_i.k_j    (j <= i)
#include <hip/hip_runtime.h>

#include "delta_device.h"

namespace vmk {
namespace {

constexpr int kThreads = 256;

// One workgroup per (chunk slot, key head): wave w owns rows 16w .. 16w+15.
// The products of the keys with themselves and with the queries serve every
// value head of the key head.  G is summed in fp64: its differences then keep
// fp32 accuracy however strong the decay before them was.
template <typename T, int DK, bool NEED_P>
__global__ __launch_bounds__(kThreads) void delta_prep_kernel(DeltaArgs A) {
  constexpr int kPitch = DK + 4;
  __shared__ float sk[kC * kPitch];
  __shared__ float sq[NEED_P ? kC * kPitch : 4];
  __shared__ float sa[kC * kPitchC];
  __shared__ float sd[4][16 * 20];        // inverses of the diagonal blocks
  __shared__ double sg[kC];
  __shared__ float sbeta[kC];
  const int64_t slot = blockIdx.x;
  const int s = sequence_of(A, slot);
  const Seq q = sequence(A, s);
  const int64_t c0 = (slot - q.slot0) * kC;
  if (c0 >= q.len || c0 < 0) return;
  const int n = q.len - c0 < kC ? static_cast<int>(q.len - c0) : kC;
  const int kh = blockIdx.y;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16, lg = lane / 16;
  const int64_t t0 = token_of(A, q, c0, 0), dt = A.reverse ? -1 : 1;
  {
    const T *k = static_cast<const T *>(A.k) + t0 * A.ks + static_cast<int64_t>(kh) * A.dk;
    stage_rows<DK, kPitch, kThreads>(sk, k, dt * A.ks, n, A.dk, can_vec4(A.k, A.ks, A.dk, sizeof(T)));
    if (NEED_P) {
      const T *qq = static_cast<const T *>(A.q) + t0 * A.qs + static_cast<int64_t>(kh) * A.dk;
      stage_rows<DK, kPitch, kThreads>(sq, qq, dt * A.qs, n, A.dk, can_vec4(A.q, A.qs, A.dk, sizeof(T)));
    }
  }
  __syncthreads();
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) kk[c] = qk[c] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int kt = 0; kt < DK / 16; ++kt) {
    const f32x4 ak = load4(sk + (16 * wave + li) * kPitch + 16 * kt + 4 * lg);
    f32x4 aq;
    if (NEED_P) aq = load4(sq + (16 * wave + li) * kPitch + 16 * kt + 4 * lg);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c > wave) break;
      const f32x4 b = load4(sk + (16 * c + li) * kPitch + 16 * kt + 4 * lg);
      kk[c] = mfma16(ak, b, kk[c]);
      if (NEED_P) qk[c] = mfma16(aq, b, qk[c]);
    }
  }
  const int group = A.hv / A.hk;
  for (int e = 0; e < group; ++e) {
    const int h = kh * group + e;
    const int64_t at = slot * A.hv + h;
    __syncthreads();                       // the previous head's use of sa, sg
    if (wave == 0) {
      double x = 0;
      float b = 0;
      if (lane < n) {
        const int64_t i = token_of(A, q, c0, lane) * A.hv + h;
        const float gv = A.g[i];
        x = gv < kMinLogDecay ? kMinLogDecay : gv;
        b = A.beta[i];
      }
      for (int o = 1; o < 64; o *= 2) {
        const double y = __shfl_up(x, o);
        if (lane >= o) x += y;
      }
      sg[lane] = x;
      sbeta[lane] = b;
      A.gam[at * kC + lane] = x;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c > wave) break;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * wave + 4 * lg + r, j = 16 * c + li;
        const float d = i >= j ? hw_exp2(static_cast<float>(sg[i] - sg[j]) * kLog2e) : 0.0f;
        sa[i * kPitchC + j] = i > j ? sbeta[i] * d * kk[c][r] : 0.0f;
        if (NEED_P) A.P[at * kC * kC + i * kC + j] = i >= j ? A.scale * d * qk[c][r] : 0.0f;
      }
    }
    __syncthreads();
    // T by block columns of 16: wave b inverts diagonal block b by forward
    // substitution (one column to a lane; as stable as the recurrence itself,
    // where powers of A would cancel), then T_ab = -T_aa sum_m A_am T_mb.
    {
      float x[16];
      const float *d = sa + 16 * wave * kPitchC + 16 * wave;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float v = i == li ? 1.0f : 0.0f;
#pragma unroll
        for (int m = 0; m < i; ++m) v = __builtin_fmaf(-d[i * kPitchC + m], x[m], v);
        x[i] = v;
      }
      if (lg == 0)
#pragma unroll
        for (int i = 0; i < 16; ++i) sd[wave][i * 20 + li] = x[i];
    }
    __syncthreads();
    float *out = A.T + at * kC * kC;
    f32x4 t[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a < wave) continue;
      if (a == wave) {
#pragma unroll
        for (int r = 0; r < 4; ++r) t[a][r] = sd[a][(4 * lg + r) * 20 + li];
      } else {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (m >= wave && m < a) acc = mfma16(load4(sa + (16 * a + li) * kPitchC + 16 * m + 4 * lg), t[m], acc);
        const f32x4 zero = {0, 0, 0, 0};
        t[a] = zero - mfma16(load4(&sd[a][li * 20 + 4 * lg]), acc, zero);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) out[(16 * a + 4 * lg + r) * kC + 16 * wave + li] = t[a][r];
    }
  }
}

template <typename T, int DK>
hipError_t launch(const DeltaArgs &a, bool need_p, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(a.slots), a.hk);
  if (need_p)
    hipLaunchKernelGGL((delta_prep_kernel<T, DK, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((delta_prep_kernel<T, DK, false>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int64_t delta_slots(int64_t batch, int64_t L, int64_t n, bool packed) {
  return packed ? L / kC + n : batch * ((L + kC - 1) / kC);
}

hipError_t launch_delta_prep(const DeltaArgs &a, bool bf16, bool need_p, hipStream_t s) {
  if (a.dk <= 64)
    return bf16 ? launch<bf16_t, 64>(a, need_p, s) : launch<float, 64>(a, need_p, s);
  return bf16 ? launch<bf16_t, 128>(a, need_p, s) : launch<float, 128>(a, need_p, s);
}

}  // namespace vmk
