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

// One workgroup per (chunk slot, key head).  The products of the keys with
// themselves and with the queries serve every value head of the key head.  G is
// summed in fp64: its differences then keep fp32 accuracy however strong the
// decay before them was.
//
// Wave w computes columns 16w .. of the transposed products (rows j, columns i):
// a lane then holds, for one i, the 8 values of j that a 16 x 32 block of P asks
// of it as a left operand, so P goes to memory from the registers.
template <typename T, int DK, bool BACK, bool VEC>
__global__ __launch_bounds__(kThreads) void delta_prep_kernel(DeltaArgs A) {
  constexpr int kNi = kInputTerms<T>, kTerm = kC * DK, kPieces = DK / 8;
  constexpr int kTermsP = kNi == 1 ? 2 : 3;
  constexpr int kRows = 2 * kNi * kTerm;                    // bf16 values of K and Q
  constexpr int kUnion = kRows * 2 > kC * kPitchC * 4 ? kRows * 2 : kC * kPitchC * 4;
  __shared__ __attribute__((aligned(16))) char raw[kUnion];  // K and Q, later T
  __shared__ __attribute__((aligned(16))) float sa[kC * kPitchC];
  __shared__ __attribute__((aligned(16))) float sd[4][16 * 20];  // inverses of the diagonal blocks
  __shared__ double sg[kC];
  __shared__ float sbeta[kC];
  uint16_t *sk = reinterpret_cast<uint16_t *>(raw), *sq = sk + kNi * kTerm;
  float *st = reinterpret_cast<float *>(raw);
  const int64_t slot = blockIdx.x;
  const Seq q = sequence(A, sequence_of(A, slot));
  const int64_t c0 = (slot - q.slot0) * kC;
  if (c0 >= q.len || c0 < 0) return;
  const int n = q.len - c0 < kC ? static_cast<int>(q.len - c0) : kC;
  const int kh = blockIdx.y;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16,
            lg = lane / 16;
  {
    const Window w = window(A, q, c0);
    const Rsrc k = buffer(static_cast<const T *>(A.k) + w.low * A.ks + static_cast<int64_t>(kh) * A.dk);
    const Rsrc qq = buffer(static_cast<const T *>(A.q) + w.low * A.qs + static_cast<int64_t>(kh) * A.dk);
    Piece<T> pk[kC * kPieces / kThreads], pq[kC * kPieces / kThreads];
#pragma unroll
    for (int x = 0; x < kC * kPieces / kThreads; ++x) {
      const int i = threadIdx.x + x * kThreads, row = i / kPieces, p = i % kPieces;
      const bool in = row < n && 8 * p < A.dk;
      pk[x] = load_piece<VEC>(k, in ? w.at(A, row, A.ks * sizeof(T)) + 8 * p * sizeof(T) : kNowhere, 8 * p, A.dk, T());
      pq[x] = load_piece<VEC>(qq, in ? w.at(A, row, A.qs * sizeof(T)) + 8 * p * sizeof(T) : kNowhere, 8 * p, A.dk, T());
    }
#pragma unroll
    for (int x = 0; x < kC * kPieces / kThreads; ++x) {
      const int i = threadIdx.x + x * kThreads, row = i / kPieces, p = i % kPieces;
      store_piece<DK>(sk, kTerm, row, p, pk[x]);
      store_piece<DK>(sq, kTerm, row, p, pq[x]);
    }
  }
  __syncthreads();
  // kk[c]: k_j.k_i, rows j of tile c, columns i of tile wave (c <= wave);
  // qk[c]: forward q_i.k_j of the same; backward rows i of tile c, columns j of
  // tile wave (c >= wave)
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) kk[c] = qk[c] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int ks = 0; ks < DK / 32; ++ks) {
    const int piece = 4 * ks + lg;
    bf16x8 bk[kNi], bq[kNi];
#pragma unroll
    for (int t = 0; t < kNi; ++t) {
      bk[t] = read8(sk + t * kTerm + swizzled<DK>(16 * wave + li, piece));
      bq[t] = read8(sq + t * kTerm + swizzled<DK>(16 * wave + li, piece));
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      bf16x8 ak[kNi];
#pragma unroll
      for (int t = 0; t < kNi; ++t) ak[t] = read8(sk + t * kTerm + swizzled<DK>(16 * c + li, piece));
      if (c <= wave) {
#pragma unroll
        for (int t = 0; t < kNi; ++t)
#pragma unroll
          for (int u = 0; t + u < kNi; ++u) {
            kk[c] = mfma32(ak[t], bk[u], kk[c]);
            if (!BACK) qk[c] = mfma32(ak[t], bq[u], qk[c]);
          }
      }
      if (BACK && c >= wave) {
#pragma unroll
        for (int t = 0; t < kNi; ++t) {
          const bf16x8 aq = read8(sq + t * kTerm + swizzled<DK>(16 * c + li, piece));
#pragma unroll
          for (int u = 0; t + u < kNi; ++u) qk[c] = mfma32(aq, bk[u], qk[c]);
        }
      }
    }
  }
  const int group = A.hv / A.hk;
  for (int e = 0; e < group; ++e) {
    const int h = kh * group + e;
    const int64_t at = slot * A.hv + h;
    __syncthreads();                       // the previous use of sa, sg and of raw
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
      A.eg[at * kC + lane] = hw_exp2(static_cast<float>(x) * kLog2e);
      A.ew[at * kC + lane] = hw_exp2(static_cast<float>(__shfl(x, 63) - x) * kLog2e);
      if (BACK) A.gam[at * kC + lane] = x;
    }
    __syncthreads();
    f32x4 pt[4];
    {
      const int i = 16 * wave + li;        // (backward P: this is j)
      const double gi = sg[i];
      const float bi = sbeta[i];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        pt[c] = f32x4{0, 0, 0, 0};
        f32x4 a = {0, 0, 0, 0};
        if (c <= wave || BACK) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * c + 4 * lg + r;
            const double diff = gi - sg[j];
            if (c <= wave) {
              const float d = hw_exp2(static_cast<float>(diff) * kLog2e);
              a[r] = j < i ? bi * d * kk[c][r] : 0.0f;
              if (!BACK) pt[c][r] = j <= i ? A.scale * d * qk[c][r] : 0.0f;
            }
            if (BACK && c >= wave) {
              const float d = hw_exp2(static_cast<float>(-diff) * kLog2e);
              pt[c][r] = j >= i ? A.scale * d * qk[c][r] : 0.0f;
            }
          }
          if (c <= wave) *reinterpret_cast<f32x4 *>(sa + i * kPitchC + 16 * c + 4 * lg) = a;
        }
      }
    }
    {
      uint16_t *dst = (BACK ? A.TT : A.T) + (at * (kTermsT + kTermsP) + kTermsT) * kTriTerm;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (BACK ? (wave >= 2 && ks == 0) : (wave < 2 && ks == 1)) continue;
        const Terms<kTermsP> t = split<kTermsP>(pt[2 * ks], pt[2 * ks + 1]);
        const int block = BACK ? tri_block_t(wave, ks) : tri_block(wave, ks);
#pragma unroll
        for (int x = 0; x < kTermsP; ++x)
          *reinterpret_cast<bf16x8 *>(dst + x * kTriTerm + (block * 64 + lane) * 8) = t.t[x];
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
    f32x4 t[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      t[a] = f32x4{0, 0, 0, 0};
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
      for (int r = 0; r < 4; ++r) st[(16 * a + 4 * lg + r) * kPitchC + 16 * wave + li] = t[a][r];
    }
    if (BACK) {                            // the transpose from the registers
      uint16_t *dst = A.TT + at * (kTermsT + kTermsP) * kTriTerm;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (wave >= 2 && ks == 0) continue;
        const Terms<kTermsT> x = split<kTermsT>(t[2 * ks], t[2 * ks + 1]);
#pragma unroll
        for (int y = 0; y < kTermsT; ++y)
          *reinterpret_cast<bf16x8 *>(dst + y * kTriTerm + (tri_block_t(wave, ks) * 64 + lane) * 8) = x.t[y];
      }
    }
    __syncthreads();
    uint16_t *dst = A.T + at * (kTermsT + (BACK ? 0 : kTermsP)) * kTriTerm;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (wave < 2 && ks == 1) continue;
      const float *row = st + (16 * wave + li) * kPitchC + 32 * ks + 4 * lg;
      const f32x4 zero = {0, 0, 0, 0};
      const f32x4 lo = load4(row), hi = 2 * ks + 1 <= wave ? load4(row + 16) : zero;
      const Terms<kTermsT> x = split<kTermsT>(lo, hi);
#pragma unroll
      for (int y = 0; y < kTermsT; ++y)
        *reinterpret_cast<bf16x8 *>(dst + y * kTriTerm + (tri_block(wave, ks) * 64 + lane) * 8) = x.t[y];
    }
  }
}

template <typename T, int DK, bool VEC>
hipError_t launch(const DeltaArgs &a, bool backward, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(a.slots), a.hk);
  if (backward)
    hipLaunchKernelGGL((delta_prep_kernel<T, DK, true, VEC>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((delta_prep_kernel<T, DK, false, VEC>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}
template <typename T, int DK>
hipError_t launch(const DeltaArgs &a, bool backward, hipStream_t s) {
  return delta_vec(a, sizeof(T)) ? launch<T, DK, true>(a, backward, s) : launch<T, DK, false>(a, backward, s);
}

}  // namespace

int64_t delta_slots(int64_t batch, int64_t L, int64_t n, bool packed) {
  return packed ? L / kC + n : batch * ((L + kC - 1) / kC);
}

hipError_t launch_delta_prep(const DeltaArgs &a, bool bf16, bool backward, hipStream_t s) {
  if (a.dk <= 64)
    return bf16 ? launch<bf16_t, 64>(a, backward, s) : launch<float, 64>(a, backward, s);
  return bf16 ? launch<bf16_t, 128>(a, backward, s) : launch<float, 128>(a, backward, s);
}

}  // namespace vmk
