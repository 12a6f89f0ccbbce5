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
//
// Bound by the latency of its chain (loads, products, substitution, blocks), so
// LDS is kept small for as many workgroups a compute unit as the registers
// allow: forward, a wave's queries go straight to its registers, and T takes
// the place of A.  4 x 4097 tokens, 8 and 16 heads of 128, bf16: 52 us for 34 MB
// read and 155 MB written (49 with a term less of P, and then 62 with queries and T
// in LDS of their own); 128 x 197 tokens, 6 heads of 64, fp32: 44 us.
template <typename T, int DK, bool BACK, bool VEC>
__global__ __launch_bounds__(kThreads, 4) void delta_prep_kernel(DeltaArgs A) {
  constexpr int kNi = kInputTerms<T>, kTerm = kC * DK, kPieces = DK / 8;
  constexpr int kUnitsT = tri_units(kNi == 1), kUnits = 2 * kUnitsT;
  __shared__ __attribute__((aligned(16))) uint16_t sk[kNi * kTerm];
  __shared__ __attribute__((aligned(16))) uint16_t sq[BACK ? kNi * kTerm : 8];
  __shared__ __attribute__((aligned(16))) float sa[kC * kPitchC];  // A, later T
  // inverses of the diagonal blocks, once the products are done
  float(*sd)[16 * 20] = reinterpret_cast<float(*)[16 * 20]>(sk);
  static_assert(sizeof(sk) >= 4 * 16 * 20 * sizeof(float), "");
  __shared__ double sg[4][kC];                                     // of up to four heads
  __shared__ float sbeta[4][kC];
  const int64_t slot = blockIdx.x;
  const Seq q = sequence(A, sequence_of(A, slot));
  const int64_t c0 = (slot - q.slot0) * kC;
  if (c0 >= q.len || c0 < 0) return;
  const Window w = window(A, q, c0);
  const int n = w.n;
  const int kh = blockIdx.y, group = A.hv / A.hk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16,
            lg = lane / 16;
  // gates of heads wave, wave + 4, ..: running sums, and what the scans take of them
  float gv = 0, bv = 0;
  auto load_gates = [&](int e) {
    gv = bv = 0;
    if (e < group && lane < n) {
      const int64_t i = token_of(A, q, c0, lane) * A.hv + kh * group + e;
      gv = A.g[i];
      bv = A.beta[i];
    }
  };
  auto sum_gates = [&](int e) {
    if (e >= group) return;
    const int64_t at = (slot * A.hv + kh * group + e) * kC + lane;
    double x = gv < kMinLogDecay ? kMinLogDecay : gv;
    for (int o = 1; o < 64; o *= 2) {
      const double y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    sg[wave][lane] = x;
    sbeta[wave][lane] = bv;
    A.eg[at] = hw_exp2(static_cast<float>(x) * kLog2e);
    A.ew[at] = hw_exp2(static_cast<float>(__shfl(x, 63) - x) * kLog2e);
    if (BACK) A.gam[at] = x;
  };
  bf16x8 fq[BACK ? 1 : DK / 32][kNi];      // forward: this wave's queries as right operands
  {
    load_gates(wave);
    const Rsrc rk = buffer(static_cast<const T *>(A.k) + w.low * A.ks + static_cast<int64_t>(kh) * A.dk);
    const Rsrc rq = buffer(static_cast<const T *>(A.q) + w.low * A.qs + static_cast<int64_t>(kh) * A.dk);
    constexpr int kPer = kC * kPieces / kThreads;
    Piece<T> pk[kPer], pq[BACK ? kPer : DK / 32];
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int i = threadIdx.x + x * kThreads, row = i / kPieces, p = i % kPieces;
      const bool in = row < n && 8 * p < A.dk;
      pk[x] = load_piece<VEC>(rk, in ? w.at(A, row, A.ks * sizeof(T)) + 8 * p * sizeof(T) : kNowhere, 8 * p, A.dk, T());
      if (BACK)
        pq[x] = load_piece<VEC>(rq, in ? w.at(A, row, A.qs * sizeof(T)) + 8 * p * sizeof(T) : kNowhere, 8 * p, A.dk, T());
    }
    if (!BACK) {
      const int row = 16 * wave + li;
      const uint32_t at = w.at(A, row, A.qs * sizeof(T));
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        const int c = 32 * ks + 8 * lg;
        pq[ks] = load_piece<VEC>(rq, row < n && c < A.dk ? at + c * sizeof(T) : kNowhere, c, A.dk, T());
      }
    }
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int i = threadIdx.x + x * kThreads, row = i / kPieces, p = i % kPieces;
      store_piece<DK>(sk, kTerm, row, p, pk[x]);
      if (BACK) store_piece<DK>(sq, kTerm, row, p, pq[x]);
    }
    if (!BACK)
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) piece_terms(pq[ks], fq[ks]);
    sum_gates(wave);
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
    bf16x8 bk[kNi];
#pragma unroll
    for (int t = 0; t < kNi; ++t) bk[t] = read8(sk + t * kTerm + swizzled<DK>(16 * wave + li, piece));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c <= wave) {
#pragma unroll
        for (int t = 0; t < kNi; ++t) {
          const bf16x8 ak = read8(sk + t * kTerm + swizzled<DK>(16 * c + li, piece));
#pragma unroll
          for (int u = 0; t + u < kNi; ++u) {
            kk[c] = mfma32(ak, bk[u], kk[c]);
            if (!BACK) qk[c] = mfma32(ak, fq[BACK ? 0 : ks][u], qk[c]);
          }
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
  for (int e = 0; e < group; ++e) {
    const int h = kh * group + e, s4 = e % 4;
    const int64_t at = slot * A.hv + h;
    if (e > 0) {
      __syncthreads();                     // the previous head's use of sa and sd
      if (s4 == 0) {
        load_gates(e + wave);
        sum_gates(e + wave);
        __syncthreads();
      }
    }
    f32x4 pt[4];
    {
      const int i = 16 * wave + li;        // (backward P: this is j)
      const double gi = sg[s4][i];
      const float bi = sbeta[s4][i];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        pt[c] = f32x4{0, 0, 0, 0};
        f32x4 a = {0, 0, 0, 0};
        if (c <= wave || BACK) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * c + 4 * lg + r;
            const double diff = gi - sg[s4][j];
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
      uint16_t *dst = (BACK ? A.TT : A.T) + (at * kUnits + kUnitsT) * kTriTerm;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (BACK ? (wave >= 2 && ks == 0) : (wave < 2 && ks == 1)) continue;
        put_block<T, kTerms>(dst, BACK ? tri_block_t(wave, ks) : tri_block(wave, ks), lane, pt[2 * ks], pt[2 * ks + 1]);
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
    }
    if (BACK) {                            // the transpose from the registers
      uint16_t *dst = A.TT + at * kUnits * kTriTerm;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (wave >= 2 && ks == 0) continue;
        put_block<T, kTerms>(dst, tri_block_t(wave, ks), lane, t[2 * ks], t[2 * ks + 1]);
      }
    }
    __syncthreads();                       // every wave has read A
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (a >= wave)
#pragma unroll
        for (int r = 0; r < 4; ++r) sa[(16 * a + 4 * lg + r) * kPitchC + 16 * wave + li] = t[a][r];
    __syncthreads();
    uint16_t *dst = A.T + at * (BACK ? kUnitsT : kUnits) * kTriTerm;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (wave < 2 && ks == 1) continue;
      const float *row = sa + (16 * wave + li) * kPitchC + 32 * ks + 4 * lg;
      const f32x4 zero = {0, 0, 0, 0};
      const f32x4 lo = load4(row), hi = 2 * ks + 1 <= wave ? load4(row + 16) : zero;
      put_block<T, kTerms>(dst, tri_block(wave, ks), lane, lo, hi);
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
