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
//        = <S, dS before the chunk> - sum of dG over the steps < t
// (the second form where S is 0, so that the first token of a sequence without a
// state has a gradient of 0 and not what rounding leaves of the sum)
// (every decay factor of a product of i and j counts once for i and once
// against j, so the sums over its terms are dot products of what is there).
#include <hip/hip_runtime.h>

#include "delta_device.h"

namespace vmk {
namespace {

constexpr int kThreads = 512;
constexpr int kSlice = 32;              // value columns of one pass, one inner step of the products
constexpr int kSlicePieces = kSlice / 8;

// Rows of a slice: 64 bytes a term; piece p of row r at place p ^ (r / 4).
__device__ __forceinline__ int slice_at(int row, int piece) {
  return row * kSlice + ((piece ^ ((row >> 2) & 3)) << 3);
}

// The first phase's operands, in terms.
template <typename T, int DK>
struct SliceLds {
  static constexpr int kState = DK * kSlice, kRows = kC * kSlice;   // values of a term
  __attribute__((aligned(16))) uint16_t s[3 * kState], d[3 * kState], v[3 * kRows], r[3 * kRows],
      o[kInputTerms<T> * kRows];
};
// The second phase's: K and Q, and the masked products as left operands.
template <typename T, int DK>
struct KeyLds {
  static constexpr int kTerm = kC * DK;
  __attribute__((aligned(16))) uint16_t m[kInputTerms<T> * kTerm];
};
struct MaskedLds {
  __attribute__((aligned(16))) uint16_t m[4][3 * kTriTerm];   // M, its transpose, N, its transpose
};

__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
  return __builtin_fmaf(a[0], b[0], __builtin_fmaf(a[1], b[1], __builtin_fmaf(a[2], b[2], a[3] * b[3])));
}
__device__ __forceinline__ f32x4 as_f32(u32x4 x) { return __builtin_bit_cast(f32x4, x); }
// The piece's values in fp32.
__device__ __forceinline__ void widen(const Piece<float> &p, f32x4 &a, f32x4 &b) {
  a = as_f32(p.x[0]);
  b = as_f32(p.x[1]);
}
__device__ __forceinline__ void widen(const Piece<bf16_t> &p, f32x4 &a, f32x4 &b) {
  a = f32x4{__uint_as_float(p.x[0] << 16), __uint_as_float(p.x[0] & 0xffff0000u), __uint_as_float(p.x[1] << 16),
            __uint_as_float(p.x[1] & 0xffff0000u)};
  b = f32x4{__uint_as_float(p.x[2] << 16), __uint_as_float(p.x[2] & 0xffff0000u), __uint_as_float(p.x[3] << 16),
            __uint_as_float(p.x[3] & 0xffff0000u)};
}
template <int TERMS, int TERM>
__device__ __forceinline__ void put_terms(uint16_t *m, int row, int piece, f32x4 a, f32x4 b) {
  const Terms<TERMS> t = split<TERMS>(a, b);
#pragma unroll
  for (int i = 0; i < TERMS; ++i) *reinterpret_cast<bf16x8 *>(m + i * TERM + slice_at(row, piece)) = t.t[i];
}

// c += a b over the terms whose places add up to less than three.
template <int NA, int NB>
__device__ __forceinline__ f32x4 product(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
#pragma unroll
  for (int t = 0; t < NA; ++t)
#pragma unroll
    for (int u = 0; u < NB; ++u)
      if (t + u < 3) c = mfma32(a[t], b[u], c);
  return c;
}
template <int N, int TERM>
__device__ __forceinline__ void read_slice(const uint16_t *m, int row, int lg, bf16x8 (&x)[N]) {
#pragma unroll
  for (int t = 0; t < N; ++t) x[t] = read8(m + t * TERM + slice_at(row, lg));
}
// Columns 16 ct .. of four rows at `row`, transposed (natural column order).
template <int DK>
__device__ __forceinline__ s16x4 read_tile(const uint16_t *m, int row, int ct, int li) {
  const int c = li % 4;
  const uint16_t *p = m + swizzled<DK>(row + li / 4, 2 * ct + c / 2) + 4 * (c % 2);
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4 *)const_cast<uint16_t *>(p));
}
template <int N, int DK>
__device__ __forceinline__ f32x4 tile_values(const uint16_t *m, int row, int ct, int li) {
  f32x4 x = {0, 0, 0, 0};
#pragma unroll
  for (int t = N - 1; t >= 0; --t) {
    const s16x4 y = read_tile<DK>(m + t * kC * DK, row, ct, li);
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] += to_f32(static_cast<bf16_t>(y[r]));
  }
  return x;
}
// Columns 16 ct .. of K or Q as a right operand over rows 32 ks ..
template <int N, int DK>
__device__ __forceinline__ void read_right(const uint16_t *m, int ks, int ct, int li, int lg, bf16x8 (&x)[N]) {
#pragma unroll
  for (int t = 0; t < N; ++t)
    x[t] = join(read_tile<DK>(m + t * kC * DK, 32 * ks + 4 * lg, ct, li),
                read_tile<DK>(m + t * kC * DK, 32 * ks + 16 + 4 * lg, ct, li));
}

// Tiles (c, pt0) and (c, pt1) of rows of `a` by rows of `b`, c <= pt (UP: c >= pt).
template <int NA, int NB, int TERM, bool UP>
__device__ __forceinline__ void masked_tiles(const uint16_t *a, const uint16_t *b, int pt0, int pt1, int li, int lg,
                                             f32x4 (&p0)[2], f32x4 (&p1)[4]) {
  bf16x8 b0[NB], b1[NB];
  read_slice<NB, TERM>(b, 16 * pt0 + li, lg, b0);
  read_slice<NB, TERM>(b, 16 * pt1 + li, lg, b1);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    bf16x8 x[NA];
    read_slice<NA, TERM>(a, 16 * c + li, lg, x);
    if (UP ? c >= 2 && c >= pt0 : c < 2 && c <= pt0) p0[c % 2] = product(x, b0, p0[c % 2]);
    if (UP ? c >= pt1 : c <= pt1) p1[c] = product(x, b1, p1[c]);
  }
}

// One workgroup per (chunk slot, key head), the value heads of the key head in
// turn: dq and dk are summed over them in registers.
//
// 2 x 4097 tokens, 8 and 16 heads of 128, bf16: 250 us for 480 MB, mostly states
// (matrix instructions busy 17 % of it, the vector ones 27 %, LDS 26 %); 64 x 197
// tokens, 6 heads of 64, fp32: 115 us.  One workgroup fills a compute unit's LDS
// and registers, so its phases (a slice's loads, their splitting, the products,
// the second phase) do not overlap with another's.  Measured and not better:
// slices loaded two ahead (293 us, spills), states from memory to the registers
// of the one wave that needs them (270 to 300), 16 waves (290), the next head's
// loads before the second phase (no change), staying for another chunk with its
// first loads issued (fp32 109, bf16 310: spills).
//
// Products with S and dS: wave w owns rows 16 (w % 4) .. and half w / 4 of the
// columns.  Of the four masked products (M, N and their transposes, each as
// the left operand that the second phase needs) two waves compute one, five
// 16 x 16 tiles a wave: the rows (lanes) of tiles 0 and 3, or of 1 and 2.
template <typename T, int DK, bool VEC>
__global__ __launch_bounds__(kThreads) void delta_grad_kernel(DeltaArgs A) {
  constexpr int kNt = DK / 32, kNi = kInputTerms<T>;
  typedef SliceLds<T, DK> Slice;
  typedef KeyLds<T, DK> Key;
  // The masked products take the slices' place.  K and Q have their own where
  // there is room, and are loaded once; else (fp32 rows of 128) they are loaded
  // for every head, one after the other into one place.
  constexpr size_t kMost = 157 * 1024, kPhase1 = sizeof(Slice) > sizeof(MaskedLds) ? sizeof(Slice) : sizeof(MaskedLds);
  constexpr bool kOwnKeys = kPhase1 + 2 * sizeof(Key) <= kMost;
  constexpr int kBuffers = 2 * sizeof(Slice) + (kOwnKeys ? 2 * sizeof(Key) : 0) <= kMost ? 2 : 1;
  constexpr size_t kShared1 = kBuffers * sizeof(Slice) > kPhase1 ? kBuffers * sizeof(Slice) : kPhase1;
  constexpr size_t kShared2 = sizeof(MaskedLds) + sizeof(Key);
  constexpr size_t kBytes = kOwnKeys ? kShared1 + 2 * sizeof(Key) : kShared1 > kShared2 ? kShared1 : kShared2;
  __shared__ __attribute__((aligned(16))) char raw[kBytes];
  __shared__ double sg[kC];
  __shared__ __attribute__((aligned(16))) float seg[kC], sw[kC], sbeta[kC], srv[kC];
  __shared__ float swk[8], sdot[8], sgam[2][kC], sbet[2][kC], sgate[kC];
  __shared__ bool sstate[8];
  Slice *slices = reinterpret_cast<Slice *>(raw);
  MaskedLds &pr = *reinterpret_cast<MaskedLds *>(raw);
  Key *keys = reinterpret_cast<Key *>(raw + (kOwnKeys ? kShared1 : sizeof(MaskedLds)));
  uint16_t *key_k = keys[0].m, *key_q = keys[kOwnKeys ? 1 : 0].m;
  const int64_t slot = blockIdx.x;
  const Seq q = sequence(A, sequence_of(A, slot));
  const int64_t c0 = (slot - q.slot0) * kC;
  if (c0 >= q.len || c0 < 0) return;
  const Window win = window(A, q, c0);
  const int n = win.n;
  const int kh = blockIdx.y, group = A.hv / A.hk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16,
            lg = lane / 16;
  const int rt = wave % 4, half = wave / 4;
  // masked products: of pt0 at most two tiles are not zero, c % 2 in p0
  const int pm = wave / 2, pta = wave % 2, pt0 = pm % 2 == 0 ? pta : 3 - pta, pt1 = 3 - pt0;
  const f32x4 zero = {0, 0, 0, 0};
  // a thread's piece of S and dS, and of dR and v (first half) or V and dout
  const int srow = threadIdx.x / kSlicePieces, piece = threadIdx.x % kSlicePieces, row = srow % kC;
  static_assert(kC * kSlicePieces == 4 * 64, "the first half is waves 0 to 3");
  const bool first = wave < 4;
  const int64_t os = static_cast<int64_t>(A.hv) * A.dv;
  const uint32_t at_v = row < n ? win.at(A, row, (first ? A.vs : os) * sizeof(T)) : kNowhere;
  Piece<float> ls, ld, lx;
  Piece<T> ly;
  auto load = [&](int h, int v0) {
    const int64_t at = slot * A.hv + h;
    const int c = v0 + 8 * piece;
    if (wave < DK / 16) {                  // (16 rows of a state to a wave)
      const uint32_t o = c < A.dvp ? (srow * A.dvp + c) * 4 : kNowhere;
      ls = load_piece<true>(buffer(A.S + at * A.dk * A.dvp, A.dk * A.dvp * 4), o, c, A.dvp, 0.0f);
      ld = load_piece<true>(buffer(A.dS + at * A.dk * A.dvp, A.dk * A.dvp * 4), o, c, A.dvp, 0.0f);
    }
    lx = load_piece<true>(buffer((first ? A.dR : A.V) + at * kC * A.dvp), c < A.dvp ? (row * A.dvp + c) * 4 : kNowhere, c,
                          A.dvp, 0.0f);
    const T *t = first ? static_cast<const T *>(A.v) + win.low * A.vs : static_cast<const T *>(A.dout) + win.low * os;
    ly = load_piece<VEC>(buffer(t + static_cast<int64_t>(h) * A.dv), c < A.dv ? at_v + c * sizeof(T) : kNowhere, c, A.dv, T());
  };
  double gate_g = 0;
  float gate_eg = 0, gate_ew = 0, gate_b = 0, gate_in = 0;
  auto load_gates = [&](int h) {           // (wave 7, which has least to do)
    if (wave == 7) {
      const int64_t at = (slot * A.hv + h) * kC + lane;
      gate_g = A.gam[at];
      gate_eg = A.eg[at];
      gate_ew = A.ew[at];
      if (lane < n) {
        const int64_t i = token_of(A, q, c0, lane) * A.hv + h;
        gate_b = A.beta[i];
        gate_in = A.g[i];
      }
    }
  };
  constexpr int kPieces = DK / 8, kPer = kC * kPieces / kThreads;
  auto load_keys = [&](const void *base, int64_t stride, uint16_t *dst) {
    const Rsrc r = buffer(static_cast<const T *>(base) + win.low * stride + static_cast<int64_t>(kh) * A.dk);
    Piece<T> x[kPer];
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const int i = threadIdx.x + y * kThreads, row = i / kPieces, p = i % kPieces;
      const uint32_t o = row < n && 8 * p < A.dk ? win.at(A, row, stride * sizeof(T)) + 8 * p * sizeof(T) : kNowhere;
      x[y] = load_piece<VEC>(r, o, 8 * p, A.dk, T());
    }
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const int i = threadIdx.x + y * kThreads;
      store_piece<DK>(dst, Key::kTerm, i / kPieces, i % kPieces, x[y]);
    }
  };
  // everything that the first head needs is on its way at once
  load_gates(kh * group);
  load(kh * group, 0);
  if (kOwnKeys) {
    load_keys(A.k, A.ks, key_k);
    load_keys(A.q, A.qs, key_q);
  }
  f32x4 dq[kNt], dk[kNt];
#pragma unroll
  for (int c = 0; c < kNt; ++c) dq[c] = dk[c] = zero;
  for (int e = 0; e < group; ++e) {
    const int h = kh * group + e;
    __syncthreads();
    if (wave == 7) {
      sg[lane] = gate_g;
      seg[lane] = gate_eg;
      sw[lane] = gate_ew;
      sbeta[lane] = gate_b;
      sgate[lane] = gate_in;
    }
    const int lane0 = lane;
    f32x4 aq[kNt], ak[kNt], ax[kNt], p0[2], p1[4];
#pragma unroll
    for (int c = 0; c < kNt; ++c) aq[c] = ak[c] = ax[c] = zero;
#pragma unroll
    for (int c = 0; c < 4; ++c) p0[c / 2] = p1[c] = zero;
    float dot = 0, rv = 0;
    uint32_t bits = 0;                       // of the state, to see whether it is 0
    auto store = [&](Slice &l) {
      f32x4 a, b, x, y;
      if (wave < DK / 16) {                  // (16 rows of a state to a wave)
        widen(ls, a, b);
        widen(ld, x, y);
        dot += dot4(a, x) + dot4(b, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) bits |= ls.x[0][i] | ls.x[1][i];
        put_terms<3, Slice::kState>(l.s, srow, piece, a, b);
        put_terms<3, Slice::kState>(l.d, srow, piece, x, y);
      }
      widen(lx, a, b);
      widen(ly, x, y);
      put_terms<3, Slice::kRows>(first ? l.r : l.v, row, piece, a, b);
      if (first)
        rv += dot4(a, x) + dot4(b, y);
      else
        put_terms<kNi, Slice::kRows>(l.o, row, piece, x, y);
    };
    store(slices[0]);
    __syncthreads();
    int buf = 0;
    for (int v0 = 0; v0 < A.dv; v0 += kSlice) {
      const Slice &l = slices[buf];
      // (so that the addresses of this phase are not held through the second)
      int lane1 = lane0;
      asm volatile("" : "+v"(lane1));
      const int li = lane1 % 16, lg = lane1 / 16;
      const bool more = v0 + kSlice < A.dv;
      if (more) load(h, v0 + kSlice);
      {
        bf16x8 o[kNi], v[3], r[3];
        read_slice<kNi, Slice::kRows>(l.o, 16 * rt + li, lg, o);
        read_slice<3, Slice::kRows>(l.v, 16 * rt + li, lg, v);
        read_slice<3, Slice::kRows>(l.r, 16 * rt + li, lg, r);
#pragma unroll
        for (int c = 0; c < kNt; ++c) {
          bf16x8 b[3];
          read_slice<3, Slice::kState>(l.s, 16 * (half * kNt + c) + li, lg, b);
          aq[c] = product(o, b, aq[c]);
          ax[c] = product(r, b, ax[c]);
          read_slice<3, Slice::kState>(l.d, 16 * (half * kNt + c) + li, lg, b);
          ak[c] = product(v, b, ak[c]);
        }
      }
      // masked products: rows (inner indices of the next phase) of tile c,
      // columns (lanes) of tiles pt0 and pt1
      if (pm == 0) {                       // M: V_j by dout_i, j <= i
        masked_tiles<3, kNi, Slice::kRows, false>(l.v, l.o, pt0, pt1, li, lg, p0, p1);
      } else if (pm == 1) {                // its transpose: dout_i by V_j, i >= j
        masked_tiles<kNi, 3, Slice::kRows, true>(l.o, l.v, pt0, pt1, li, lg, p0, p1);
      } else if (pm == 2) {                // N: V_j by dR_i
        masked_tiles<3, 3, Slice::kRows, false>(l.v, l.r, pt0, pt1, li, lg, p0, p1);
      } else {                             // its transpose
        masked_tiles<3, 3, Slice::kRows, true>(l.r, l.v, pt0, pt1, li, lg, p0, p1);
      }
      if (kBuffers == 1) __syncthreads();
      buf = kBuffers == 2 ? buf ^ 1 : 0;
      if (more) store(slices[buf]);
      __syncthreads();
    }
    // second phase, with the sums that the loading threads hold (lane indices of
    // its own: its many LDS addresses are then formed here, instead of being held
    // in registers through the first)
    int lane = lane0;
    asm volatile("" : "+v"(lane));
    const int li = lane % 16, lg = lane / 16;
    if (!kOwnKeys) load_keys(A.k, A.ks, key_k);
#pragma unroll
    for (int o = 1; o < kSlicePieces; o *= 2) rv += __shfl_xor(rv, o);
    if (first && piece == 0) srv[row] = rv;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) dot += __shfl_xor(dot, o);
    const bool state = __any((bits << 1) != 0);
    if (lane == 0) {
      sdot[wave] = dot;
      sstate[wave] = state;
    }
    // the masked products' factors, and their way to LDS as left operands
    auto put_masked = [&](uint16_t *dst, const bool transposed, const bool is_n) {
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int ct = side == 0 ? pt0 : pt1, a = 16 * ct + li;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          if (side == 0 ? ks != (transposed ? 1 : 0) : (transposed ? ct >= 2 && ks == 0 : ct < 2 && ks == 1)) continue;
          f32x4 x[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            x[u] = side == 0 ? p0[u] : p1[2 * ks + u];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int b = 16 * (2 * ks + u) + 4 * lg + r, i = transposed ? b : a, j = transposed ? a : b;
              const bool in = is_n ? i > j : i >= j;
              const float d = hw_exp2(static_cast<float>(sg[i] - sg[j]) * kLog2e);
              const float f = is_n ? (transposed ? -sbeta[i] : -1.0f) : A.scale;
              x[u][r] = in ? x[u][r] * d * f : 0.0f;
            }
          }
          const Terms<3> t = split<3>(x[0], x[1]);
          const int block = transposed ? tri_block_t(ct, ks) : tri_block(ct, ks);
#pragma unroll
          for (int y = 0; y < 3; ++y) *reinterpret_cast<bf16x8 *>(dst + y * kTriTerm + (block * 64 + lane) * 8) = t.t[y];
        }
      }
    };
    put_masked(pr.m[pm], pm % 2 == 1, pm >= 2);
    __syncthreads();
    const f32x4 eg = load4(seg + 16 * rt + 4 * lg), w = load4(sw + 16 * rt + 4 * lg),
                be = load4(sbeta + 16 * rt + 4 * lg);
    f32x4 sum_g = zero, sum_b = zero, sum_w = zero;     // over this wave's columns
    f32x4 y[kNt];
#pragma unroll
    for (int c = 0; c < kNt; ++c) {
      aq[c] = aq[c] * eg * A.scale;
      y[c] = zero;
    }
    // with K: M K, N K, (beta N)^T K
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (rt < 2 && ks == 1) continue;
      bf16x8 m[3], nn[3];
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        m[t] = read8(pr.m[0] + t * kTriTerm + (tri_block(rt, ks) * 64 + lane) * 8);
        nn[t] = read8(pr.m[2] + t * kTriTerm + (tri_block(rt, ks) * 64 + lane) * 8);
      }
#pragma unroll
      for (int c = 0; c < kNt; ++c) {
        bf16x8 b[kNi];
        read_right<kNi, DK>(key_k, ks, half * kNt + c, li, lg, b);
        aq[c] = product(m, b, aq[c]);
        y[c] = product(nn, b, y[c]);
      }
    }
    f32x4 kr[kNt];
#pragma unroll
    for (int c = 0; c < kNt; ++c) {
      kr[c] = tile_values<kNi, DK>(key_k, 16 * rt + 4 * lg, half * kNt + c, li);
      ak[c] *= w;
      sum_w += ak[c] * kr[c];
      y[c] -= ax[c] * eg;
      sum_b += kr[c] * y[c];
      sum_g += kr[c] * y[c] * be;
      dk[c] += y[c] * be;
      dq[c] += aq[c];
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (rt >= 2 && ks == 0) continue;
      bf16x8 nn[3];
#pragma unroll
      for (int t = 0; t < 3; ++t) nn[t] = read8(pr.m[3] + t * kTriTerm + (tri_block_t(rt, ks) * 64 + lane) * 8);
#pragma unroll
      for (int c = 0; c < kNt; ++c) {
        bf16x8 b[kNi];
        read_right<kNi, DK>(key_k, ks, half * kNt + c, li, lg, b);
        ak[c] = product(nn, b, ak[c]);
      }
    }
    // with Q: M^T Q
    if (!kOwnKeys) {
      __syncthreads();
      load_keys(A.q, A.qs, key_q);
      __syncthreads();
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (rt >= 2 && ks == 0) continue;
      bf16x8 m[3];
#pragma unroll
      for (int t = 0; t < 3; ++t) m[t] = read8(pr.m[1] + t * kTriTerm + (tri_block_t(rt, ks) * 64 + lane) * 8);
#pragma unroll
      for (int c = 0; c < kNt; ++c) {
        bf16x8 b[kNi];
        read_right<kNi, DK>(key_q, ks, half * kNt + c, li, lg, b);
        ak[c] = product(m, b, ak[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < kNt; ++c) {
      const f32x4 qr = tile_values<kNi, DK>(key_q, 16 * rt + 4 * lg, half * kNt + c, li);
      sum_g += qr * aq[c] - kr[c] * ak[c];
      dk[c] += ak[c];
    }
    if (e + 1 < group) {
      load_gates(h + 1);
      load(h + 1, 0);
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
      bool any = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) any = any || sstate[i];
      if (any) {
        for (int o = 1; o < 64; o *= 2) {
          const float z = __shfl_down(x, o);
          if (lane + o < 64) x += z;
        }
      } else {
        for (int o = 1; o < 64; o *= 2) {
          const float z = __shfl_up(x, o);
          if (lane >= o) x += z;
        }
        x = __shfl_up(x, 1);
        x = lane == 0 ? 0.0f : -x;
      }
      if (lane < n) {
        const int64_t i = token_of(A, q, c0, lane) * A.hv + h;
        A.dg[i] = sgate[lane] < kMinLogDecay ? 0.0f : x;
        A.dbeta[i] = srv[lane] + sbet[0][lane] + sbet[1][lane];
      }
    }
  }
  const int64_t ks = static_cast<int64_t>(A.hk) * A.dk;
  const Rsrc oq = buffer(static_cast<T *>(A.dq) + win.low * ks + static_cast<int64_t>(kh) * A.dk);
  const Rsrc ok = buffer(static_cast<T *>(A.dkey) + win.low * ks + static_cast<int64_t>(kh) * A.dk);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = 16 * rt + 4 * lg + r;
    const uint32_t at = i < n ? win.at(A, i, ks * sizeof(T)) : kNowhere;
#pragma unroll
    for (int c = 0; c < kNt; ++c) {
      const int col = 16 * (half * kNt + c) + li;
      const uint32_t o = col < A.dk ? at + col * sizeof(T) : kNowhere;
      if constexpr (kNi == 1) {
        const uint32_t y = pack2(dq[c][r], dk[c][r]);
        bstore(oq, o, static_cast<bf16_t>(y));
        bstore(ok, o, static_cast<bf16_t>(y >> 16));
      } else {
        bstore(oq, o, dq[c][r]);
        bstore(ok, o, dk[c][r]);
      }
    }
  }
}

template <typename T, int DK>
hipError_t launch(const DeltaArgs &a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(a.slots), a.hk);
  if (delta_vec(a, sizeof(T)) && delta_vec_values(a, a.v, a.vs, sizeof(T), 16) && a.dv % 8 == 0 &&
      delta_vec_values(a, a.dout, static_cast<int64_t>(a.hv) * a.dv, sizeof(T), 16))
    hipLaunchKernelGGL((delta_grad_kernel<T, DK, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((delta_grad_kernel<T, DK, false>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grad(const DeltaArgs &a, bool bf16, hipStream_t s) {
  if (a.dk <= 64) return bf16 ? launch<bf16_t, 64>(a, s) : launch<float, 64>(a, s);
  return bf16 ? launch<bf16_t, 128>(a, s) : launch<float, 128>(a, s);
}

}  // namespace vmk
