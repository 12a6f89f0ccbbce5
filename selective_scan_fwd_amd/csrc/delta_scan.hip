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
// registers (a result tile is, split into terms, the next product's right
// operand) and waves share only the chunk's left operands in LDS.
//
// Rows of the state are held so that K's rows are read in whole pieces: row
// 4 lg + r of tile 2 ks + p is state row 32 ks + 8 lg + 4 p + r.
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kCols = 16 * kWaves;         // state columns of a workgroup

__device__ __forceinline__ int state_row(int d, int lg, int r) { return 32 * (d / 2) + 8 * lg + 4 * (d & 1) + r; }

// A chunk's operands in LDS: K and Q in terms, the triangles' blocks, decays.
template <typename T, int DK, int TRI, bool WITH_Q>
struct ChunkLds {
  static constexpr int kTerm = kC * DK;
  __attribute__((aligned(16))) uint16_t k[kInputTerms<T> * kTerm];
  __attribute__((aligned(16))) uint16_t q[WITH_Q ? kInputTerms<T> * kTerm : 8];
  __attribute__((aligned(16))) uint16_t tri[TRI * kTriTerm];
  __attribute__((aligned(16))) uint16_t v[sizeof(T) == 2 ? kC * kCols : 8];   // (the workgroup's columns)
  __attribute__((aligned(16))) float eg[kC], ew[kC], beta[kC];
};

// Their way there, a chunk ahead of their use.  bf16 rows in whole pieces go
// from global memory to LDS directly into the other of two buffers (DIRECT);
// else they pass through registers, where fp32 is split into terms.
// `v` stands for v or dout: token rows of dv values, of which a workgroup takes
// kCols columns.  Byte offsets from a chunk's lowest token are the same for all
// whole chunks and kept in registers.
template <typename T, int DK, int TRI, int TERMS1, bool WITH_Q, bool VEC, bool DIRECT>
struct ChunkLoad {
  typedef ChunkLds<T, DK, TRI, WITH_Q> Lds;
  static constexpr int kPieces = DK / 8, kPer = kC * kPieces / kThreads;
  static constexpr int kTri = (TRI * kTriBlocks + kWaves - 1) / kWaves;
  Piece<T> k[DIRECT ? 1 : kPer], q[!DIRECT && WITH_Q ? kPer : 1];
  u32x4 tri[DIRECT ? 1 : kTri];
  float eg, ew, beta;
  T v[DIRECT ? 1 : 4][4];
  uint32_t ok[kPer], oq[WITH_Q ? kPer : 1], ov[DIRECT ? 8 : 16], ob;
  int n = -1;                               // steps that the offsets are for
  int wave, lane, li, lg, col0, kh, h;
  bool v16;                                 // DIRECT: v in pieces of 16 bytes, else of 4
  const T *vbase;
  int64_t vstride;

  __device__ __forceinline__ void init(const DeltaArgs &A, int h_, int cb, const T *vb, int64_t vs) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    lane = threadIdx.x % 64;
    li = lane % 16;
    lg = lane / 16;
    col0 = cb * kCols;
    h = h_;
    kh = h / (A.hv / A.hk);
    vbase = vb + static_cast<int64_t>(h) * A.dv;
    vstride = vs;
    v16 = (A.dv & 7) == 0 && (vs & 7) == 0 && (reinterpret_cast<uintptr_t>(vb) & 15) == 0;
  }

  __device__ __forceinline__ void plan(const DeltaArgs &A, const Window &w) {
    n = w.n;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = (i * kWaves + wave) * 64 + lane, row = x / kPieces;
      // (place x holds piece `place ^ row` of its row; see swizzled())
      const int p = DIRECT ? (x % kPieces) ^ (row & (kPieces - 1)) : x % kPieces;
      const bool in = row < n && 8 * p < A.dk;
      ok[i] = in ? w.at(A, row, A.ks * sizeof(T)) + 8 * p * sizeof(T) : kNowhere;
      if (WITH_Q) oq[i] = in ? w.at(A, row, A.qs * sizeof(T)) + 8 * p * sizeof(T) : kNowhere;
    }
    ob = lane < n ? w.at(A, lane, A.hv * 4) : kNowhere;
    if constexpr (DIRECT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // 16 bytes: 8 rows of 8 pieces an instruction, 2 of them; 4 bytes: 2 rows of 32
        const int row = v16 ? (i * kWaves + wave) * 8 + lane / 8 : (i * kWaves + wave) * 2 + lane / 32;
        const int c = col0 + (v16 ? 8 * (lane % 8) : 2 * (lane % 32));
        ov[i] = row < n && c < A.dv ? w.at(A, row, vstride * sizeof(T)) + c * sizeof(T) : kNowhere;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = 16 * (i / 4) + 4 * lg + i % 4, c = col0 + 16 * wave + li;
        ov[i] = row < n && c < A.dv ? w.at(A, row, vstride * sizeof(T)) + c * sizeof(T) : kNowhere;
      }
    }
  }

  // m1 (TERMS1 of the TRI terms) and m2: the triangular operands.
  __device__ __forceinline__ void load(const DeltaArgs &A, const Seq &s, int64_t c0, const uint16_t *m1,
                                       const uint16_t *m2, Lds &l) {
    const Window w = window(A, s, c0);
    if (w.n != n) plan(A, w);
    const int64_t at = (s.slot0 + c0 / kC) * A.hv + h;
    const Rsrc rk = buffer(static_cast<const T *>(A.k) + w.low * A.ks + static_cast<int64_t>(kh) * A.dk);
    const Rsrc rq = buffer(static_cast<const T *>(A.q) + w.low * A.qs + static_cast<int64_t>(kh) * A.dk);
    const Rsrc r1 = buffer(m1 + at * TERMS1 * kTriTerm), r2 = buffer(m2 + at * (TRI - TERMS1) * kTriTerm);
    const Rsrc reg = buffer(A.eg + at * kC), rew = buffer(A.ew + at * kC), rbeta = buffer(A.beta + w.low * A.hv + h);
    const Rsrc rv = buffer(vbase + w.low * vstride);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (DIRECT) {
        to_lds16(rk, l.k + (i * kWaves + wave) * 512, ok[i]);
        if (WITH_Q) to_lds16(rq, l.q + (i * kWaves + wave) * 512, oq[i]);
      } else {
        const int c = 8 * (((i * kWaves + wave) * 64 + lane) % kPieces);
        k[i] = load_piece<VEC>(rk, ok[i], c, A.dk, T());
        if (WITH_Q) q[i] = load_piece<VEC>(rq, oq[i], c, A.dk, T());
      }
    }
#pragma unroll
    for (int i = 0; i < kTri; ++i) {
      const int b = wave + i * kWaves, t1 = TERMS1 * kTriBlocks;
      const uint32_t off = (b < t1 ? b : b - t1) * 1024 + lane * 16;
      if constexpr (DIRECT) {
        if (b < TRI * kTriBlocks) to_lds16(b < t1 ? r1 : r2, l.tri + b * 512, off);
      } else {
        tri[i] = bload16(b < t1 ? r1 : r2, b < TRI * kTriBlocks ? off : kNowhere);
      }
    }
    if constexpr (DIRECT) {
      if (wave == 0) to_lds4(reg, l.eg, lane * 4);
      if (wave == 1) to_lds4(rew, l.ew, lane * 4);
      if (wave == 2) to_lds4(rbeta, l.beta, ob);
      if (v16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) to_lds16(rv, l.v + (i * kWaves + wave) * 512, ov[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) to_lds4(rv, l.v + (i * kWaves + wave) * 128, ov[i]);
      }
    } else {
      eg = bload<float>(reg, lane * 4);
      ew = bload<float>(rew, lane * 4);
      beta = bload<float>(rbeta, ob);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i / 4][i % 4] = bload<T>(rv, ov[i]);
    }
  }

  __device__ __forceinline__ void store(Lds &l) const {
    if constexpr (DIRECT) {
      wait_loads();
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = (i * kWaves + wave) * 64 + lane, row = x / kPieces, p = x % kPieces;
        store_piece<DK>(l.k, Lds::kTerm, row, p, k[i]);
        if (WITH_Q) store_piece<DK>(l.q, Lds::kTerm, row, p, q[i]);
      }
#pragma unroll
      for (int i = 0; i < kTri; ++i) {
        const int b = wave + i * kWaves;
        if (b < TRI * kTriBlocks) *reinterpret_cast<u32x4 *>(l.tri + b * 512 + lane * 8) = tri[i];
      }
      if (wave == 0) {
        l.eg[lane] = eg;
        l.ew[lane] = ew;
        l.beta[lane] = beta;
      }
    }
  }

  // The wave's 64 x 16 of v, as D tiles.  From registers they are taken as soon
  // as they have come, from LDS with the chunk.
  __device__ __forceinline__ void values(const Lds &l, f32x4 (&x)[4]) const {
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      if constexpr (DIRECT) {
        const uint16_t *p = l.v + (16 * rt + 4 * lg + li / 4) * kCols + 16 * wave + 4 * (li % 4);
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4 *)const_cast<uint16_t *>(p));
#pragma unroll
        for (int r = 0; r < 4; ++r) x[rt][r] = to_f32(static_cast<bf16_t>(y[r]));
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) x[rt][r] = to_f32(v[rt][r]);
      }
    }
  }
};

// Byte offsets of a wave's D tiles in token rows of `stride` values.
struct RowOffsets {
  uint32_t at[16];
  int n = -1;
  __device__ __forceinline__ void plan(const DeltaArgs &A, const Window &w, int64_t stride_bytes, int esize, int lg,
                                       int col) {
    if (w.n == n) return;
    n = w.n;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = 16 * (i / 4) + 4 * lg + i % 4;
      at[i] = row < n && col < A.dv ? w.at(A, row, stride_bytes) + col * esize : kNowhere;
    }
  }
};
__device__ __forceinline__ void store_tokens(bf16_t *base, const RowOffsets &o, const f32x4 (&x)[4]) {
  const Rsrc r = buffer(base);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const uint32_t y = pack2(x[i / 4][i % 4], x[i / 4][i % 4 + 1]);
    bstore(r, o.at[i], static_cast<bf16_t>(y));
    bstore(r, o.at[i + 1], static_cast<bf16_t>(y >> 16));
  }
}
__device__ __forceinline__ void store_tokens(float *base, const RowOffsets &o, const f32x4 (&x)[4]) {
  const Rsrc r = buffer(base);
#pragma unroll
  for (int i = 0; i < 16; ++i) bstore(r, o.at[i], x[i / 4][i % 4]);
}

// x[rt] += rows (tiles rt) of m times b, over all columns of m (whole rows).
template <int DK, int NA, int NB>
__device__ __forceinline__ void rows_times(const uint16_t *m, const Terms<NB> (&b)[DK / 32], int li, int lg,
                                           f32x4 (&x)[4]) {
#pragma unroll
  for (int ks = 0; ks < DK / 32; ++ks) {
    bf16x8 a[4][NA];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int t = 0; t < NA; ++t) a[rt][t] = read8(m + t * kC * DK + swizzled<DK>(16 * rt + li, 4 * ks + lg));
#pragma unroll
    for (int t = 0; t < NA; ++t)
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        if (t + u >= (NA > NB ? NA : NB)) continue;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) x[rt] = mfma32(a[rt][t], b[ks].t[u], x[rt]);
      }
  }
}

// The columns (state rows) of one term of m as left operands, over the 64 rows of
// m.  Where the next chunk is on its way to LDS they are read before it is sent
// for: the compiler lets no transposing read pass a load to LDS without waiting
// for that load.
template <int DK>
struct Columns {
  bf16x8 a[2][DK / 16];
  __device__ __forceinline__ void read(const uint16_t *m, int li, int lg) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int d = 0; d < DK / 16; ++d)
        a[kt][d] = join(read_columns<DK>(m, 32 * kt + 4 * lg, d / 2, d & 1, li),
                        read_columns<DK>(m, 32 * kt + 16 + 4 * lg, d / 2, d & 1, li));
  }
};

// x[d] += columns (state rows of tile d) of m times b.  first: m's first term.
template <int DK, int NA, int NB>
__device__ __forceinline__ void columns_times(const Columns<DK> &first, const uint16_t *m, const Terms<NB> (&b)[2], int li,
                                              int lg, f32x4 (&x)[DK / 16]) {
#pragma unroll
  for (int t = 0; t < NA; ++t) {
    Columns<DK> c = first;
    if (t > 0) c.read(m + t * kC * DK, li, lg);
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        if (t + u >= (NA > NB ? NA : NB)) continue;
#pragma unroll
        for (int d = 0; d < DK / 16; ++d) x[d] = mfma32(c.a[kt][d], b[kt].t[u], x[d]);
      }
  }
}

// x[rt] += row tiles of a triangular operand (TR: of its transpose) times b.
template <int NA, int NB, bool TR>
__device__ __forceinline__ void triangle_times(const uint16_t *m, const Terms<NB> (&b)[2], int lane, f32x4 (&x)[4]) {
  constexpr int kMost = NA > NB ? NA : NB;
#pragma unroll
  for (int t = 0; t < NA; ++t)
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      if (t + u >= kMost) continue;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          if (TR ? (rt >= 2 && ks == 0) : (rt < 2 && ks == 1)) continue;
          const int block = TR ? tri_block_t(rt, ks) : tri_block(rt, ks);
          x[rt] = mfma32(read8(m + t * kTriTerm + (block * 64 + lane) * 8), b[ks].t[u], x[rt]);
        }
    }
}

template <int N>
__device__ __forceinline__ void split_rows(const f32x4 (&x)[4], Terms<N> (&t)[2]) {
  t[0] = split<N>(x[0], x[1]);
  t[1] = split<N>(x[2], x[3]);
}

// Workgroups of one sequence and head (which share K, Q and the triangles) are
// neighbours on one XCD.
struct Place {
  int s, h, cb;
};
__device__ __forceinline__ Place place(const DeltaArgs &A, int colblocks) {
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  Place p;
  p.cb = id % colblocks;
  const int sh = id / colblocks;
  p.h = sh % A.hv;
  p.s = sh / A.hv;
  return p;
}

// D tiles [DK][16] at [dk][cols] memory, and [64][16] at [64][dvp]; columns past
// them go nowhere.
template <int DK>
__device__ __forceinline__ void store_state(const DeltaArgs &A, float *base, int cols, const f32x4 (&S)[DK / 16], int lg, int col) {
  // (rows past dk lie past the resource's end)
  const Rsrc r = buffer(base, A.dk * cols * 4);
  const uint32_t first = col < cols ? (8 * lg * cols + col) * 4 : kNowhere;
#pragma unroll
  for (int d = 0; d < DK / 16; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) bstore(r, first + state_row(d, 0, e) * cols * 4, S[d][e]);
}
template <int DK>
__device__ __forceinline__ void load_state(const DeltaArgs &A, const float *base, f32x4 (&S)[DK / 16], int lg, int col) {
  const Rsrc r = buffer(base);
#pragma unroll
  for (int d = 0; d < DK / 16; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = state_row(d, lg, e);
      S[d][e] = bload<float>(r, base != nullptr && row < A.dk && col < A.dv ? (row * A.dv + col) * 4 : kNowhere);
    }
}
__device__ __forceinline__ void store_rows(const DeltaArgs &A, float *base, const f32x4 (&x)[4], int lg, int col) {
  const Rsrc r = buffer(base);
  const uint32_t first = col < A.dvp ? (4 * lg * A.dvp + col) * 4 : kNowhere;
#pragma unroll
  for (int rt = 0; rt < 4; ++rt)
#pragma unroll
    for (int e = 0; e < 4; ++e) bstore(r, first + (16 * rt + e) * A.dvp * 4, x[rt][e]);
}
template <typename T> constexpr bool kDirect = sizeof(T) == 2;

// Forward.  KEEP: S and V are stored for the backward pass, out and state not.
template <typename T, int DK, bool KEEP, bool VEC>
__global__ __launch_bounds__(kThreads) void delta_scan_kernel(DeltaArgs A, int colblocks) {
  constexpr int kNi = kInputTerms<T>, kNs = 3;
  constexpr int kTermsP = KEEP ? 0 : kNi == 1 ? 2 : 3;
  constexpr int kNo = kNi == 1 ? 2 : 3;               // terms of S and V on their way to out only
  constexpr bool kDma = VEC && kDirect<T>;
  typedef ChunkLoad<T, DK, kTermsT + kTermsP, kTermsT, !KEEP, VEC, kDma> Load;
  typedef typename Load::Lds Lds;
  constexpr int kBuffers = kDma ? 2 : 1;
  __shared__ Lds lds[kBuffers];
  const Place pl = place(A, colblocks);
  const int s = pl.s, h = pl.h, kh = h / (A.hv / A.hk);
  const Seq q = sequence(A, s);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16,
            lg = lane / 16;
  const int col = (pl.cb * kWaves + wave) * 16 + li;
  const int64_t state_at = (static_cast<int64_t>(s) * A.hv + h) * A.dk * A.dv;
  f32x4 S[DK / 16];
  load_state<DK>(A, A.h0 != nullptr ? A.h0 + state_at : nullptr, S, lg, col);
  Load next;
  next.init(A, h, pl.cb, static_cast<const T *>(A.v), A.vs);
  RowOffsets rows;
  if (q.len > 0) {
    next.load(A, q, 0, A.T, A.P, lds[0]);
    next.store(lds[0]);
  }
  __syncthreads();
  int buf = 0;
  for (int64_t c0 = 0; c0 < q.len; c0 += kC) {
    const Window w = window(A, q, c0);
    const int64_t at = (q.slot0 + c0 / kC) * A.hv + h;
    const Lds &l = lds[buf];
    f32x4 v[4];
    next.values(l, v);
    Columns<DK> kc;
    if (kDma) kc.read(l.k, li, lg);
    const bool more = c0 + kC < q.len;
    if (more) next.load(A, q, c0 + kC, A.T, A.P, lds[kBuffers == 2 ? buf ^ 1 : 0]);
    Terms<kNs> st[DK / 32];
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) st[ks] = split<kNs>(S[2 * ks], S[2 * ks + 1]);
    if (KEEP) store_state<DK>(A, A.S + at * A.dk * A.dvp, A.dvp, S, lg, col);
    f32x4 x[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) x[rt] = f32x4{0, 0, 0, 0};
    rows_times<DK, kNi, kNs>(l.k, st, li, lg, x);
    f32x4 o[4];
    if (!KEEP) {
      Terms<kNo> so[DK / 32];
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks)
#pragma unroll
        for (int t = 0; t < kNo; ++t) so[ks].t[t] = st[ks].t[t];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) o[rt] = f32x4{0, 0, 0, 0};
      rows_times<DK, kNi, kNo>(l.q, so, li, lg, o);
    }
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const f32x4 eg = load4(l.eg + 16 * rt + 4 * lg), b = load4(l.beta + 16 * rt + 4 * lg);
      x[rt] = b * (v[rt] - eg * x[rt]);
      if (!KEEP) o[rt] = o[rt] * eg * A.scale;
    }
    Terms<kNs> r3[2];
    split_rows<kNs>(x, r3);
    f32x4 V[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) V[rt] = f32x4{0, 0, 0, 0};
    triangle_times<kTermsT, kNs, false>(l.tri, r3, lane, V);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) x[rt] = V[rt] * load4(l.ew + 16 * rt + 4 * lg);
    split_rows<kNs>(x, r3);
    const float last = l.eg[kC - 1];
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) S[d] *= last;
    if (!kDma) kc.read(l.k, li, lg);
    columns_times<DK, kNi, kNs>(kc, l.k, r3, li, lg, S);
    if constexpr (!KEEP) {
      Terms<kNo> vo[2];
      split_rows<kNo>(V, vo);
      triangle_times<kTermsP, kNo, false>(l.tri + kTermsT * kTriTerm, vo, lane, o);
    }
    if (kBuffers == 1) __syncthreads();
    buf = kBuffers == 2 ? buf ^ 1 : 0;
    if (more) next.store(lds[buf]);
    // (stores come after the wait for the next chunk's loads, which would
    // otherwise wait for them too)
    if constexpr (!KEEP) {
      rows.plan(A, w, static_cast<int64_t>(A.hv) * A.dv * sizeof(T), sizeof(T), lg, col);
      store_tokens(static_cast<T *>(A.out) + (w.low * A.hv + h) * A.dv, rows, o);
    } else {
      store_rows(A, A.V + at * kC * A.dvp, V, lg, col);
    }
    __syncthreads();
  }
  if (!KEEP && A.state != nullptr) store_state<DK>(A, A.state + state_at, A.dv, S, lg, col);
}

template <typename T, int DK, bool VEC>
__global__ __launch_bounds__(kThreads) void delta_scan_bwd_kernel(DeltaArgs A, int colblocks) {
  constexpr int kNi = kInputTerms<T>, kNs = 3;
  constexpr int kTermsP = kNi == 1 ? 2 : 3;
  constexpr bool kDma = VEC && kDirect<T>;
  typedef ChunkLoad<T, DK, kTermsT + kTermsP, kTermsT, true, VEC, kDma> Load;
  typedef typename Load::Lds Lds;
  constexpr int kBuffers = kDma ? 2 : 1;
  __shared__ Lds lds[kBuffers];
  const Place pl = place(A, colblocks);
  const int s = pl.s, h = pl.h, kh = h / (A.hv / A.hk);
  const Seq q = sequence(A, s);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, li = lane % 16,
            lg = lane / 16;
  const int col = (pl.cb * kWaves + wave) * 16 + li;
  const int64_t state_at = (static_cast<int64_t>(s) * A.hv + h) * A.dk * A.dv;
  const int64_t row = static_cast<int64_t>(A.hv) * A.dv;      // token stride of dout and dv
  f32x4 D[DK / 16];
  load_state<DK>(A, A.dstate != nullptr ? A.dstate + state_at : nullptr, D, lg, col);
  Load next;
  next.init(A, h, pl.cb, static_cast<const T *>(A.dout), row);
  RowOffsets rows;
  const int64_t first = (static_cast<int64_t>(q.len + kC - 1) / kC - 1) * kC;
  if (q.len > 0) {
    next.load(A, q, first, A.TT, A.PT, lds[0]);
    next.store(lds[0]);
  }
  __syncthreads();
  int buf = 0;
  for (int64_t c0 = first; c0 >= 0; c0 -= kC) {
    const Window w = window(A, q, c0);
    const int64_t at = (q.slot0 + c0 / kC) * A.hv + h;
    const Lds &l = lds[buf];
    f32x4 o[4];
    next.values(l, o);
    Columns<DK> kc, qc;
    if (kDma) {
      kc.read(l.k, li, lg);
      qc.read(l.q, li, lg);
    }
    if (c0 > 0) next.load(A, q, c0 - kC, A.TT, A.PT, lds[kBuffers == 2 ? buf ^ 1 : 0]);
    store_state<DK>(A, A.dS + at * A.dk * A.dvp, A.dvp, D, lg, col);
    f32x4 V[4], R[4];
    {
      Terms<kNs> st[DK / 32];
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) st[ks] = split<kNs>(D[2 * ks], D[2 * ks + 1]);
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) V[rt] = f32x4{0, 0, 0, 0};
      rows_times<DK, kNi, kNs>(l.k, st, li, lg, V);
    }
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) V[rt] = V[rt] * load4(l.ew + 16 * rt + 4 * lg);
    {
      Terms<kNi> ot[2];
      split_rows<kNi>(o, ot);
      triangle_times<kTermsP, kNi, true>(l.tri + kTermsT * kTriTerm, ot, lane, V);
    }
    Terms<kNs> t3[2];
    split_rows<kNs>(V, t3);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) R[rt] = f32x4{0, 0, 0, 0};
    triangle_times<kTermsT, kNs, true>(l.tri, t3, lane, R);
    const float last = l.eg[kC - 1];
    f32x4 dv[4], x[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const f32x4 eg = load4(l.eg + 16 * rt + 4 * lg);
      dv[rt] = R[rt] * load4(l.beta + 16 * rt + 4 * lg);
      x[rt] = f32x4{0, 0, 0, 0} - dv[rt] * eg;
      o[rt] = o[rt] * eg * A.scale;
    }
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) D[d] *= last;
    split_rows<kNs>(x, t3);
    if (!kDma) kc.read(l.k, li, lg);
    columns_times<DK, kNi, kNs>(kc, l.k, t3, li, lg, D);
    split_rows<kNs>(o, t3);
    if (!kDma) qc.read(l.q, li, lg);
    columns_times<DK, kNi, kNs>(qc, l.q, t3, li, lg, D);
    if (kBuffers == 1) __syncthreads();
    buf = kBuffers == 2 ? buf ^ 1 : 0;
    if (c0 > 0) next.store(lds[buf]);
    store_rows(A, A.dR + at * kC * A.dvp, R, lg, col);
    rows.plan(A, w, row * sizeof(T), sizeof(T), lg, col);
    store_tokens(static_cast<T *>(A.dval) + (w.low * A.hv + h) * A.dv, rows, dv);
    __syncthreads();
  }
  if (A.dh0 != nullptr) store_state<DK>(A, A.dh0 + state_at, A.dv, D, lg, col);
}

int column_blocks(const DeltaArgs &a) { return (a.dv + 16 * kWaves - 1) / (16 * kWaves); }

template <typename T, int DK, bool VEC>
hipError_t launch_fwd(const DeltaArgs &a, bool keep, hipStream_t s) {
  const int cb = column_blocks(a);
  const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(a.nseq) * a.hv * cb));
  if (keep)
    hipLaunchKernelGGL((delta_scan_kernel<T, DK, true, VEC>), grid, dim3(kThreads), 0, s, a, cb);
  else
    hipLaunchKernelGGL((delta_scan_kernel<T, DK, false, VEC>), grid, dim3(kThreads), 0, s, a, cb);
  return hipGetLastError();
}
template <typename T, int DK>
hipError_t launch_fwd(const DeltaArgs &a, bool keep, hipStream_t s) {
  return delta_vec(a, sizeof(T)) && delta_vec_values(a, a.v, a.vs, sizeof(T), 4)
             ? launch_fwd<T, DK, true>(a, keep, s) : launch_fwd<T, DK, false>(a, keep, s);
}
template <typename T, int DK>
hipError_t launch_bwd(const DeltaArgs &a, hipStream_t s) {
  const int cb = column_blocks(a);
  const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(a.nseq) * a.hv * cb));
  if (delta_vec(a, sizeof(T)) && delta_vec_values(a, a.dout, static_cast<int64_t>(a.hv) * a.dv, sizeof(T), 4))
    hipLaunchKernelGGL((delta_scan_bwd_kernel<T, DK, true>), grid, dim3(kThreads), 0, s, a, cb);
  else
    hipLaunchKernelGGL((delta_scan_bwd_kernel<T, DK, false>), grid, dim3(kThreads), 0, s, a, cb);
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
