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

// A pair of waves owns 16 columns of the state: every product of the chunk stays
// within those columns, so the chain of products passes from registers to
// registers (a result tile is, split into terms, the next product's right
// operand) and workgroup-wide only the chunk's left operands are shared.  Wave
// p of the pair holds half p of the state's rows and of the chunk's steps: it
// forms half of the sum of K S over the state's rows, for all steps, and the
// halves meet through LDS, as do the parts of the triangular products and the
// corrected values.  The chain of a chunk is what bounds a long sequence; a wave
// issues about one instruction in five cycles however idle the rest of its SIMD
// is, so halving the instructions of the chain is worth three exchanges: 4 x 4097
// tokens, 16 value heads of 128, bf16, 65 chunks, took 211 us where one wave to 16
// columns took 281, and 183 with waves of their own for the loads, see
// load_chunks(); with nothing loaded after the first chunk 163.  Those were with
// two terms of what enters the output only; with all three it takes 203 (3.1 us a
// chunk).  (128 x 197 tokens, 6 heads of 64, fp32: 83 us; 40 packed sequences of
// up to 1500 tokens, 8 value heads of 100: 86 us, of two terms 77, and 84 in the
// order given and in runs over the XCDs.)
//
// Rows of the state are held so that K's rows are read in whole pieces: row
// 4 lg + r of tile 2 ks + p is state row 32 ks + 8 lg + 4 p + r.
__device__ __forceinline__ int state_row(int d, int lg, int r) { return 32 * (d / 2) + 8 * lg + 4 * (d & 1) + r; }

// NP pairs of waves, 16 NP columns, to a workgroup.
template <int NP>
struct Shape {
  static constexpr int kWaves = 2 * NP, kThreads = 64 * kWaves, kCols = 16 * NP;
};

// A chunk's operands in LDS: K and Q in terms, the triangles' blocks, decays.
template <typename T, int DK, int TRI, bool WITH_Q>
struct ChunkLds {
  static constexpr int kTerm = kC * DK;
  __attribute__((aligned(16))) uint16_t k[kInputTerms<T> * kTerm];
  __attribute__((aligned(16))) uint16_t q[WITH_Q ? kInputTerms<T> * kTerm : 8];
  __attribute__((aligned(16))) uint16_t tri[TRI * kTriTerm];
  __attribute__((aligned(16))) float eg[kC], ew[kC], beta[kC];
};

// Their way there, a chunk ahead of their use.  bf16 rows in whole pieces go
// from global memory to LDS directly into the other of two buffers (DIRECT);
// else they pass through registers, where fp32 is split into terms.
// `v` stands for v or dout: token rows of dv values, of which a workgroup takes
// kCols columns.  Byte offsets from a chunk's lowest token are the same for all
// whole chunks and kept in registers.
template <typename T, int DK, int TRI, bool WITH_Q, bool VEC, bool DIRECT, int NP>
struct ChunkLoad {
  typedef ChunkLds<T, DK, TRI, WITH_Q> Lds;
  static constexpr int kWaves = Shape<NP>::kWaves, kThreads = Shape<NP>::kThreads, kCols = Shape<NP>::kCols;
  static constexpr int kPieces = DK / 8, kPer = kC * kPieces / kThreads;
  // v to LDS: rows of an instruction with 16 or 4 bytes a lane, and instructions of a wave
  static constexpr int kRows16 = 512 / kCols, kRows4 = 128 / kCols;
  static constexpr int kV16 = kC / kRows16 / kWaves, kV4 = kC / kRows4 / kWaves;
  static constexpr int kValues = DIRECT ? kC * kCols : 8;   // (the workgroup's columns)
  // triangular operands in memory: blocks of whole terms, or of fp32 matrices
  static constexpr bool kWhole = sizeof(T) == 4;
  static constexpr int kBlocks = (kWhole ? TRI / 3 : TRI) * kTriBlocks, kBlockBytes = kWhole ? 2048 : 1024;
  static constexpr int kTri = (kBlocks + kWaves - 1) / kWaves;
  Piece<T> k[DIRECT ? 1 : kPer], q[!DIRECT && WITH_Q ? kPer : 1];
  u32x4 tri[DIRECT ? 1 : kTri][kWhole ? 2 : 1];
  float eg, ew, beta;
  T v[DIRECT ? 1 : 4][4];
  uint32_t ok[kPer], oq[WITH_Q ? kPer : 1], ov[DIRECT ? kV4 : 16], ob;
  int n = -1;                               // steps that the offsets are for
  int wave, lane, li, lg, col0, kh, h;      // (wave 2 i + p: pair i, half p)
  bool v16;                                 // DIRECT: v in pieces of 16 bytes, else of 4
  const T *vbase;
  int64_t vstride;
  int64_t low, at;                          // of the chunk aimed at: lowest token, (slot, head)

  __device__ __forceinline__ void init(const DeltaArgs &A, int h_, int cb, const T *vb, int64_t vs) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64) % kWaves;
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
      for (int i = 0; i < kV4; ++i) {
        const int per16 = kCols / 8, per4 = kCols / 2;
        const int row = v16 ? (i * kWaves + wave) * kRows16 + lane / per16 : (i * kWaves + wave) * kRows4 + lane / per4;
        const int c = col0 + (v16 ? 8 * (lane % per16) : 2 * (lane % per4));
        ov[i] = row < n && c < A.dv ? w.at(A, row, vstride * sizeof(T)) + c * sizeof(T) : kNowhere;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = 16 * (i / 4) + 4 * lg + i % 4, c = col0 + 16 * (wave / 2) + li;
        ov[i] = row < n && c < A.dv ? w.at(A, row, vstride * sizeof(T)) + c * sizeof(T) : kNowhere;
      }
    }
  }

  // Takes aim at chunk c0, whose parts are then loaded one by one.
  __device__ __forceinline__ void aim(const DeltaArgs &A, const Seq &s, int64_t c0) {
    const Window w = window(A, s, c0);
    if (w.n != n) plan(A, w);
    low = w.low;
    at = (s.slot0 + c0 / kC) * A.hv + h;
  }
  __device__ __forceinline__ void load_v(uint16_t *lv) {
    const Rsrc rv = buffer(vbase + low * vstride);
    if constexpr (DIRECT) {
      if (v16) {
#pragma unroll
        for (int i = 0; i < kV16; ++i) to_lds16(rv, lv + (i * kWaves + wave) * 512, ov[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kV4; ++i) to_lds4(rv, lv + (i * kWaves + wave) * 128, ov[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i / 4][i % 4] = bload<T>(rv, ov[i]);
    }
  }
  __device__ __forceinline__ void load_gates(const DeltaArgs &A, Lds &l) {
    const Rsrc reg = buffer(A.eg + at * kC), rew = buffer(A.ew + at * kC), rbeta = buffer(A.beta + low * A.hv + h);
    if constexpr (DIRECT) {
      if (wave == 0) to_lds4(reg, l.eg, lane * 4);
      if (wave == 1) to_lds4(rew, l.ew, lane * 4);
      if (wave == 2 % kWaves) to_lds4(rbeta, l.beta, ob);
    } else {
      eg = bload<float>(reg, lane * 4);
      ew = bload<float>(rew, lane * 4);
      beta = bload<float>(rbeta, ob);
    }
  }
  __device__ __forceinline__ void load_k(const DeltaArgs &A, Lds &l) {
    const Rsrc rk = buffer(static_cast<const T *>(A.k) + low * A.ks + static_cast<int64_t>(kh) * A.dk);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (DIRECT)
        to_lds16(rk, l.k + (i * kWaves + wave) * 512, ok[i]);
      else
        k[i] = load_piece<VEC>(rk, ok[i], 8 * (((i * kWaves + wave) * 64 + lane) % kPieces), A.dk, T());
    }
  }
  __device__ __forceinline__ void load_q(const DeltaArgs &A, Lds &l) {
    if constexpr (WITH_Q) {
      const Rsrc rq = buffer(static_cast<const T *>(A.q) + low * A.qs + static_cast<int64_t>(kh) * A.dk);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if constexpr (DIRECT)
          to_lds16(rq, l.q + (i * kWaves + wave) * 512, oq[i]);
        else
          q[i] = load_piece<VEC>(rq, oq[i], 8 * (((i * kWaves + wave) * 64 + lane) % kPieces), A.dk, T());
      }
    }
  }
  // the triangular operands of the chunk and head
  __device__ __forceinline__ void load_tri(const uint16_t *m, Lds &l, int from = 0, int to = kTri) {
    const Rsrc r = buffer(m + at * (kBlocks * kBlockBytes / 2), kBlocks * kBlockBytes);
#pragma unroll
    for (int i = 0; i < kTri; ++i) {
      if (i < from || i >= to) continue;
      // (waves with no block left read zeros past the resource's end)
      const int b = wave + i * kWaves;
      if constexpr (DIRECT) {
        if ((i + 1) * kWaves <= kBlocks || b < kBlocks)
          to_lds16(r, l.tri + b * 512, (b * 64 + lane) * 16);
      } else {
#pragma unroll
        for (int j = 0; j < (kWhole ? 2 : 1); ++j)
          tri[i][j] = bload16(r, (b * 64 + lane) * (kBlockBytes / 64) + 16 * j);
      }
    }
  }
  // All but v.
  __device__ __forceinline__ void load(const DeltaArgs &A, const Seq &s, int64_t c0, const uint16_t *m, Lds &l) {
    aim(A, s, c0);
    load_gates(A, l);
    load_k(A, l);
    load_q(A, l);
    load_tri(m, l);
  }
  // Loads that every wave issues for a chunk's K and Q (DIRECT).
  static constexpr int kLeast = kPer * (WITH_Q ? 2 : 1);

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
        if (b >= kBlocks) continue;
        if constexpr (kWhole) {
          const Terms<3> t = split<3>(__builtin_bit_cast(f32x4, tri[i][0]), __builtin_bit_cast(f32x4, tri[i][1]));
          uint16_t *to = l.tri + (b / kTriBlocks * 3 * kTriBlocks + b % kTriBlocks) * 512 + lane * 8;
#pragma unroll
          for (int x = 0; x < 3; ++x) *reinterpret_cast<bf16x8 *>(to + x * kTriTerm) = t.t[x];
        } else {
          *reinterpret_cast<u32x4 *>(l.tri + b * 512 + lane * 8) = tri[i][0];
        }
      }
      if (wave == 0) {
        l.eg[lane] = eg;
        l.ew[lane] = ew;
        l.beta[lane] = beta;
      }
    }
  }

  // Step tile rt of the pair's 16 columns of v, as a D tile.  From registers it is
  // taken as soon as it has come, from LDS with the chunk.
  __device__ __forceinline__ f32x4 values(const uint16_t *lv, int rt) const {
    f32x4 x;
    if constexpr (DIRECT) {
      const uint16_t *p = lv + (16 * rt + 4 * lg + li / 4) * kCols + 16 * (wave / 2) + 4 * (li % 4);
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4 *)const_cast<uint16_t *>(p));
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = to_f32(static_cast<bf16_t>(y[r]));
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = to_f32(rt == 0 ? v[0][r] : rt == 1 ? v[1][r] : rt == 2 ? v[2][r] : v[3][r]);
    }
    return x;
  }
};

// Byte offsets of a wave's two D tiles (its half's steps) in token rows of
// `stride` values.
struct RowOffsets {
  uint32_t at[8];
  int n = -1;
  __device__ __forceinline__ void plan(const DeltaArgs &A, const Window &w, int64_t stride_bytes, int esize, int p,
                                       int lg, int col) {
    if (w.n == n) return;
    n = w.n;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 32 * p + 16 * (i / 4) + 4 * lg + i % 4;
      at[i] = row < n && col < A.dv ? w.at(A, row, stride_bytes) + col * esize : kNowhere;
    }
  }
};
__device__ __forceinline__ void store_tokens(bf16_t *base, const RowOffsets &o, const f32x4 (&x)[2]) {
  const Rsrc r = buffer(base);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t y = pack2(x[i / 4][i % 4], x[i / 4][i % 4 + 1]);
    bstore(r, o.at[i], static_cast<bf16_t>(y));
    bstore(r, o.at[i + 1], static_cast<bf16_t>(y >> 16));
  }
}
__device__ __forceinline__ void store_tokens(float *base, const RowOffsets &o, const f32x4 (&x)[2]) {
  const Rsrc r = buffer(base);
#pragma unroll
  for (int i = 0; i < 8; ++i) bstore(r, o.at[i], x[i / 4][i % 4]);
}

// Left operands in registers.  Where K and Q are single terms they are read
// ahead of the products that use them, before the exchange that those wait for.
//
// Rows of m, all four tiles, the columns of half p; x[rt] += their product with b.
template <int DK, int NA>
struct RowTiles {
  bf16x8 a[DK / 64][4][NA];
  __device__ __forceinline__ void read(const uint16_t *m, int p, int li, int lg) {
#pragma unroll
    for (int ks = 0; ks < DK / 64; ++ks)
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int t = 0; t < NA; ++t)
          a[ks][rt][t] = read8(m + t * kC * DK + swizzled<DK>(16 * rt + li, 4 * (p * (DK / 64) + ks) + lg));
  }
  template <int NB>
  __device__ __forceinline__ void times(const Terms<NB> (&b)[DK / 64], f32x4 (&x)[4]) const {
#pragma unroll
    for (int ks = 0; ks < DK / 64; ++ks)
#pragma unroll
      for (int t = 0; t < NA; ++t)
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          if (t + u >= (NA > NB ? NA : NB)) continue;
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) x[rt] = mfma32(a[ks][rt][t], b[ks].t[u], x[rt]);
        }
  }
};

// Columns (the state rows of half p) of m, one term, over its 64 rows.
template <int DK>
struct ColumnTiles {
  bf16x8 a[2][DK / 32];
  __device__ __forceinline__ void read(const uint16_t *m, int p, int li, int lg) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int d = 0; d < DK / 32; ++d)
        a[kt][d] = join(read_columns<DK>(m, 32 * kt + 4 * lg, p * (DK / 64) + d / 2, d & 1, li),
                        read_columns<DK>(m, 32 * kt + 16 + 4 * lg, p * (DK / 64) + d / 2, d & 1, li));
  }
  // The same while loads to LDS are under way: the compiler lets no transposing
  // read of its own pass those without waiting for them.  (Rows 16 apart lie at
  // the same place of their row, see swizzled().)
  __device__ __forceinline__ void read_past_loads(const uint16_t *m, int p, int li, int lg) {
#pragma unroll
    for (int b = 0; b < DK / 64; ++b) {
      const uint16_t *at = m + swizzled<DK>(4 * lg + li / 4, 4 * (p * (DK / 64) + b) + li % 4);
      const uint32_t addr = static_cast<uint32_t>(
          reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint16_t *)at));
      s16x4 x[8];
      constexpr int kStep = 16 * DK * 2;
      asm volatile(
          "ds_read_b64_tr_b16 %0, %8 offset:%9\n\t"
          "ds_read_b64_tr_b16 %1, %8 offset:%10\n\t"
          "ds_read_b64_tr_b16 %2, %8 offset:%11\n\t"
          "ds_read_b64_tr_b16 %3, %8 offset:%12\n\t"
          "ds_read_b64_tr_b16 %4, %8 offset:%13\n\t"
          "ds_read_b64_tr_b16 %5, %8 offset:%14\n\t"
          "ds_read_b64_tr_b16 %6, %8 offset:%15\n\t"
          "ds_read_b64_tr_b16 %7, %8 offset:%16\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
          : "v"(addr), "n"(0), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep), "n"(8), "n"(kStep + 8), "n"(2 * kStep + 8),
            "n"(3 * kStep + 8)
          : "memory");
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int half = 0; half < 2; ++half) a[kt][2 * b + half] = join(x[4 * half + 2 * kt], x[4 * half + 2 * kt + 1]);
    }
  }
  // The first of NA terms of m; the others are read as they are used.
  template <int NA, int NB>
  __device__ __forceinline__ void times(const uint16_t *m, const Terms<NB> (&b)[2], int p, int li, int lg,
                                        f32x4 (&x)[DK / 32]) const {
#pragma unroll
    for (int t = 0; t < NA; ++t) {
      ColumnTiles c = *this;
      if (t > 0) c.read(m + t * kC * DK, p, li, lg);
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          if (t + u >= (NA > NB ? NA : NB)) continue;
#pragma unroll
          for (int d = 0; d < DK / 32; ++d) x[d] = mfma32(c.a[kt][d], b[kt].t[u], x[d]);
        }
    }
  }
};

// Two blocks of a triangular operand; x[i] += block i times y.
template <int NA>
struct Blocks {
  bf16x8 a[2][NA];
  __device__ __forceinline__ void read(const uint16_t *m, int b0, int b1, int lane) {
#pragma unroll
    for (int t = 0; t < NA; ++t) {
      a[0][t] = read8(m + t * kTriTerm + (b0 * 64 + lane) * 8);
      a[1][t] = read8(m + t * kTriTerm + (b1 * 64 + lane) * 8);
    }
  }
  template <int NB>
  __device__ __forceinline__ void times(const Terms<NB> &y, f32x4 (&x)[2]) const {
#pragma unroll
    for (int t = 0; t < NA; ++t)
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        if (t + u >= (NA > NB ? NA : NB)) continue;
        x[0] = mfma32(a[0][t], y.t[u], x[0]);
        x[1] = mfma32(a[1][t], y.t[u], x[1]);
      }
  }
};

// A wave's registers through LDS: [item][lane] of 16 bytes.
__device__ __forceinline__ void put(char *x, int item, int lane, f32x4 v) {
  *reinterpret_cast<f32x4 *>(x + item * 1024 + lane * 16) = v;
}
__device__ __forceinline__ f32x4 take(const char *x, int item, int lane) {
  return *reinterpret_cast<const f32x4 *>(x + item * 1024 + lane * 16);
}
template <int N>
__device__ __forceinline__ void put(char *x, int item, int lane, const Terms<N> &t) {
#pragma unroll
  for (int i = 0; i < N; ++i) *reinterpret_cast<bf16x8 *>(x + (item + i) * 1024 + lane * 16) = t.t[i];
}
template <int N>
__device__ __forceinline__ Terms<N> take_terms(const char *x, int item, int lane) {
  Terms<N> t;
#pragma unroll
  for (int i = 0; i < N; ++i) t.t[i] = *reinterpret_cast<const bf16x8 *>(x + (item + i) * 1024 + lane * 16);
  return t;
}
// The two tiles of half p, and of the other half (with constant indices: arrays
// indexed by p would live in memory).
__device__ __forceinline__ void halves(const f32x4 (&x)[4], int p, f32x4 (&mine)[2], f32x4 (&other)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      mine[i][e] = p == 0 ? x[i][e] : x[2 + i][e];
      other[i][e] = p == 0 ? x[2 + i][e] : x[i][e];
    }
}
// All waves' writes to LDS are visible after it; loads and stores of global
// memory (and loads to LDS) stay under way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The sequence at place r of the packed ones in order of falling length (the
// lengths need not make sense: any values have an order).
__device__ __forceinline__ int by_length(const DeltaArgs &A, int r) {
  const int lane = threadIdx.x & 63, n = A.nseq;
  const int len = lane < n ? static_cast<int>(static_cast<uint32_t>(A.off[lane + 1]) - static_cast<uint32_t>(A.off[lane])) : 0;
  int before = 0;
  for (int j = 0; j < n; ++j) {
    const int other = __builtin_amdgcn_readlane(len, j);
    before += other > len || (other == len && j < lane) ? 1 : 0;
  }
  return __builtin_ctzll(__ballot(lane < n && before == r));
}

// Workgroups of one sequence and head (which share K, Q and the triangles) are
// neighbours on one XCD.  Sequences of one length: each XCD takes a run of them
// (with their heads, which share K and Q too).  Packed sequences: the heads go
// round the XCDs, and up to 64 sequences are taken in order of falling length,
// so that no XCD and no compute unit is left with the long ones at the end.
struct Place {
  int s, h, cb;
};
__device__ __forceinline__ bool place(const DeltaArgs &A, int colblocks, int block, int blocks, Place *p) {
  int sh;
  if (A.off == nullptr) {
    const int id = xcd_remap(block, blocks);
    p->cb = id % colblocks;
    sh = id / colblocks;
  } else {
    const int k = block / kXcd;
    p->cb = k % colblocks;
    sh = k / colblocks * kXcd + block % kXcd;
    if (sh >= A.nseq * A.hv) return false;      // (the grid is whole rounds of the XCDs)
  }
  p->h = sh % A.hv;
  p->s = sh / A.hv;
  if (A.off != nullptr && A.nseq > 1 && A.nseq <= 64) p->s = by_length(A, p->s);
  return true;
}

// Half p's D tiles of a state at [dk][cols] memory, and of [64][16] at [64][dvp];
// columns past them go nowhere, rows past dk lie past the resource's end.  (What
// the backward pass hands on is read after the whole scan; held in the caches it
// would push the triangles out: backward scan of 2 x 4097 tokens 246 us, 232.)
template <int DK>
__device__ __forceinline__ void store_state(const DeltaArgs &A, float *base, int cols, const f32x4 (&S)[DK / 32], int p,
                                            int lg, int col) {
  const Rsrc r = buffer(base, A.dk * cols * 4);
  const uint32_t first = col < cols ? ((p * (DK / 2) + 8 * lg) * cols + col) * 4 : kNowhere;
#pragma unroll
  for (int d = 0; d < DK / 32; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) bstore_far(r, first + state_row(d, 0, e) * cols * 4, S[d][e]);
}
template <int DK>
__device__ __forceinline__ void load_state(const DeltaArgs &A, const float *base, f32x4 (&S)[DK / 32], int p, int lg,
                                           int col) {
  const Rsrc r = buffer(base, base != nullptr ? A.dk * A.dv * 4 : 0);
  const uint32_t first = col < A.dv ? ((p * (DK / 2) + 8 * lg) * A.dv + col) * 4 : kNowhere;
#pragma unroll
  for (int d = 0; d < DK / 32; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[d][e] = bload<float>(r, first + state_row(d, 0, e) * A.dv * 4);
}
__device__ __forceinline__ void store_rows(const DeltaArgs &A, float *base, const f32x4 (&x)[2], int p, int lg, int col) {
  const Rsrc r = buffer(base);
  const uint32_t first = col < A.dvp ? ((32 * p + 4 * lg) * A.dvp + col) * 4 : kNowhere;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) bstore_far(r, first + (16 * i + e) * A.dvp * 4, x[i][e]);
}

// Whether whole pieces go to LDS directly.
template <typename T, bool VEC> constexpr bool kDirect = VEC && sizeof(T) == 2;
// Whether as many waves again do nothing but load: where the others leave half
// of the registers (one wave a SIMD) and nothing has to pass through registers
// on its way (which it might: 250 us instead of 183, of two terms).
template <typename T, bool VEC, int NP> constexpr bool kLoaders = kDirect<T, VEC> && NP <= 2;
template <typename T, bool VEC, int NP>
constexpr int kBlock = Shape<NP>::kThreads * (kLoaders<T, VEC, NP> ? 2 : 1);
// The loading waves' part of a scan from chunk c0 on, chunks `step` apart: as many
// barriers a chunk as the others have.  A buffer's parts are loaded again, for
// the chunk after next, once the others have them in registers, some between
// any two barriers (issuing loads takes its time too, and the others wait at the
// barriers): BACK, the triangles after the first barrier, Q after the second, K
// and the gates after the third; forward Q and the gates after the first, K and
// the triangles after the second; what is left of the triangles (blocks from kEnd
// on) at the start of the next chunk.  v (BACK: dout) has one buffer, which is
// read at a chunk's start and loaded again, for the next chunk, after the first
// barrier (a second one would not fit beside the triangles of keys of 128).  Loads
// return in order: what the next chunk needs has come when no more are out than
// were issued since.
template <bool BACK, typename Load, typename Lds>
__device__ __forceinline__ void load_chunks(Load &next, const DeltaArgs &A, const Seq &q, const uint16_t *m, int64_t c0,
                                            int64_t step, Lds (&lds)[2], uint16_t *v) {
  constexpr int kTri = Load::kTri, kEnd = BACK ? 4 : (kTri + 1) / 2;
  static_assert(kEnd <= Load::kBlocks / Load::kWaves, "every wave issues the triangles' first kEnd loads");
  const auto in = [&](int64_t c) { return c >= 0 && c < q.len; };
  if (in(c0)) {
    next.load(A, q, c0, m, lds[0]);
    next.load_v(v);
  }
  if (in(c0 + step)) next.load(A, q, c0 + step, m, lds[1]);
  wait_loads();
  __syncthreads();
  int buf = 0;
  bool rest = false;                       // of the next chunk's triangles, aimed at still
  for (; in(c0); c0 += step) {
    const bool more = in(c0 + 2 * step);
    Lds &l = lds[buf];
    if (rest) next.load_tri(m, lds[buf ^ 1], kEnd, kTri);
    lds_barrier();
    if (in(c0 + step)) next.load_v(v);     // (aimed at it still)
    if (more) {
      next.aim(A, q, c0 + 2 * step);
      if (BACK) {
        next.load_tri(m, l, 0, 3);
      } else {
        next.load_gates(A, l);
        next.load_q(A, l);
      }
    }
    lds_barrier();
    if (more) {
      if (BACK) {
        next.load_q(A, l);
        next.load_tri(m, l, 3, kEnd);
      } else {
        next.load_k(A, l);
        next.load_tri(m, l, 0, 1);
      }
    }
    lds_barrier();
    if (more) {
      if (BACK) {
        next.load_k(A, l);
        next.load_gates(A, l);
      } else {
        next.load_tri(m, l, 1, kEnd);
      }
      wait_loads<Load::kLeast + kEnd>();
    } else {
      wait_loads();
    }
    rest = more;
    lds_barrier();
    buf ^= 1;
  }
}
// Exchanged items (1 KB) of a pair, reused from one exchange to the next; without
// outputs six.
constexpr int kItems = 9, kItemsBwd = 6;
// Buffers of v: where the waves load for themselves, they do so for the next chunk
// while others may still read this one's.
template <typename T, bool VEC, int NP> constexpr int kBuffersV = kDirect<T, VEC> && !kLoaders<T, VEC, NP> ? 2 : 1;

// Where token rows of T are whole pieces (VEC), two chunks' operands.
template <typename T, int DK, bool KEEP, bool VEC, int NP>
struct Forward {
  static constexpr int kNi = kInputTerms<T>;
  static constexpr bool kDma = kDirect<T, VEC>;
  typedef ChunkLoad<T, DK, KEEP ? kTerms : 2 * kTerms, !KEEP, VEC, kDma, NP> Load;
  static constexpr int kBuffers = kDma ? 2 : 1;
  struct Shared {
    typename Load::Lds lds[kBuffers];
    __attribute__((aligned(16))) uint16_t v[kBuffersV<T, VEC, NP>][Load::kValues];
    __attribute__((aligned(16))) char xch[NP][(KEEP ? kItemsBwd : kItems) * 1024];
  };
};
template <typename T, int DK, bool VEC, int NP>
struct Backward {
  static constexpr int kNi = kInputTerms<T>;
  static constexpr bool kDma = kDirect<T, VEC>;
  typedef ChunkLoad<T, DK, 2 * kTerms, true, VEC, kDma, NP> Load;
  static constexpr int kBuffers = kDma ? 2 : 1;
  struct Shared {
    typename Load::Lds lds[kBuffers];
    __attribute__((aligned(16))) uint16_t v[kBuffersV<T, VEC, NP>][Load::kValues];
    __attribute__((aligned(16))) char xch[NP][kItemsBwd * 1024];
  };
};

// Forward.  KEEP: S and V are stored for the backward pass, out and state not.
// `block` of `blocks` workgroups.
template <typename T, int DK, bool KEEP, bool VEC, int NP>
__device__ __forceinline__ void scan_forward(const DeltaArgs &A, int colblocks, int block, int blocks,
                                             typename Forward<T, DK, KEEP, VEC, NP>::Shared &sh) {
  typedef Forward<T, DK, KEEP, VEC, NP> F;
  typedef typename F::Load Load;
  typedef typename Load::Lds Lds;
  constexpr int kNi = F::kNi, kNs = kTerms, kHalf = DK / 64, kBuffers = F::kBuffers;
  constexpr bool kDma = F::kDma, kAhead = kNi == 1, kSelf = !kLoaders<T, VEC, NP>;   // (kSelf: waves load for themselves)
  Place pl;
  if (!place(A, colblocks, block, blocks, &pl)) return;
  const int s = pl.s, h = pl.h;
  const Seq q = sequence(A, s);
  Load next;
  next.init(A, h, pl.cb, static_cast<const T *>(A.v), A.vs);
  const int lane = next.lane, li = next.li, lg = next.lg, p = next.wave % 2;
  char *xa = sh.xch[next.wave / 2];
  const int col = next.col0 + 16 * (next.wave / 2) + li;
  const int64_t state_at = (static_cast<int64_t>(s) * A.hv + h) * A.dk * A.dv;
  const f32x4 zero = {0, 0, 0, 0};
  if constexpr (!kSelf)
    if (uniform(static_cast<int>(threadIdx.x / 64)) >= Shape<NP>::kWaves) {
      load_chunks<false>(next, A, q, A.T, 0, kC, sh.lds, sh.v[0]);
      return;
    }
  f32x4 S[DK / 32];
  load_state<DK>(A, A.h0 != nullptr ? A.h0 + state_at : nullptr, S, p, lg, col);
  RowOffsets rows;
  if (q.len > 0) {
    if (kSelf) {
      next.load(A, q, 0, A.T, sh.lds[0]);
      next.load_v(sh.v[0]);
      next.store(sh.lds[0]);
    }
    if (KEEP) store_state<DK>(A, A.S + (q.slot0 * A.hv + h) * A.dk * A.dvp, A.dvp, S, p, lg, col);
  }
  __syncthreads();
  int buf = 0;
  for (int64_t c0 = 0; c0 < q.len; c0 += kC) {
    const Window w = window(A, q, c0);
    const int64_t at = (q.slot0 + c0 / kC) * A.hv + h;
    const Lds &l = sh.lds[buf];
    Lds &ln = sh.lds[kBuffers == 2 ? buf ^ 1 : 0];
    const bool more = c0 + kC < q.len;
    constexpr int kBv = kBuffersV<T, VEC, NP>;
    const f32x4 v[2] = {next.values(sh.v[buf % kBv], 2 * p), next.values(sh.v[buf % kBv], 2 * p + 1)};
    RowTiles<DK, kNi> kr, qr;
    if (kAhead) {
      kr.read(l.k, p, li, lg);
      if (!KEEP) qr.read(l.q, p, li, lg);
      __builtin_amdgcn_sched_barrier(0);
    }
    const f32x4 eg[2] = {load4(l.eg + 32 * p + 4 * lg), load4(l.eg + 32 * p + 16 + 4 * lg)};
    const f32x4 be[2] = {load4(l.beta + 32 * p + 4 * lg), load4(l.beta + 32 * p + 16 + 4 * lg)};
    const f32x4 ew[2] = {load4(l.ew + 32 * p + 4 * lg), load4(l.ew + 32 * p + 16 + 4 * lg)};
    const float last = l.eg[kC - 1];
    if (kSelf && more) {                    // (the loads' issue spreads over the chunk)
      next.aim(A, q, c0 + kC);
      next.load_v(sh.v[(buf + 1) % kBv]);
      next.load_gates(A, ln);
      next.load_k(A, ln);
    }
    // K S and Q S over this half's state rows
    f32x4 xm[2], om[2];
    Blocks<kNs> ta, tb;
    {
      f32x4 x[4] = {zero, zero, zero, zero}, other[2];
      Terms<kNs> st[kHalf];
#pragma unroll
      for (int ks = 0; ks < kHalf; ++ks) st[ks] = split<kNs>(S[2 * ks], S[2 * ks + 1]);
      if (!kAhead) kr.read(l.k, p, li, lg);
      kr.times(st, x);
      if (kAhead) {
        ta.read(l.tri, tri_block(2 * p, p), tri_block(2 * p + 1, p), lane);
        tb.read(l.tri, tri_block(2, 0), tri_block(3, 0), lane);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (kSelf && !KEEP && more) next.load_q(A, ln);
      halves(x, p, xm, other);
      put(xa, 2 - 2 * p, lane, other[0]);  // (items in the order of the halves that take them)
      put(xa, 3 - 2 * p, lane, other[1]);
      if (!KEEP) {
        f32x4 o4[4] = {zero, zero, zero, zero};
        if (!kAhead) qr.read(l.q, p, li, lg);
        qr.times(st, o4);
        halves(o4, p, om, other);
        put(xa, 6 - 2 * p, lane, other[0]);
        put(xa, 7 - 2 * p, lane, other[1]);
      }
    }
    lds_barrier();
    // this half's steps: R, and V = T R (of the second half's the first half's part)
    f32x4 r[2], o[2], V[2] = {zero, zero};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[i] = be[i] * (v[i] - eg[i] * (xm[i] + take(xa, 2 * p + i, lane)));
      if (!KEEP) o[i] = (om[i] + take(xa, 4 + 2 * p + i, lane)) * (eg[i] * A.scale);
    }
    if (kSelf && more) next.load_tri(A.T, ln);
    const Terms<kNs> rt = split<kNs>(r[0], r[1]);
    if (!kAhead) {
      ta.read(l.tri, tri_block(2 * p, p), tri_block(2 * p + 1, p), lane);
      tb.read(l.tri, tri_block(2, 0), tri_block(3, 0), lane);
    }
    if (p == 0) {
      f32x4 y[2] = {zero, zero};
      tb.times(rt, y);
      put(xa, 0, lane, y[0]);              // (where this wave alone has read)
      put(xa, 1, lane, y[1]);
    }
    ta.times(rt, V);
    const uint16_t *tp = l.tri + kTerms * kTriTerm;
    Blocks<kNs> pa, pb;
    if (!KEEP && kAhead) {
      pa.read(tp, tri_block(2 * p, p), tri_block(2 * p + 1, p), lane);
      pb.read(tp, tri_block(2, 0), tri_block(3, 0), lane);
    }
    ColumnTiles<DK> kc;
    if (!kSelf) kc.read(l.k, p, li, lg);
    lds_barrier();
    if (p == 1) {
      V[0] += take(xa, 0, lane);
      V[1] += take(xa, 1, lane);
    }
    Terms<kNs> vw[2];
    const Terms<kNs> mine = split<kNs>(V[0] * ew[0], V[1] * ew[1]);
    put(xa, 3 - 3 * p, lane, mine);        // (the second half's where it alone has just read)
    Terms<kNs> vo;
    if (!KEEP) {
      vo = split<kNs>(V[0], V[1]);
      if (p == 0) put(xa, 6, lane, vo);
    }
#pragma unroll
    for (int d = 0; d < DK / 32; ++d) S[d] *= last;
    if (kDma && kSelf)
      kc.read_past_loads(l.k, p, li, lg);
    else if (kSelf)
      kc.read(l.k, p, li, lg);
    lds_barrier();
    if (p == 0) {
      vw[0] = mine;
      vw[1] = take_terms<kNs>(xa, 0, lane);
    } else {
      vw[0] = take_terms<kNs>(xa, 3, lane);
      vw[1] = mine;
    }
    kc.template times<kNi>(l.k, vw, p, li, lg, S);
    if constexpr (!KEEP) {
      if (!kAhead) {
        pa.read(tp, tri_block(2 * p, p), tri_block(2 * p + 1, p), lane);
        pb.read(tp, tri_block(2, 0), tri_block(3, 0), lane);
      }
      pa.times(vo, o);
      if (p == 1) pb.times(take_terms<kNs>(xa, 6, lane), o);
    }
    if (kBuffers == 1) lds_barrier();
    buf = kBuffers == 2 ? buf ^ 1 : 0;
    if (kSelf && more) next.store(ln);
    // (stores come after the wait for the next chunk's loads, which would
    // otherwise wait for them too)
    if constexpr (!KEEP) {
      rows.plan(A, w, static_cast<int64_t>(A.hv) * A.dv * sizeof(T), sizeof(T), p, lg, col);
      store_tokens(static_cast<T *>(A.out) + (w.low * A.hv + h) * A.dv, rows, o);
    } else {
      store_rows(A, A.V + at * kC * A.dvp, V, p, lg, col);
      if (more) store_state<DK>(A, A.S + (at + A.hv) * A.dk * A.dvp, A.dvp, S, p, lg, col);
    }
    lds_barrier();
  }
  if (!KEEP && A.state != nullptr) store_state<DK>(A, A.state + state_at, A.dv, S, p, lg, col);
}

// Backward: the gradient of the state, from the last chunk to the first.
template <typename T, int DK, bool VEC, int NP>
__device__ __forceinline__ void scan_backward(const DeltaArgs &A, int colblocks, int block, int blocks,
                                              typename Backward<T, DK, VEC, NP>::Shared &sh) {
  typedef Backward<T, DK, VEC, NP> B;
  typedef typename B::Load Load;
  typedef typename Load::Lds Lds;
  constexpr int kNi = B::kNi, kNs = kTerms, kHalf = DK / 64, kBuffers = B::kBuffers;
  constexpr bool kDma = B::kDma, kAhead = kNi == 1, kSelf = !kLoaders<T, VEC, NP>;
  Place pl;
  if (!place(A, colblocks, block, blocks, &pl)) return;
  const int s = pl.s, h = pl.h;
  const Seq q = sequence(A, s);
  const int64_t row = static_cast<int64_t>(A.hv) * A.dv;      // token stride of dout and dv
  Load next;
  next.init(A, h, pl.cb, static_cast<const T *>(A.dout), row);
  const int lane = next.lane, li = next.li, lg = next.lg, p = next.wave % 2;
  char *xa = sh.xch[next.wave / 2];
  const int col = next.col0 + 16 * (next.wave / 2) + li;
  const int64_t state_at = (static_cast<int64_t>(s) * A.hv + h) * A.dk * A.dv;
  const f32x4 zero = {0, 0, 0, 0};
  const int64_t first = (static_cast<int64_t>(q.len + kC - 1) / kC - 1) * kC;
  if constexpr (!kSelf)
    if (uniform(static_cast<int>(threadIdx.x / 64)) >= Shape<NP>::kWaves) {
      load_chunks<true>(next, A, q, A.TT, first, -kC, sh.lds, sh.v[0]);
      return;
    }
  f32x4 D[DK / 32];
  load_state<DK>(A, A.dstate != nullptr ? A.dstate + state_at : nullptr, D, p, lg, col);
  RowOffsets rows;
  if (q.len > 0) {
    if (kSelf) {
      next.load(A, q, first, A.TT, sh.lds[0]);
      next.load_v(sh.v[0]);
      next.store(sh.lds[0]);
    }
    store_state<DK>(A, A.dS + ((q.slot0 + first / kC) * A.hv + h) * A.dk * A.dvp, A.dvp, D, p, lg, col);
  }
  __syncthreads();
  int buf = 0;
  for (int64_t c0 = first; c0 >= 0; c0 -= kC) {
    const Window w = window(A, q, c0);
    const int64_t at = (q.slot0 + c0 / kC) * A.hv + h;
    const Lds &l = sh.lds[buf];
    Lds &ln = sh.lds[kBuffers == 2 ? buf ^ 1 : 0];
    const bool more = c0 > 0;
    // all of dout for P^T dout and Q^T dout
    constexpr int kBv = kBuffersV<T, VEC, NP>;
    f32x4 o[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) o[rt] = next.values(sh.v[buf % kBv], rt);
    RowTiles<DK, kNi> kr;
    const uint16_t *tp = l.tri + kTerms * kTriTerm;
    Blocks<kNs> pa, pb;                     // P^T: this half's rows by the second half's steps, and the first's
    if (kAhead) {
      kr.read(l.k, p, li, lg);
      __builtin_amdgcn_sched_barrier(0);
    }
    const f32x4 eg[2] = {load4(l.eg + 32 * p + 4 * lg), load4(l.eg + 32 * p + 16 + 4 * lg)};
    const f32x4 be[2] = {load4(l.beta + 32 * p + 4 * lg), load4(l.beta + 32 * p + 16 + 4 * lg)};
    const f32x4 ew[2] = {load4(l.ew + 32 * p + 4 * lg), load4(l.ew + 32 * p + 16 + 4 * lg)};
    const float last = l.eg[kC - 1];
    if (kSelf && more) {
      next.aim(A, q, c0 - kC);
      next.load_v(sh.v[(buf + 1) % kBv]);
      next.load_gates(A, ln);
      next.load_k(A, ln);
    }
    f32x4 xm[2];
    Blocks<kNs> ta, tb;
    {
      f32x4 x[4] = {zero, zero, zero, zero}, other[2];
      Terms<kNs> st[kHalf];
#pragma unroll
      for (int ks = 0; ks < kHalf; ++ks) st[ks] = split<kNs>(D[2 * ks], D[2 * ks + 1]);
      if (!kAhead) kr.read(l.k, p, li, lg);
      kr.times(st, x);
      if (kAhead) {
        ta.read(l.tri, tri_block_t(2 * p, p), tri_block_t(2 * p + 1, p), lane);
        if (p == 1) tb.read(l.tri, tri_block_t(0, 1), tri_block_t(1, 1), lane);
        pa.read(tp, tri_block_t(2 * p, 1), tri_block_t(2 * p + 1, 1), lane);
        if (p == 0) pb.read(tp, tri_block_t(0, 0), tri_block_t(1, 0), lane);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (kSelf && more) next.load_q(A, ln);
      halves(x, p, xm, other);
      put(xa, 2 * p, lane, other[0]);
      put(xa, 2 * p + 1, lane, other[1]);
    }
    lds_barrier();
    f32x4 V[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) V[i] = (xm[i] + take(xa, 2 - 2 * p + i, lane)) * ew[i];
    if (kSelf && more) next.load_tri(A.TT, ln);
    if (!kAhead) {
      pa.read(tp, tri_block_t(2 * p, 1), tri_block_t(2 * p + 1, 1), lane);
      pb.read(tp, tri_block_t(0, 0), tri_block_t(1, 0), lane);
    }
    pa.times(split<kNi>(o[2], o[3]), V);
    if (p == 0) pb.times(split<kNi>(o[0], o[1]), V);
    const Terms<kNs> vt = split<kNs>(V[0], V[1]);
    f32x4 R[2] = {zero, zero};
    if (!kAhead) {
      ta.read(l.tri, tri_block_t(2 * p, p), tri_block_t(2 * p + 1, p), lane);
      tb.read(l.tri, tri_block_t(0, 1), tri_block_t(1, 1), lane);
    }
    if (p == 1) {
      f32x4 y[2] = {zero, zero};
      tb.times(vt, y);
      put(xa, 0, lane, y[0]);             // (where this wave alone has read)
      put(xa, 1, lane, y[1]);
    }
    ta.times(vt, R);
    ColumnTiles<DK> qc, kc;
    if (kDma && kSelf)
      qc.read_past_loads(l.q, p, li, lg);
    else
      qc.read(l.q, p, li, lg);
    lds_barrier();
    if (p == 0) {
      R[0] += take(xa, 0, lane);
      R[1] += take(xa, 1, lane);
    }
    const f32x4 dv[2] = {R[0] * be[0], R[1] * be[1]};
    Terms<kNs> xw[2];
    const Terms<kNs> mine = split<kNs>(zero - dv[0] * eg[0], zero - dv[1] * eg[1]);
    put(xa, 3 * p, lane, mine);
#pragma unroll
    for (int d = 0; d < DK / 32; ++d) D[d] *= last;
    Terms<kNs> ow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      ow[i] = split<kNs>(o[2 * i] * (load4(l.eg + 32 * i + 4 * lg) * A.scale),
                         o[2 * i + 1] * (load4(l.eg + 32 * i + 16 + 4 * lg) * A.scale));
    qc.template times<kNi>(l.q, ow, p, li, lg, D);
    if (kDma && kSelf)
      kc.read_past_loads(l.k, p, li, lg);
    else
      kc.read(l.k, p, li, lg);
    lds_barrier();
    if (p == 0) {
      xw[0] = mine;
      xw[1] = take_terms<kNs>(xa, 3, lane);
    } else {
      xw[0] = take_terms<kNs>(xa, 0, lane);
      xw[1] = mine;
    }
    kc.template times<kNi>(l.k, xw, p, li, lg, D);
    if (kBuffers == 1) lds_barrier();
    buf = kBuffers == 2 ? buf ^ 1 : 0;
    if (kSelf && more) next.store(ln);
    store_rows(A, A.dR + at * kC * A.dvp, R, p, lg, col);
    if (more) store_state<DK>(A, A.dS + (at - A.hv) * A.dk * A.dvp, A.dvp, D, p, lg, col);
    rows.plan(A, w, row * sizeof(T), sizeof(T), p, lg, col);
    store_tokens(static_cast<T *>(A.dval) + (w.low * A.hv + h) * A.dv, rows, dv);
    lds_barrier();
  }
  if (A.dh0 != nullptr) store_state<DK>(A, A.dh0 + state_at, A.dv, D, p, lg, col);
}

template <typename T, int DK, bool VEC, int NP>
__global__ __launch_bounds__((kBlock<T, VEC, NP>)) void delta_scan_kernel(DeltaArgs A, int colblocks) {
  __shared__ typename Forward<T, DK, false, VEC, NP>::Shared sh;
  scan_forward<T, DK, false, VEC, NP>(A, colblocks, blockIdx.x, gridDim.x, sh);
}

// The backward scan needs nothing of the forward one, so one launch runs both:
// half of the workgroups each, the longer backward ones first.  (2 x 4097 tokens,
// 16 value heads of 128, bf16: 290 us, one after the other 154 and 232, and 224 to
// 234 with loading waves; 64 x 197, 6 heads of 64, fp32: 96, 44 and 62.)
template <typename T, int DK, bool VEC, int NP>
__global__ __launch_bounds__((kBlock<T, VEC, NP>)) void delta_scans_kernel(DeltaArgs A, int colblocks) {
  __shared__ union {
    typename Forward<T, DK, true, VEC, NP>::Shared f;
    typename Backward<T, DK, VEC, NP>::Shared b;
  } sh;
  const int blocks = gridDim.x / 2, block = blockIdx.x;
  if (block < blocks)
    scan_backward<T, DK, VEC, NP>(A, colblocks, block, blocks, sh.b);
  else
    scan_forward<T, DK, true, VEC, NP>(A, colblocks, block - blocks, blocks, sh.f);
}

// Workgroups of a scan with cb column blocks, as place() takes them apart.
int64_t scan_blocks(const DeltaArgs &a, int cb) {
  int64_t heads = static_cast<int64_t>(a.nseq) * a.hv;
  if (a.off != nullptr) heads = (heads + kXcd - 1) / kXcd * kXcd;
  return heads * cb;
}

// One variant of the kernels and its launch.
template <typename T, int DK, bool VEC, int NP>
struct Scan {
  static int columns(const DeltaArgs &a) { return (a.dv + 16 * NP - 1) / (16 * NP); }
  static int64_t blocks(const DeltaArgs &a, bool back) { return scan_blocks(a, columns(a)) * (back ? 2 : 1); }
  static int64_t items(const DeltaArgs &a, bool back) { return blocks(a, back) * kBlock<T, VEC, NP>; }
  static hipError_t launch(const DeltaArgs &a, bool back, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(blocks(a, back))), block(kBlock<T, VEC, NP>);
    if (back)
      hipLaunchKernelGGL((delta_scans_kernel<T, DK, VEC, NP>), grid, block, 0, s, a, columns(a));
    else
      hipLaunchKernelGGL((delta_scan_kernel<T, DK, VEC, NP>), grid, block, 0, s, a, columns(a));
    return hipGetLastError();
  }
};
// As few pairs of waves to a workgroup as give no more workgroups than the card
// has compute units: each wave then has a SIMD of its own, and fewer wait for
// each other.  With more workgroups, as many pairs as LDS and registers hold
// share what is loaded: four, of rows of 128 two.  Calls over 4096 tokens, us,
// with one, two and four pairs, the rule's choice marked:
//   heads            8            32            64           80           256
//   of 64, bf16      132* 152 236 144* 161 247  170* 187 274 294 206* 288 675 511 466*
//     backward       169* 184 264 292* 308 387  594 529* 592 749 659 682* 2341 2073 2008*
//   of 64, fp32      - 272* 311   - 310* 362    - 334* 392   - 353* 429   - 797 636*
//   of 128, bf16     157* 185 -   164* 193 -    343 226* -   498 400* -   (128: 674 441* -)
//     backward       223* 251 -   512 446* -    1098 920* -  1379 1188* - (128: 2153 1772* -)
// Just past the number of compute units a second, nearly empty round begins: 64
// heads of 128 are 256 workgroups of two pairs, 80 heads 320 (226 and 400 us).
template <typename T, int DK, bool VEC, typename F>
auto with_scan(const DeltaArgs &a, bool back, F f) {
  if constexpr (kLoaders<T, VEC, 1>)
    if (Scan<T, DK, VEC, 1>::blocks(a, back) <= 256) return f(Scan<T, DK, VEC, 1>());
  if constexpr (DK == 64)
    if (Scan<T, DK, VEC, 2>::blocks(a, back) > 256) return f(Scan<T, DK, VEC, 4>());
  return f(Scan<T, DK, VEC, 2>());
}
template <typename T, int DK, typename F>
auto with_scan(const DeltaArgs &a, bool back, F f) {
  const bool vec = delta_vec(a, sizeof(T)) && delta_vec_values(a, a.v, a.vs, sizeof(T), 4) &&
                   (!back || delta_vec_values(a, a.dout, static_cast<int64_t>(a.hv) * a.dv, sizeof(T), 4));
  return vec ? with_scan<T, DK, true>(a, back, f) : with_scan<T, DK, false>(a, back, f);
}
template <typename F>
auto with_scan(const DeltaArgs &a, bool bf16, bool back, F f) {
  if (a.dk <= 64) return bf16 ? with_scan<bf16_t, 64>(a, back, f) : with_scan<float, 64>(a, back, f);
  return bf16 ? with_scan<bf16_t, 128>(a, back, f) : with_scan<float, 128>(a, back, f);
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs &a, bool bf16, bool back, hipStream_t s) {
  return with_scan(a, bf16, back, [&](auto scan) { return scan.launch(a, back, s); });
}

int64_t delta_scan_items(const DeltaArgs &a, bool bf16, bool back) {
  return with_scan(a, bf16, back, [&](auto scan) { return scan.items(a, back); });
}

}  // namespace vmk
