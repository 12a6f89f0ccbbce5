// Device helpers shared by the gated delta rule's kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "mixer_internal.h"
#include "vm_internal.h"

namespace vmk {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kC = kDeltaChunk;
// Row pitch in floats of a [64][64] tile in LDS: 4 past a multiple of 64 banks,
// so that 16 rows of 16-byte accesses meet 64 different banks.
constexpr int kPitchC = kC + 4;
// Smallest log decay: exp(-120) is 0 in fp32.  Running sums in a chunk stay
// finite, so a state that a token clears (g = -Inf) gives 0 and not NaN.
constexpr float kMinLogDecay = -120.0f;

// D[16][16] += A[16][4] B[4][16]: lane l holds A[l % 16][l / 16],
// B[l / 16][l % 16] and D[4 (l / 16) + r][l % 16] in register r.
__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// D += A[16][16] B[16][16] with the 16 inner indices taken in the order in
// which a D tile holds its rows: step r takes inner index 4 (l / 16) + r of
// lane l.  So a D tile is the next product's B (or transposed A) as it is.
__device__ __forceinline__ f32x4 mfma16(f32x4 a, f32x4 b, f32x4 c) {
  c = mfma4(a[0], b[0], c);
  c = mfma4(a[1], b[1], c);
  c = mfma4(a[2], b[2], c);
  return mfma4(a[3], b[3], c);
}

// ------------------------------------------------------ fp32 in bf16 terms
// bf16 matrix instructions run 16 times faster than fp32 ones.  An fp32 value is
// the sum of three bf16 terms (8 bits each); the product of two values is the
// sum of the products of their terms, of which those past the third place are
// left out.  With bf16 tokens one factor is a single term.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int N>
struct Terms {
  bf16x8 t[N];
};

// Two values rounded to nearest even, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

template <int N>
__device__ __forceinline__ Terms<N> split(f32x8 x) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  Terms<N> y;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    u32x4 p;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p[j] = pack2(x[2 * j], x[2 * j + 1]);
      if (i + 1 < N) {                     // (the remainder, exact)
        x[2 * j] -= __uint_as_float(p[j] << 16);
        x[2 * j + 1] -= __uint_as_float(p[j] & 0xffff0000u);
      }
    }
    y.t[i] = __builtin_bit_cast(bf16x8, p);
  }
  return y;
}
template <int N>
__device__ __forceinline__ Terms<N> split(f32x4 a, f32x4 b) {
  return split<N>(__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// D[16][16] += A[16][32] B[32][16]: lane l holds 8 inner values of row (column)
// l % 16 and D[4 (l / 16) + r][l % 16] in register r.  Which 8 of the 32 inner
// indices a lane group holds is free as long as A and B agree.
__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Rows of bf16 in LDS, COLS values each, in pieces of 8.  Piece p of row r is
// stored at place p ^ r, so that 16 rows read at the same column meet
// different banks.
template <int COLS>
__device__ __forceinline__ int swizzled(int row, int piece) {
  return row * COLS + ((piece ^ (row & (COLS / 8 - 1))) << 3);
}

// Four rows at `row`, transposed: lane l of each 16 lanes gets column
// 8 (l % 16 / 4) + 4 half + l % 4 past 32 block of the rows row .. row + 3, where
// row may differ between the groups of 16 lanes.
template <int COLS>
__device__ __forceinline__ s16x4 read_columns(const uint16_t *m, int row, int block, int half, int li) {
  const uint16_t *p = m + swizzled<COLS>(row + li / 4, 4 * block + li % 4) + 4 * half;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4 *)const_cast<uint16_t *>(p));
}
__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 x = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, x);
}
__device__ __forceinline__ bf16x8 read8(const uint16_t *p) { return *reinterpret_cast<const bf16x8 *>(p); }

// Block of the lower triangle [64][64] in 16 x 32 blocks: row tile rt, column
// block ks (0, or 1 from row tile 2 on), and of its transpose.
__device__ __forceinline__ constexpr int tri_block(int rt, int ks) { return rt < 2 ? rt : 2 * rt - 2 + ks; }
__device__ __forceinline__ constexpr int tri_block_t(int rt, int ks) { return rt < 2 ? 2 * rt + ks : rt + 2; }

// Eight values of a triangular operand on their way to the scans (see DeltaArgs).
template <typename T, int TERMS>
__device__ __forceinline__ void put_block(uint16_t *m, int block, int lane, f32x4 a, f32x4 b) {
  if constexpr (sizeof(T) == 2) {
    const Terms<TERMS> t = split<TERMS>(a, b);
#pragma unroll
    for (int x = 0; x < TERMS; ++x) *reinterpret_cast<bf16x8 *>(m + x * kTriTerm + (block * 64 + lane) * 8) = t.t[x];
  } else {
    f32x4 *p = reinterpret_cast<f32x4 *>(m) + (block * 64 + lane) * 2;
    p[0] = a;
    p[1] = b;
  }
}

// Global memory through buffer resources: 32-bit byte offsets from a base, and
// an offset of kNowhere reads zero and writes nothing, so rows past a chunk's
// end and columns past a head's need no branch.
using Rsrc = __amdgpu_buffer_rsrc_t;
constexpr uint32_t kNowhere = 0x80000000u;  // (and what is added to it)
__device__ __forceinline__ Rsrc buffer(const void *base, uint32_t bytes = kNowhere) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, static_cast<int>(bytes), 0x00020000);
}
template <typename T> __device__ __forceinline__ T bload(Rsrc r, uint32_t off);
template <> __device__ __forceinline__ float bload<float>(Rsrc r, uint32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, static_cast<int>(off), 0, 0));
}
template <> __device__ __forceinline__ bf16_t bload<bf16_t>(Rsrc r, uint32_t off) {
  return static_cast<bf16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, static_cast<int>(off), 0, 0));
}
__device__ __forceinline__ void bstore(Rsrc r, uint32_t off, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, static_cast<int>(off), 0, 0);
}
// Of what no kernel reads before the caches have passed on to other lines.
__device__ __forceinline__ void bstore_far(Rsrc r, uint32_t off, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, static_cast<int>(off), 0, /*nontemporal*/ 2);
}
__device__ __forceinline__ void bstore(Rsrc r, uint32_t off, bf16_t v) {
  __builtin_amdgcn_raw_buffer_store_b16(v, r, static_cast<int>(off), 0, 0);
}
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 bload16(Rsrc r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(off), 0, 0));
}
__device__ __forceinline__ void bstore16(Rsrc r, uint32_t off, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, static_cast<int>(off), 0, 0);
}
// 16 (4) bytes of every lane straight to LDS at `lds` + 16 (4) * lane.
__device__ __forceinline__ void to_lds16(Rsrc r, void *lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16,
                                           static_cast<int>(off), 0, 0, 0);
}
__device__ __forceinline__ void to_lds4(Rsrc r, void *lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 4,
                                           static_cast<int>(off), 0, 0, 0);
}
// Waits until no more than the last LEFT of this wave's loads (to LDS) are under
// way; other waves' follow with the barrier.
template <int LEFT = 0>
__device__ __forceinline__ void wait_loads() {
  static_assert(LEFT < 64, "six bits, the upper two apart");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (LEFT & 15) | (LEFT >> 4) << 14);
}

// Eight values of a token row, as they are in memory.
template <typename T> struct Piece;
template <> struct Piece<bf16_t> {
  u32x4 x;
};
template <> struct Piece<float> {
  u32x4 x[2];
};
// The 8 values at byte offset `at` (column c of a row of d), zero past column d
// and at kNowhere.  VEC: d is a multiple of 8 and the rows 16-byte aligned; else
// value by value.
template <bool VEC>
__device__ __forceinline__ Piece<bf16_t> load_piece(Rsrc r, uint32_t at, int c, int d, bf16_t) {
  Piece<bf16_t> p;
  if (VEC) {
    p.x = bload16(r, at);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = bload<bf16_t>(r, c + 2 * e < d ? at + 4 * e : kNowhere);
      const uint32_t hi = bload<bf16_t>(r, c + 2 * e + 1 < d ? at + 4 * e + 2 : kNowhere);
      p.x[e] = lo | hi << 16;
    }
  }
  return p;
}
template <bool VEC>
__device__ __forceinline__ Piece<float> load_piece(Rsrc r, uint32_t at, int c, int d, float) {
  Piece<float> p;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (VEC) {
      p.x[half] = bload16(r, at + 16 * half);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        p.x[half][e] = __float_as_uint(bload<float>(r, c + 4 * half + e < d ? at + 16 * half + 4 * e : kNowhere));
    }
  }
  return p;
}
// Into rows of bf16 terms, `term` values apart.
template <int COLS>
__device__ __forceinline__ void store_piece(uint16_t *m, int /*term*/, int row, int piece, const Piece<bf16_t> &p) {
  *reinterpret_cast<u32x4 *>(m + swizzled<COLS>(row, piece)) = p.x;
}
template <int COLS>
__device__ __forceinline__ void store_piece(uint16_t *m, int term, int row, int piece, const Piece<float> &p) {
  const Terms<3> t = split<3>(__builtin_bit_cast(f32x4, p.x[0]), __builtin_bit_cast(f32x4, p.x[1]));
#pragma unroll
  for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x8 *>(m + i * term + swizzled<COLS>(row, piece)) = t.t[i];
}
// The piece's terms.
__device__ __forceinline__ void piece_terms(const Piece<bf16_t> &p, bf16x8 (&t)[1]) {
  t[0] = __builtin_bit_cast(bf16x8, p.x);
}
__device__ __forceinline__ void piece_terms(const Piece<float> &p, bf16x8 (&t)[3]) {
  const Terms<3> x = split<3>(__builtin_bit_cast(f32x4, p.x[0]), __builtin_bit_cast(f32x4, p.x[1]));
  t[0] = x.t[0];
  t[1] = x.t[1];
  t[2] = x.t[2];
}
template <typename T> constexpr int kInputTerms = sizeof(T) == 2 ? 1 : 3;

// A value that is the same for the whole wave, where the compiler cannot tell:
// buffer resources made from it would be taken apart lane by lane.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(x));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(x >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

struct Seq {
  int64_t base;   // first token
  int64_t slot0;  // first chunk slot
  int len;
};

__device__ __forceinline__ int64_t packed_offset(const DeltaArgs &A, int s) {
  const int64_t o = uniform(A.off[s]);
  return o < 0 ? 0 : o > A.L ? A.L : o;
}
__device__ __forceinline__ Seq sequence(const DeltaArgs &A, int s) {
  Seq q;
  if (A.off == nullptr) {
    q.base = s * A.L;
    q.len = static_cast<int>(A.L);
    q.slot0 = s * ((A.L + kC - 1) / kC);
  } else {
    q.base = packed_offset(A, s);
    const int64_t end = packed_offset(A, s + 1);
    q.len = end > q.base ? static_cast<int>(end - q.base) : 0;
    q.slot0 = q.base / kC + s;
  }
  q.base = uniform(q.base);
  q.slot0 = uniform(q.slot0);
  q.len = uniform(q.len);
  return q;
}
// The sequence of a chunk slot: the last one whose first slot is <= slot.
__device__ __forceinline__ int sequence_of(const DeltaArgs &A, int64_t slot) {
  if (A.off == nullptr)                  // (fewer than 2^23 slots)
    return static_cast<int>(static_cast<uint32_t>(slot) / static_cast<uint32_t>((A.L + kC - 1) / kC));
  int lo = 0, hi = A.nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (packed_offset(A, mid) / kC + mid <= slot) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// Token of the i-th visited step of a chunk whose first visited step is c0.
__device__ __forceinline__ int64_t token_of(const DeltaArgs &A, const Seq &q, int64_t c0, int i) {
  return A.reverse ? q.base + q.len - 1 - (c0 + i) : q.base + c0 + i;
}

// The chunk's steps as byte offsets from its lowest token: step i is at
// `first + i * step` (step negative in reverse).
struct Window {
  int64_t low;      // the lowest token
  int n;            // steps
  __device__ __forceinline__ uint32_t at(const DeltaArgs &A, int i, int64_t stride_bytes) const {
    return static_cast<uint32_t>(A.reverse ? n - 1 - i : i) * static_cast<uint32_t>(stride_bytes);
  }
};
__device__ __forceinline__ Window window(const DeltaArgs &A, const Seq &q, int64_t c0) {
  Window w;
  w.n = q.len - c0 < kC ? static_cast<int>(q.len - c0) : kC;
  w.low = token_of(A, q, c0, A.reverse ? w.n - 1 : 0);
  return w;
}

__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

}  // namespace vmk
