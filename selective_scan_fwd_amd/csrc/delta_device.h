// Device helpers shared by the gated delta rule's kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "mixer_internal.h"
#include "vm_internal.h"

namespace vmk {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

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

struct Seq {
  int64_t base;   // first token
  int64_t slot0;  // first chunk slot
  int len;
};

__device__ __forceinline__ int64_t packed_offset(const DeltaArgs &A, int s) {
  const int64_t o = A.off[s];
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
  return q;
}
// The sequence of a chunk slot: the last one whose first slot is <= slot.
__device__ __forceinline__ int sequence_of(const DeltaArgs &A, int64_t slot) {
  if (A.off == nullptr) return static_cast<int>(slot / ((A.L + kC - 1) / kC));
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

__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ f32x4 load4(const bf16_t *p) {
  const u16x4 r = *reinterpret_cast<const u16x4 *>(p);
  return f32x4{to_f32(r[0]), to_f32(r[1]), to_f32(r[2]), to_f32(r[3])};
}

// Rows 0 .. n-1 (tokens t0, t0 + dt, ...) of src[token][d] into dst[64][PITCH],
// zero elsewhere up to column COLS.  vec: d, the stride and the pointer are
// multiples of 4 values.
template <int COLS, int PITCH, int THREADS, typename T>
__device__ __forceinline__ void stage_rows(float *dst, const T *src, int64_t stride, int n, int d, bool vec) {
  for (int i = threadIdx.x; i < kC * (COLS / 4); i += THREADS) {
    const int row = i / (COLS / 4), c = (i % (COLS / 4)) * 4;
    f32x4 v = {0, 0, 0, 0};
    if (row < n && c < d) {
      const T *p = src + row * stride + c;
      if (vec) {
        v = load4(p);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < d) v[e] = to_f32(p[e]);
      }
    }
    *reinterpret_cast<f32x4 *>(dst + row * PITCH + c) = v;
  }
}

__device__ __forceinline__ bool can_vec4(const void *p, int64_t stride, int d, int esize) {
  return (d & 3) == 0 && (stride & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & (4 * esize - 1)) == 0;
}

}  // namespace vmk
