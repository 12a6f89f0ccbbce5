// Device helpers of the prompt kernels: sequences and their chunks, and the lane
// layout of the selective scan.
#pragma once

#include <hip/hip_runtime.h>

#include "prompt_internal.h"
#include "scan_device.h"
#include "vm_internal.h"

namespace vmk {
namespace {

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// One chunk of a sequence.
struct Piece {
  int seq;
  int c, count;          // the chunk's number and how many the sequence has
  int64_t lo, hi;        // the sequence's tokens
  int64_t t0;            // the chunk's first token
  int len;               // its tokens; 0 for an empty sequence's only chunk, -1: no chunk
};

__device__ __forceinline__ int64_t clamped(int32_t x, int64_t most) {
  const int64_t y = x;
  return y < 0 ? 0 : y > most ? most : y;
}

// Offsets that do not rise from 0 to L give wrong chunks, but none outside [0, L).
__device__ __forceinline__ Piece piece_of(const SeqArgs &q, int64_t slot) {
  Piece p;
  if (q.off == nullptr) {
    const int64_t per = (q.L + q.chunk - 1) / q.chunk;
    const int64_t seq = slot / per;
    p.seq = static_cast<int>(seq);
    p.c = static_cast<int>(slot - seq * per);
    p.lo = seq * q.L;
    p.hi = p.lo + q.L;
  } else {
    int a = 0, b = q.nseq;                 // the last sequence whose slots start at or before this one
    while (b - a > 1) {
      const int m = (a + b) / 2;
      if (clamped(q.off[m], q.L) / q.chunk + m <= slot) a = m; else b = m;
    }
    p.seq = a;
    p.lo = clamped(q.off[a], q.L);
    p.hi = clamped(q.off[a + 1], q.L);
    p.c = static_cast<int>(slot - p.lo / q.chunk - a);
  }
  const int64_t all = p.hi - p.lo;
  p.count = all > q.chunk ? static_cast<int>((all + q.chunk - 1) / q.chunk) : 1;
  p.t0 = p.lo + p.c * q.chunk;
  const int64_t left = p.hi - p.t0;
  p.len = static_cast<int>(left < q.chunk ? left : q.chunk);
  if (p.c < 0 || p.c >= p.count || p.len < 0) p.len = p.c == 0 && all <= 0 ? 0 : -1;
  return p;
}

// Where a sequence's state is kept, -1: nowhere.
__device__ __forceinline__ int64_t kept_at(const SeqArgs &q, int seq) {
  const int64_t s = q.where != nullptr ? q.where[seq] : seq;
  return s >= 0 && s < q.kept ? s : -1;
}
__device__ __forceinline__ bool starts_kept(const SeqArgs &q, int seq) {
  return q.fresh == nullptr || q.fresh[seq] == 0;
}

// ------------------------------------------------------ the scan's lane layout
// A wave holds 16 channels with 4 states in each lane: lane l has channel l % 16
// and states 4 q .. 4 q + 3, q = l / 16.  Tokens go by in groups of 4, and what is
// one value per token and channel (dt, dt u, y, ...) lies with token q in lane
// (channel, q).  Such a layout is that of a 4 x 4 x 1 matrix instruction's 16
// products: rows are the states (or the group's tokens), columns 4 of the
// channels, and the instruction's broadcasts hand the 4 tokens out:
//   update    h[i] += B_t[4 q + i] (dt u)[channel]    B in `by state`
//   read-out  sum_i C_t[4 q + i] h[i]                 C in `by token`
// by state: lane (q, s, i) holds token s, state 4 q + i; by token: lane (q, i, s)
// the same.  So neither the outer product nor the read-out's sum over a lane's
// states costs vector instructions, and both are exact fp32 products and sums.
typedef float f32x4 __attribute__((ext_vector_type(4)));

// h += b_s x_s of token S of the group.
template <int S>
__device__ __forceinline__ f32x4 rank1(float b, float x, f32x4 h) {
  return __builtin_amdgcn_mfma_f32_4x4x1f32(b, x, h, 2, S, 4 + S);
}
// Row S of the products is token S's sum over this lane's states; the others
// (another token's C with this token's states) are not used.
template <int S>
__device__ __forceinline__ float read_out(float c, f32x4 h) {
  f32x4 y = {0, 0, 0, 0};
  y = __builtin_amdgcn_mfma_f32_4x4x1f32(c, h[0], y, 2, 0, 0);
  y = __builtin_amdgcn_mfma_f32_4x4x1f32(c, h[1], y, 2, 1, 0);
  y = __builtin_amdgcn_mfma_f32_4x4x1f32(c, h[2], y, 2, 2, 0);
  y = __builtin_amdgcn_mfma_f32_4x4x1f32(c, h[3], y, 2, 3, 0);
  return y[S];
}

__device__ __forceinline__ void swap32(float &a, float &b) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap16(float &a, float &b) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
// Every lane gets its channel's values of the group's four tokens.
__device__ __forceinline__ void hand_out(float x, float (&y)[4]) {
  float a = x, b = x;
  swap32(a, b);                       // rows 0 1 0 1 and 2 3 2 3
  y[0] = y[1] = a;
  swap16(y[0], y[1]);
  y[2] = y[3] = b;
  swap16(y[2], y[3]);
}
// The other way: four values of each lane, summed over a channel's four lanes; lane
// (channel, q) gets that of token q.
__device__ __forceinline__ float gather(const float (&y)[4]) {
  float a = y[0], c = y[2], b = y[1], d = y[3];
  swap32(a, c);
  swap32(b, d);
  float e = a + c, f = b + d;
  swap16(e, f);
  return e + f;
}

// What a lane needs to reach its values: offsets in bytes, past every resource
// where there is no value.
struct Lane {
  int ch, q;                          // channel of the block, row of 16 lanes
  int cw;                             // channels of the block that exist
  bool live;
  uint32_t u, d, z;                   // token q of a tile
  uint32_t b, c;                      // B by state, C by token
  uint32_t bt, ct;                    // B by token, C by state (backward pass)
  uint32_t state[4];                  // in a block's [16][n]
};

template <typename T>
__device__ __forceinline__ Lane lane_of(const PromptScanArgs &a, int c0, int lane) {
  Lane l;
  l.ch = lane & 15;
  l.q = lane >> 4;
  l.cw = a.dim - c0 < 16 ? (a.dim > c0 ? a.dim - c0 : 0) : 16;
  l.live = l.ch < l.cw;
  const uint32_t es = sizeof(T), q = l.q, ch = l.ch, lo = lane & 3, hi = (lane >> 2) & 3;
  const auto at = [&](bool has, int64_t stride, uint32_t token, uint32_t col) {
    return has ? (token * static_cast<uint32_t>(stride) + col) * es : kOob;
  };
  l.u = at(l.live, a.us, q, ch);
  l.d = at(l.live, a.ds, q, ch);
  l.z = at(l.live, a.zs, q, ch);
  const uint32_t n = a.n, sl = 4 * q + lo, sh = 4 * q + hi;
  l.b = at(sl < n, a.bs, hi, sl);
  l.c = at(sh < n, a.cs, lo, sh);
  l.bt = at(sh < n, a.bs, lo, sh);
  l.ct = at(sl < n, a.cs, hi, sl);
#pragma unroll
  for (int i = 0; i < 4; ++i) l.state[i] = l.live && 4 * l.q + i < a.n ? (l.ch * a.n + 4 * l.q + i) * 4 : kOob;
  return l;
}

__device__ __forceinline__ float channel_value(const float *v, int c0, const Lane &l) {
  return v != nullptr && l.live ? v[c0 + l.ch] : 0.0f;
}

// `tokens` rows of `width` values from (token, col) on; none where tokens <= 0.
template <typename T>
__device__ __forceinline__ Rsrc rows(const void *base, int64_t stride, int64_t token, int64_t col, int tokens, int width) {
  const int bytes = tokens > 0 ? static_cast<int>(((tokens - 1) * stride + width) * sizeof(T)) : 0;
  return make_rsrc(static_cast<const T *>(base) + token * stride + col, bytes);
}

// Decay rates, ready for 2^x.  A rate of -Inf (which decays to 0 in any step) is
// held finite, so that the steps of 0 that fill up a group leave a state alone.
__device__ __forceinline__ float rate2(float a) {
  const float r = a * kLog2e;
  return r < -3.0e38f ? -3.0e38f : r;      // (NaN stays)
}

}  // namespace
}  // namespace vmk
