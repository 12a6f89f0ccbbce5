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
  int64_t id;            // its slot in the tokens' order
};

__device__ __forceinline__ int64_t clamped(int32_t x, int64_t most) {
  const int64_t y = x;
  return y < 0 ? 0 : y > most ? most : y;
}

// Of packed sequence i: its first token over the tokens of a chunk.
__device__ __forceinline__ int slots_before(const SeqArgs &q, int i) {
  return static_cast<int>(static_cast<uint32_t>(clamped(q.off[i], q.L)) / static_cast<uint32_t>(q.chunk));
}

// The same in scalar registers (all lanes hold the same): addresses that the compiler
// takes for the lanes' own cost a loop over them at every load.
__device__ __forceinline__ int64_t uniform64(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x)),
                 hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ Piece uniform(Piece p) {
  p.seq = uniform(p.seq);
  p.c = uniform(p.c);
  p.count = uniform(p.count);
  p.lo = uniform64(p.lo);
  p.hi = uniform64(p.hi);
  p.t0 = uniform64(p.t0);
  p.len = uniform(p.len);
  p.id = uniform64(p.id);
  return p;
}

// The piece of a slot, the same for all lanes of a wave.  Packed: the last sequence whose
// slots start at or before this one is looked for by 64 lanes at once (one load for up to
// 64 sequences).  Offsets that do not rise from 0 to L give wrong chunks, but none
// outside [0, L).
__device__ __forceinline__ Piece piece_of(const SeqArgs &q, int64_t slot) {
  Piece p;
  if (q.off == nullptr) {
    // (all below 2^31: a 64-bit division takes 150 instructions)
    const uint32_t per = (static_cast<uint32_t>(q.L) + static_cast<uint32_t>(q.chunk) - 1) / static_cast<uint32_t>(q.chunk);
    const uint32_t seq = static_cast<uint32_t>(slot) / per;
    p.seq = static_cast<int>(seq);
    p.c = static_cast<int>(static_cast<uint32_t>(slot) - seq * per);
    p.lo = seq * q.L;
    p.hi = p.lo + q.L;
  } else {
    const int lane = threadIdx.x % 64;
    int a = 0, n = q.nseq;                 // among sequences a .. a + n - 1
    while (n > 1) {
      const int step = (n + 63) / 64, at = a + lane * step;
      const bool before = lane * step < n && slots_before(q, at < q.nseq ? at : 0) + at <= slot;
      const uint64_t m = __ballot(before);
      const int k = m != 0 ? 63 - __builtin_clzll(m) : 0;
      n = n - k * step < step ? n - k * step : step;
      a += k * step;
    }
    p.seq = a;
    p.lo = clamped(q.off[a], q.L);
    p.hi = clamped(q.off[a + 1], q.L);
    p.c = static_cast<int>(slot - slots_before(q, a) - a);
  }
  p.id = slot;
  const int64_t all = p.hi - p.lo;
  p.count = all > q.chunk ? static_cast<int>((static_cast<uint32_t>(all) + static_cast<uint32_t>(q.chunk) - 1) /
                                             static_cast<uint32_t>(q.chunk)) : 1;
  p.t0 = p.lo + p.c * q.chunk;
  const int64_t left = p.hi - p.t0;
  p.len = static_cast<int>(left < q.chunk ? left : q.chunk);
  if (p.c < 0 || p.c >= p.count || p.len < 0) p.len = p.c == 0 && all <= 0 ? 0 : -1;
  return uniform(p);
}

// The same for a whole wave with up to 64 packed sequences, whose slots then go by
// falling length, so that no long sequence starts last.  PART: slots of all chunks (0),
// all but the last of several (1), or all but the first (2, of which there are at most L
// over the tokens of a chunk).
template <int PART = 0>
__device__ __forceinline__ Piece piece_by_length(const SeqArgs &q, int64_t slot) {
  if (q.off == nullptr || q.nseq > 64) return piece_of(q, slot);
  const int lane = threadIdx.x % 64;
  const bool has = lane < q.nseq;
  const int lo = has ? static_cast<int>(clamped(q.off[lane], q.L)) : 0;
  const int len = has ? static_cast<int>(clamped(q.off[lane + 1], q.L)) - lo : -1;
  const int chunk = static_cast<int>(q.chunk);
  const int count = !has ? 0 : len > chunk ? (len - 1) / chunk + 1 : 1;
  const int here = PART == 0 ? count : PART == 1 ? (count > 1 ? count - 1 : count) : (count > 1 ? count - 1 : 0);
  // (lengths past 2^24 in the sequences' order; no two keys alike)
  constexpr int kMost = 1 << 24;
  const int key = has ? (len < 0 ? 0 : len < kMost ? len : kMost) * 64 + 63 - lane : -1;
  int start = 0;
  for (int i = 0; i < q.nseq; ++i)
    start += __builtin_amdgcn_readlane(key, i) > key ? __builtin_amdgcn_readlane(here, i) : 0;
  Piece p;
  const uint64_t mine = __ballot(has && slot >= start && slot < start + here);
  p.seq = mine != 0 ? __builtin_ctzll(mine) : 0;
  p.lo = __builtin_amdgcn_readlane(lo, p.seq);
  const int all = __builtin_amdgcn_readlane(len, p.seq);
  p.hi = p.lo + (all > 0 ? all : 0);
  const int begin = __builtin_amdgcn_readlane(start, p.seq);
  p.count = __builtin_amdgcn_readlane(count, p.seq);
  if (PART == 0) {
    // (of offsets that overlap, sequences may have more chunks than there are slots)
    const int room = static_cast<int>(q.slots) - begin;
    p.count = p.count < room ? p.count : room;
  }
  p.c = static_cast<int>(slot) - begin + (PART == 2 ? 1 : 0);
  p.id = static_cast<uint32_t>(p.lo) / static_cast<uint32_t>(chunk) + p.seq + p.c;
  p.t0 = p.lo + static_cast<int64_t>(p.c) * chunk;
  const int64_t left = p.hi - p.t0;
  p.len = mine == 0 ? -1 : static_cast<int>(left < chunk ? left : chunk);
  return uniform(p);
}

// Sets the rows of `dim` values behind the last sequence to 0, by workgroup `block` of a launch's
// q.clear last ones.
template <typename T>
__device__ __forceinline__ void clear_rest(const SeqArgs &q, void *out, int64_t dim, int64_t block) {
  if (out == nullptr) return;
  T *p = static_cast<T *>(out);
  const int64_t first = clamped(q.off[q.nseq], q.L) * dim, end = q.L * dim, step = static_cast<int64_t>(q.clear) * blockDim.x;
  const int64_t me = block * blockDim.x + threadIdx.x;
  // whole pieces of 16 bytes, and what is left on either side of them
  constexpr int64_t kEach = 16 / sizeof(T);
  const int64_t skew = static_cast<int64_t>((reinterpret_cast<uintptr_t>(p + first) & 15) / sizeof(T));
  int64_t from = first + (skew != 0 ? kEach - skew : 0);
  from = from < end ? from : end;
  const int64_t pieces = (end - from) / kEach, to = from + pieces * kEach;
  typedef uint32_t Piece16 __attribute__((ext_vector_type(4)));
  for (int64_t i = me; i < pieces; i += step) reinterpret_cast<Piece16 *>(p + from)[i] = Piece16{0, 0, 0, 0};
  if (me < from - first) p[first + me] = T(0);
  if (me < end - to) p[to + me] = T(0);
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
// and states 4 q .. 4 q + 3, q = l / 16, so each row of 16 lanes wants the same four
// values of B and C.  Tokens go by in groups of 4.  What is one value per token and
// channel (dt, dt u, y, ...) lies with token q in lane (channel, q); a group's B and
// C with token s, state 4 q + i in lane 4 s + i of row q, from where a vector
// instruction's operand takes it to the whole row at once (DPP row_newbcast).
// (Matrix instructions that form the outer product and the sum over a lane's states
// are no help: a 4 x 4 x 1 product takes the SIMD 10 cycles, beside an exponential
// 15, and no vector instruction goes on meanwhile; four multiplications take 11 to 17.)
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Two states after everything before: what assembly text wrote may be read through DPP
// or a lane swap (whose waits the compiler counts for its own instructions only).
__device__ __forceinline__ void settle(float (&y)[4]) {
  asm("s_nop 1" : "+v"(y[0]), "+v"(y[1]), "+v"(y[2]), "+v"(y[3]));
}

// One token's update and read-out:  e[i] = 2^e[i],  r[i] = e[i] h[i] + b[4 S + i] x,
// y = sum_i c[4 S + i] r[i]  (y to be settled).  The state is rounded once a token.  In one
// piece, for the waits that the compiler does not count inside: an exponential's result may
// be read one state later, and what the last instruction before wrote (b or c) through DPP
// two states later.
#define VM_UPDATE_TEXT(A, B, C, D)                                                          \
  "v_exp_f32 %[e0], %[e0]\n"                                                                \
  "v_exp_f32 %[e1], %[e1]\n"                                                                \
  "v_exp_f32 %[e2], %[e2]\n"                                                                \
  "v_exp_f32 %[e3], %[e3]\n"                                                                \
  "v_mul_f32_dpp %[r0], %[b], %[x] row_newbcast:" #A " row_mask:0xf bank_mask:0xf\n"        \
  "v_mul_f32_dpp %[r1], %[b], %[x] row_newbcast:" #B " row_mask:0xf bank_mask:0xf\n"        \
  "v_mul_f32_dpp %[r2], %[b], %[x] row_newbcast:" #C " row_mask:0xf bank_mask:0xf\n"        \
  "v_mul_f32_dpp %[r3], %[b], %[x] row_newbcast:" #D " row_mask:0xf bank_mask:0xf\n"        \
  "v_fmac_f32 %[r0], %[h0], %[e0]\n"                                                        \
  "v_fmac_f32 %[r1], %[h1], %[e1]\n"                                                        \
  "v_fmac_f32 %[r2], %[h2], %[e2]\n"                                                        \
  "v_fmac_f32 %[r3], %[h3], %[e3]\n"
#define VM_UPDATE_OUT                                                                       \
  [r0] "=&v"(r[0]), [r1] "=&v"(r[1]), [r2] "=&v"(r[2]), [r3] "=&v"(r[3]), [e0] "+&v"(e[0]), \
      [e1] "+&v"(e[1]), [e2] "+&v"(e[2]), [e3] "+&v"(e[3])
#define VM_UPDATE_IN                                                                        \
  [h0] "v"(h[0]), [h1] "v"(h[1]), [h2] "v"(h[2]), [h3] "v"(h[3]), [b] "v"(b), [x] "v"(x)
template <int S> __device__ __forceinline__ void update(f32x4 &e, float b, float x, const f32x4 &h, f32x4 &r);
template <int S>
__device__ __forceinline__ float update_read(f32x4 &e, float b, float x, float c, const f32x4 &h, f32x4 &r);
#define VM_UPDATE(S, A, B, C, D)                                                            \
  template <>                                                                               \
  __device__ __forceinline__ void update<S>(f32x4 &e, float b, float x, const f32x4 &h, f32x4 &r) { \
    asm(VM_UPDATE_TEXT(A, B, C, D) : VM_UPDATE_OUT : VM_UPDATE_IN);                         \
  }                                                                                         \
  template <>                                                                               \
  __device__ __forceinline__ float update_read<S>(f32x4 &e, float b, float x, float c, const f32x4 &h, f32x4 &r) { \
    float y;                                                                                \
    asm(VM_UPDATE_TEXT(A, B, C, D)                                                          \
        "v_mul_f32_dpp %[y], %[c], %[r0] row_newbcast:" #A " row_mask:0xf bank_mask:0xf\n"  \
        "v_fmac_f32_dpp %[y], %[c], %[r1] row_newbcast:" #B " row_mask:0xf bank_mask:0xf\n" \
        "v_fmac_f32_dpp %[y], %[c], %[r2] row_newbcast:" #C " row_mask:0xf bank_mask:0xf\n" \
        "v_fmac_f32_dpp %[y], %[c], %[r3] row_newbcast:" #D " row_mask:0xf bank_mask:0xf\n" \
        : VM_UPDATE_OUT, [y] "=&v"(y)                                                       \
        : VM_UPDATE_IN, [c] "v"(c));                                                        \
    return y;                                                                               \
  }
VM_UPDATE(0, 0, 1, 2, 3) VM_UPDATE(1, 4, 5, 6, 7) VM_UPDATE(2, 8, 9, 10, 11) VM_UPDATE(3, 12, 13, 14, 15)
#undef VM_UPDATE
#undef VM_UPDATE_TEXT
#undef VM_UPDATE_OUT
#undef VM_UPDATE_IN

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
// Four values of each lane, summed over a channel's four lanes; lane
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
  uint32_t u, d, z, dense;            // token q of a tile (dense: of outputs and their gradients)
  uint32_t b, c;                      // B and C of a group: token (l / 4) % 4, state 4 q + l % 4
  uint32_t state[4];                  // in a block's [16][n]
  __device__ __forceinline__ bool has(int i) const { return state[i] != kOob; }   // a state in place i
};

// Places without a state hold 0 and read 0 for B and C, which leaves them 0 as long as every
// factor is finite.  What was formed with others is cleared by this.
__device__ __forceinline__ void clear_places(const Lane &l, f32x4 &x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = l.has(i) ? x[i] : 0.0f;
}
__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_inff(); }

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
  l.dense = at(l.live, a.dim, q, ch);
  const uint32_t state = 4 * q + lo;
  l.b = at(state < static_cast<uint32_t>(a.n), a.bs, hi, state);
  l.c = at(state < static_cast<uint32_t>(a.n), a.cs, hi, state);
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

// y = sum_i c[4 S + i] r[i], as in update_read.
template <int S>
__device__ __forceinline__ float read_out(float c, const f32x4 &r) {
  float y = row_bcast<4 * S>(c) * r[0];
  y = __builtin_fmaf(row_bcast<4 * S + 1>(c), r[1], y);
  y = __builtin_fmaf(row_bcast<4 * S + 2>(c), r[2], y);
  return __builtin_fmaf(row_bcast<4 * S + 3>(c), r[3], y);
}

// The step of a token, 0 past the chunk's end: such a step leaves the state as it is.
__device__ __forceinline__ float step_of(const PromptScanArgs &a, float x, bool in) {
  const float soft = softplus_f(x);
  const float dt = a.softplus ? soft : x;
  return in ? dt : 0.0f;
}

// One value rounded to nearest even (NaN stays NaN) and stored.
template <typename T>
__device__ __forceinline__ void put(Rsrc r, uint32_t off, float x) {
  if constexpr (sizeof(T) == 2)
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, static_cast<__bf16>(x)), r, static_cast<int>(off),
                                          0, 0);
  else
    bstore<T>(r, off, x);
}

// decay x + e for a decay over many tokens: it may round to 0 though none of its factors
// does, and an infinite x stays what it is.
__device__ __forceinline__ float carry(float decay, float x, float e) {
  return __builtin_fabsf(x) == __builtin_inff() ? x + e : __builtin_fmaf(decay, x, e);
}

// Joins chunks to x: x <- 2^(A2 t_j) x + e_j for the blocks j = first, first + step, ...
// of `many` (with loads of four under way).
__device__ __forceinline__ void join_chunks(const float *ends, const float *steps, int64_t first, int64_t step, int many,
                                            int lane, const float (&A2)[4], f32x4 &x) {
  int j = 0;
  for (; j + 4 <= many; j += 4) {
    f32x4 e[4];
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = first + (j + k) * step;
      e[k] = *reinterpret_cast<const f32x4 *>(ends + at * 256 + lane * 4);
      t[k] = steps[at * 16 + lane % 16];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = carry(hw_exp2(A2[i] * t[k]), x[i], e[k][i]);
  }
  for (; j < many; ++j) {
    const int64_t at = first + j * step;
    const f32x4 e = *reinterpret_cast<const f32x4 *>(ends + at * 256 + lane * 4);
    const float t = steps[at * 16 + lane % 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = carry(hw_exp2(A2[i] * t), x[i], e[i]);
  }
}

// Decay rates, ready for 2^x.  A rate of -Inf (which decays to 0 in any step) is
// held finite, so that the steps of 0 that fill up a group leave a state alone.
constexpr float kLeastRate2 = -3.0e38f;
__device__ __forceinline__ float rate2(float a) {
  const float r = a * kLog2e;
  return r < kLeastRate2 ? kLeastRate2 : r;      // (NaN stays)
}
// The same rate as a factor: times a decay of 0 it is 0.
__device__ __forceinline__ float rate(float a) {
  constexpr float least = kLeastRate2 / kLog2e;
  return a < least ? least : a;
}

}  // namespace
}  // namespace vmk
