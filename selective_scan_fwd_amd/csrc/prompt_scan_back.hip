// Gradients of the selective scan over rows of tokens.  With g_t the gradient of
// h_t, a_t = exp(dt A) and p_t = a_t g_t (the gradient of h_{t-1}):
//   dy = dout SiLU(z);   g_t = C_t dy_t + p_{t+1}
//   dC_t = sum_d dy h_t;  dB_t = sum_d dt u g_t;  w_t = sum_n g_t B_t
//   du = dt w + D dy;    ddt = u w + sum_n A p_t h_{t-1};  ddelta = ddt softplus'
//   dA = sum_t dt p_t h_{t-1};  dD = sum_t u dy;  dz = dout y SiLU'(z)
//
// The lane layout is the forward pass's (prompt_device.h).  A workgroup walks one
// chunk of four blocks of 16 channels: forward once, leaving the states at the
// starts of its tiles of 16 tokens in memory, then back over the tiles, whose
// states and decays are formed again and held in registers.  Where sequences have
// several chunks, a launch before it walks every chunk from a zero state and a zero
// gradient: with P_t the product of the decays from the chunk's start to t,
//   end state = sum over the chunk as forward,  gradient before it = sum P_t C_t dy_t,
// and each chunk joins what it needs from the chunks on either side.
// Sums over channels: 32 products of a group of 4 tokens are folded over the 16
// lanes of a row, halving the values at each step, then over the workgroup's waves
// in LDS; sums over blocks and chunks in a fixed order by launches of their own.
#include <hip/hip_runtime.h>

#include "prompt_device.h"

namespace vmk {
namespace {

constexpr int kGroups = kBackTile / 4;

// SiLU and its derivative.
__device__ __forceinline__ float silu_both(float z, float &slope) {
  const float s = hw_rcp(1.0f + hw_exp2(-z * kLog2e));
  slope = s * __builtin_fmaf(z, 1.0f - s, 1.0f);
  return z * s;
}

// ------------------------------------------------- chunks by themselves
// h[i] += b[4 S + i] x
template <int S> __device__ __forceinline__ void add_rank1(float b, float x, f32x4 &h);
#define VM_RANK1(S, A, B, C, D)                                                       \
  template <>                                                                         \
  __device__ __forceinline__ void add_rank1<S>(float b, float x, f32x4 &h) {          \
    asm("s_nop 1\n"                                                                   \
        "v_fmac_f32_dpp %0, %4, %5 row_newbcast:" #A " row_mask:0xf bank_mask:0xf\n"  \
        "v_fmac_f32_dpp %1, %4, %5 row_newbcast:" #B " row_mask:0xf bank_mask:0xf\n"  \
        "v_fmac_f32_dpp %2, %4, %5 row_newbcast:" #C " row_mask:0xf bank_mask:0xf\n"  \
        "v_fmac_f32_dpp %3, %4, %5 row_newbcast:" #D " row_mask:0xf bank_mask:0xf\n"  \
        : "+&v"(h[0]), "+&v"(h[1]), "+&v"(h[2]), "+&v"(h[3])                          \
        : "v"(b), "v"(x));                                                            \
  }
VM_RANK1(0, 0, 1, 2, 3) VM_RANK1(1, 4, 5, 6, 7) VM_RANK1(2, 8, 9, 10, 11) VM_RANK1(3, 12, 13, 14, 15)
#undef VM_RANK1
// g[i] += c[4 S + i] x[i]
template <int S> __device__ __forceinline__ void add_each(float c, const f32x4 &x, f32x4 &g);
#define VM_ADD_EACH(S, A, B, C, D)                                                    \
  template <>                                                                         \
  __device__ __forceinline__ void add_each<S>(float c, const f32x4 &x, f32x4 &g) {    \
    asm("s_nop 1\n"                                                                   \
        "v_fmac_f32_dpp %0, %4, %5 row_newbcast:" #A " row_mask:0xf bank_mask:0xf\n"  \
        "v_fmac_f32_dpp %1, %4, %6 row_newbcast:" #B " row_mask:0xf bank_mask:0xf\n"  \
        "v_fmac_f32_dpp %2, %4, %7 row_newbcast:" #C " row_mask:0xf bank_mask:0xf\n"  \
        "v_fmac_f32_dpp %3, %4, %8 row_newbcast:" #D " row_mask:0xf bank_mask:0xf\n"  \
        : "+&v"(g[0]), "+&v"(g[1]), "+&v"(g[2]), "+&v"(g[3])                          \
        : "v"(c), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]));                        \
  }
VM_ADD_EACH(0, 0, 1, 2, 3) VM_ADD_EACH(1, 4, 5, 6, 7) VM_ADD_EACH(2, 8, 9, 10, 11) VM_ADD_EACH(3, 12, 13, 14, 15)
#undef VM_ADD_EACH

template <int S>
__device__ __forceinline__ void local_token(const float (&A2)[4], float dt, float b, float du, float c, float dy, f32x4 &h,
                                            f32x4 &decay, f32x4 &grad) {
  f32x4 e;
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = dt * A2[i];
  update<S>(e, b, du, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) decay[i] *= e[i];
  f32x4 o = decay;                      // decay C dy: summed over the chunk
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= dy;
  add_each<S>(c, o, grad);
}

template <typename T>
__global__ __launch_bounds__(64 * kScanWaves) void scan_local_kernel(PromptScanArgs a, int wide) {
  const int lane = threadIdx.x % 64, blocks = (a.dim + 15) / 16;
  const int64_t slot = blockIdx.x / wide;
  const int blk = uniform(static_cast<int>(blockIdx.x % wide) * kScanWaves + threadIdx.x / 64);
  if (blk >= blocks) return;
  const Piece p = piece_of(a.q, slot);
  if (p.len <= 0 || p.count == 1) return;
  const int c0 = blk * 16;
  const Lane l = lane_of<T>(a, c0, lane);
  float A2[4];
  const Rsrc rA = make_rsrc(a.A + static_cast<int64_t>(c0) * a.n, l.cw * a.n * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = rate2(bload<float>(rA, l.state[i]));
  const float bias = channel_value(a.bias, c0, l);
  const uint32_t doff = l.live ? (l.q * static_cast<uint32_t>(a.dim) + l.ch) * sizeof(T) : kOob;
  f32x4 h = {0, 0, 0, 0}, decay = {1, 1, 1, 1}, grad = {0, 0, 0, 0};
  float steps = 0.0f;
  for (int at = 0; at < p.len; at += kBackTile) {
    const int m = p.len - at < kBackTile ? p.len - at : kBackTile;
    const int64_t t = p.t0 + at;
    const Rsrc ru = rows<T>(a.u, a.us, t, c0, m, l.cw), rd = rows<T>(a.delta, a.ds, t, c0, m, l.cw),
               rb = rows<T>(a.B, a.bs, t, 0, m, a.n), rc = rows<T>(a.C, a.cs, t, 0, m, a.n),
               ro = rows<T>(a.dout, a.dim, t, c0, m, l.cw),
               rz = rows<T>(a.z, a.zs, t, c0, a.z != nullptr ? m : 0, l.cw);
    float u[kGroups], d[kGroups], b[kGroups], c[kGroups], o[kGroups], z[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      u[g] = bload<T>(ru, l.u + g * static_cast<uint32_t>(4 * a.us * sizeof(T)));
      d[g] = bload<T>(rd, l.d + g * static_cast<uint32_t>(4 * a.ds * sizeof(T)));
      b[g] = bload<T>(rb, l.b + g * static_cast<uint32_t>(4 * a.bs * sizeof(T)));
      c[g] = bload<T>(rc, l.c + g * static_cast<uint32_t>(4 * a.cs * sizeof(T)));
      o[g] = bload<T>(ro, doff + g * static_cast<uint32_t>(4 * a.dim * sizeof(T)));
      z[g] = bload<T>(rz, l.z + g * static_cast<uint32_t>(4 * a.zs * sizeof(T)));
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (4 * g >= m) break;
      const float dt = step_of(a, d[g] + bias, 4 * g + l.q < m), du = dt * u[g];
      const float dy = a.z != nullptr ? o[g] * silu_f(z[g]) : o[g];
      steps += dt;
      float dts[4], dus[4], dys[4];
      hand_out(dt, dts);
      hand_out(du, dus);
      hand_out(dy, dys);
      local_token<0>(A2, dts[0], b[g], dus[0], c[g], dys[0], h, decay, grad);
      local_token<1>(A2, dts[1], b[g], dus[1], c[g], dys[1], h, decay, grad);
      local_token<2>(A2, dts[2], b[g], dus[2], c[g], dys[2], h, decay, grad);
      local_token<3>(A2, dts[3], b[g], dus[3], c[g], dys[3], h, decay, grad);
    }
  }
  const int64_t block = slot * blocks + blk;
  const float s[4] = {steps, steps, steps, steps};
  steps = gather(s);
  *reinterpret_cast<f32x4 *>(a.ends + block * 256 + lane * 4) = h;
  *reinterpret_cast<f32x4 *>(a.starts + block * 256 + lane * 4) = grad;
  if (l.q == 0) a.steps[block * 16 + l.ch] = steps;
}

// ------------------------------------------------------------ folding
// r = a + a of lane ^ 8 in lanes 0 .. 7 of a row, b + b of lane ^ 8 in the others.
// (s_nop: a vector instruction's result may be read by another lane two states later.)
__device__ __forceinline__ void fold8(const float (&a)[4], const float (&b)[4], float (&r)[4]) {
  asm("s_nop 1\n"
      "v_add_f32_dpp %0, %4, %4 row_ror:8 row_mask:0xf bank_mask:0x3\n"
      "v_add_f32_dpp %1, %5, %5 row_ror:8 row_mask:0xf bank_mask:0x3\n"
      "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n"
      "v_add_f32_dpp %3, %7, %7 row_ror:8 row_mask:0xf bank_mask:0x3\n"
      "v_add_f32_dpp %0, %8, %8 row_ror:8 row_mask:0xf bank_mask:0xc\n"
      "v_add_f32_dpp %1, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xc\n"
      "v_add_f32_dpp %2, %10, %10 row_ror:8 row_mask:0xf bank_mask:0xc\n"
      "v_add_f32_dpp %3, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xc\n"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]));
}
// The same within each half row with lane 7 - l: a in lanes 0 .. 3, b in 4 .. 7.
__device__ __forceinline__ void fold4(const float (&a)[4], const float (&b)[4], float (&r)[4]) {
  asm("s_nop 1\n"
      "v_add_f32_dpp %0, %4, %4 row_half_mirror row_mask:0xf bank_mask:0x5\n"
      "v_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0x5\n"
      "v_add_f32_dpp %2, %6, %6 row_half_mirror row_mask:0xf bank_mask:0x5\n"
      "v_add_f32_dpp %3, %7, %7 row_half_mirror row_mask:0xf bank_mask:0x5\n"
      "v_add_f32_dpp %0, %8, %8 row_half_mirror row_mask:0xf bank_mask:0xa\n"
      "v_add_f32_dpp %1, %9, %9 row_half_mirror row_mask:0xf bank_mask:0xa\n"
      "v_add_f32_dpp %2, %10, %10 row_half_mirror row_mask:0xf bank_mask:0xa\n"
      "v_add_f32_dpp %3, %11, %11 row_half_mirror row_mask:0xf bank_mask:0xa\n"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]));
}
template <int CTRL>
__device__ __forceinline__ float fold_quad(float a, float b, bool second) {
  const float x = a + __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(a), CTRL, 0xf, 0xf, true));
  const float y = b + __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(b), CTRL, 0xf, 0xf, true));
  return second ? y : x;
}
// x[s][i], y[s][i]: products of token s and this lane's state i.  Summed over the 16
// lanes of a row, lane l gets (l & 8 ? y : x) of token (l >> 1) & 3 and states
// 2 (l & 1) + {0, 1}.
__device__ __forceinline__ void fold(const float (&x)[4][4], const float (&y)[4][4], int lane, float (&r)[2]) {
  float a[4][4], b[2][4], c[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) fold8(x[s], y[s], a[s]);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    fold4(a[s], a[s + 2], b[s]);
    settle(b[s]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = fold_quad<0x4e>(b[0][i], b[1][i], (lane & 2) != 0);   // lane ^ 2
#pragma unroll
  for (int i = 0; i < 2; ++i) r[i] = fold_quad<0xb1>(c[i], c[i + 2], (lane & 1) != 0);     // lane ^ 1
}

// ------------------------------------------------------- a chunk's gradients
template <int S>
__device__ __forceinline__ void again(const float (&A2)[4], float dt, float b, float du, f32x4 &h, f32x4 &decay) {
#pragma unroll
  for (int i = 0; i < 4; ++i) decay[i] = dt * A2[i];
  update<S>(decay, b, du, h);
}

template <int S, bool GATE>
__device__ __forceinline__ void back_token(const float (&A)[4], float dts, float dus, float dys, float b, float c,
                                           const f32x4 &decay, const f32x4 &h, const f32x4 &before, f32x4 &p,
                                           float (&dA)[4], float (&x)[4], float (&yy)[4], float &w, float &through,
                                           float &y) {
  f32x4 g = p;
  add_rank1<S>(c, dys, g);
  w = read_out<S>(b, g);
  if (GATE) y = read_out<S>(c, h);
  through = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = g[i] * dus;
    yy[i] = h[i] * dys;
    p[i] = decay[i] * g[i];
    const float m = p[i] * before[i];
    dA[i] = __builtin_fmaf(m, dts, dA[i]);
    through = __builtin_fmaf(m, A[i], through);
  }
}

template <typename T, bool GATE>
__global__ __launch_bounds__(64 * kScanWaves, 2) void scan_back_kernel(PromptScanArgs a, int wide) {
  __shared__ float sums[2][kScanWaves][kBackTile * 32];
  const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), blocks = (a.dim + 15) / 16, padded = wide * kScanWaves;
  const int64_t slot = blockIdx.x / wide;
  const int group = blockIdx.x % wide, blk = group * kScanWaves + wave;
  Piece p = piece_of(a.q, slot);
  const bool none = p.len < 0;         // a slot without a chunk: its partial sums are 0
  if (none) {
    p.seq = p.c = p.len = 0;
    p.count = 1;
    p.t0 = 0;
  }
  // (waves past the last block have no channels; they keep the others' barriers)
  const int c0 = blk * 16;
  const Lane l = lane_of<T>(a, c0, lane);
  float A[4], A2[4], dA[4] = {0, 0, 0, 0};
  const Rsrc rA = make_rsrc(a.A + static_cast<int64_t>(c0) * a.n, l.cw * a.n * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    A[i] = bload<float>(rA, l.state[i]);
    A2[i] = rate2(A[i]);
  }
  const float bias = channel_value(a.bias, c0, l), D = channel_value(a.D, c0, l);
  const uint32_t doff = l.live ? (l.q * static_cast<uint32_t>(a.dim) + l.ch) * sizeof(T) : kOob,
                 dstep = 4 * static_cast<uint32_t>(a.dim) * sizeof(T);

  // the state before the chunk and the gradient of the one after it
  f32x4 h = {0, 0, 0, 0}, grad = {0, 0, 0, 0};
  const int64_t sbase = (static_cast<int64_t>(p.seq) * a.dim + c0) * a.n;
  if (a.h0 != nullptr) {
    const Rsrc r = make_rsrc(a.h0 + sbase, l.cw * a.n * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = bload<float>(r, l.state[i]);
  }
  if (a.dstate != nullptr) {
    const Rsrc r = make_rsrc(a.dstate + sbase, l.cw * a.n * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) grad[i] = bload<float>(r, l.state[i]);
  }
  if (p.count > 1 && blk < blocks) {
    const int64_t first = (slot - p.c) * blocks + blk;
    for (int j = 0; j < p.c; ++j) {
      const int64_t at = first + static_cast<int64_t>(j) * blocks;
      const f32x4 e = *reinterpret_cast<const f32x4 *>(a.ends + at * 256 + lane * 4);
      const float t = a.steps[at * 16 + l.ch];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __builtin_fmaf(hw_exp2(A2[i] * t), h[i], e[i]);
    }
    for (int j = p.count - 1; j > p.c; --j) {
      const int64_t at = first + static_cast<int64_t>(j) * blocks;
      const f32x4 e = *reinterpret_cast<const f32x4 *>(a.starts + at * 256 + lane * 4);
      const float t = a.steps[at * 16 + l.ch];
#pragma unroll
      for (int i = 0; i < 4; ++i) grad[i] = __builtin_fmaf(hw_exp2(A2[i] * t), grad[i], e[i]);
    }
  }

  // forward: the states at the tiles' starts
  const int tiles = (p.len + kBackTile - 1) / kBackTile;
  float *mark = a.marks + ((p.t0 / kBackTile + slot) * padded + blk) * 256 + lane * 4;
  const int64_t mstep = static_cast<int64_t>(padded) * 256;
  for (int tile = 0; tile + 1 < tiles; ++tile) {
    *reinterpret_cast<f32x4 *>(mark + tile * mstep) = h;
    const int64_t t = p.t0 + tile * kBackTile;
    const Rsrc ru = rows<T>(a.u, a.us, t, c0, kBackTile, l.cw), rd = rows<T>(a.delta, a.ds, t, c0, kBackTile, l.cw),
               rb = rows<T>(a.B, a.bs, t, 0, kBackTile, a.n);
    float u[kGroups], d[kGroups], b[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      u[g] = bload<T>(ru, l.u + g * static_cast<uint32_t>(4 * a.us * sizeof(T)));
      d[g] = bload<T>(rd, l.d + g * static_cast<uint32_t>(4 * a.ds * sizeof(T)));
      b[g] = bload<T>(rb, l.b + g * static_cast<uint32_t>(4 * a.bs * sizeof(T)));
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float dt = step_of(a, d[g] + bias, true), du = dt * u[g];
      float dts[4], dus[4];
      f32x4 e;
      hand_out(dt, dts);
      hand_out(du, dus);
      again<0>(A2, dts[0], b[g], dus[0], h, e);
      again<1>(A2, dts[1], b[g], dus[1], h, e);
      again<2>(A2, dts[2], b[g], dus[2], h, e);
      again<3>(A2, dts[3], b[g], dus[3], h, e);
    }
  }

  float dD = 0.0f, dbias = 0.0f;
  for (int tile = tiles - 1; tile >= 0; --tile) {
    const int64_t t = p.t0 + tile * kBackTile;
    const int m = p.len - tile * kBackTile < kBackTile ? p.len - tile * kBackTile : kBackTile;
    const Rsrc ru = rows<T>(a.u, a.us, t, c0, m, l.cw), rd = rows<T>(a.delta, a.ds, t, c0, m, l.cw),
               rb = rows<T>(a.B, a.bs, t, 0, m, a.n), rc = rows<T>(a.C, a.cs, t, 0, m, a.n),
               ro = rows<T>(a.dout, a.dim, t, c0, m, l.cw), rz = rows<T>(a.z, a.zs, t, c0, GATE ? m : 0, l.cw);
    float u[kGroups], d[kGroups], b[kGroups], c[kGroups], o[kGroups], z[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      u[g] = bload<T>(ru, l.u + g * static_cast<uint32_t>(4 * a.us * sizeof(T)));
      d[g] = bload<T>(rd, l.d + g * static_cast<uint32_t>(4 * a.ds * sizeof(T)));
      b[g] = bload<T>(rb, l.b + g * static_cast<uint32_t>(4 * a.bs * sizeof(T)));
      c[g] = bload<T>(rc, l.c + g * static_cast<uint32_t>(4 * a.cs * sizeof(T)));
      o[g] = bload<T>(ro, doff + g * dstep);
      if (GATE) {
        z[g] = bload<T>(rz, l.z + g * static_cast<uint32_t>(4 * a.zs * sizeof(T)));
      }
    }
    if (tile + 1 < tiles) h = *reinterpret_cast<const f32x4 *>(mark + tile * mstep);
    const f32x4 begin = h;
    f32x4 hs[kBackTile], es[kBackTile];
    float dt[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      dt[g] = step_of(a, d[g] + bias, 4 * g + l.q < m);
      const float du = dt[g] * u[g];
      float dts[4], dus[4];
      hand_out(dt[g], dts);
      hand_out(du, dus);
      again<0>(A2, dts[0], b[g], dus[0], h, es[4 * g]);
      hs[4 * g] = h;
      again<1>(A2, dts[1], b[g], dus[1], h, es[4 * g + 1]);
      hs[4 * g + 1] = h;
      again<2>(A2, dts[2], b[g], dus[2], h, es[4 * g + 2]);
      hs[4 * g + 2] = h;
      again<3>(A2, dts[3], b[g], dus[3], h, es[4 * g + 3]);
      hs[4 * g + 3] = h;
    }
    float *mine = sums[tile & 1][wave];
    const Rsrc rdu = rows<T>(a.du, a.dim, t, c0, m, l.cw), rdd = rows<T>(a.ddelta, a.dim, t, c0, m, l.cw),
               rdz = rows<T>(a.dz, a.dim, t, c0, GATE ? m : 0, l.cw);
#pragma unroll
    for (int g = kGroups - 1; g >= 0; --g) {
      if (4 * g >= m) continue;
      const bool in = 4 * g + l.q < m;
      const float du = dt[g] * u[g];
      float slope = 0.0f, dy = o[g];
      if (GATE) dy *= silu_both(z[g], slope);
      float dts[4], dus[4], dys[4], x[4][4], yy[4][4], w[4], th[4], y[4];
      hand_out(dt[g], dts);
      hand_out(du, dus);
      hand_out(dy, dys);
      back_token<3, GATE>(A, dts[3], dus[3], dys[3], b[g], c[g], es[4 * g + 3], hs[4 * g + 3], hs[4 * g + 2],
                          grad, dA, x[3], yy[3], w[3], th[3], y[3]);
      back_token<2, GATE>(A, dts[2], dus[2], dys[2], b[g], c[g], es[4 * g + 2], hs[4 * g + 2], hs[4 * g + 1],
                          grad, dA, x[2], yy[2], w[2], th[2], y[2]);
      back_token<1, GATE>(A, dts[1], dus[1], dys[1], b[g], c[g], es[4 * g + 1], hs[4 * g + 1], hs[4 * g],
                          grad, dA, x[1], yy[1], w[1], th[1], y[1]);
      back_token<0, GATE>(A, dts[0], dus[0], dys[0], b[g], c[g], es[4 * g], hs[4 * g],
                          g > 0 ? hs[g > 0 ? 4 * g - 1 : 0] : begin, grad, dA, x[0], yy[0], w[0], th[0], y[0]);
      settle(w);
      if (GATE) settle(y);
      const float along = gather(w), through = gather(th);
      if (GATE) {
        const float yt = __builtin_fmaf(D, u[g], gather(y));
        put<T>(rdz, doff + g * dstep, o[g] * yt * slope);
      }
      put<T>(rdu, doff + g * dstep, __builtin_fmaf(along, dt[g], D * dy));
      float dd = __builtin_fmaf(along, u[g], through);
      const float slope2 = hw_rcp(1.0f + hw_exp2((d[g] + bias) * -kLog2e));
      dd *= a.softplus ? slope2 : 1.0f;
      put<T>(rdd, doff + g * dstep, dd);
      dD = __builtin_fmaf(dy, u[g], dD);
      dbias += in ? dd : 0.0f;
      float r[2];
      fold(x, yy, lane, r);
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const int at = (4 * g + ((lane >> 1) & 3)) * 32 + (lane & 8) * 2 + 4 * l.q + 2 * (lane & 1);
      *reinterpret_cast<f32x2 *>(mine + at) = f32x2{r[0], r[1]};
    }
    // (the other tile's sums may still be read by waves behind this barrier)
    __syncthreads();
    for (int i = threadIdx.x; i < kBackTile * 32; i += 64 * kScanWaves) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kScanWaves; ++w) s += sums[tile & 1][w][i];
      const int tok = i / 32, which = (i / 16) % 2, n = i % 16;
      if (tok < m && n < a.n) a.partBC[((group * a.q.L * (a.q.off != nullptr ? 1 : a.q.nseq) + t + tok) * 2 + which) * a.n + n] = s;
    }
    h = begin;
  }

  if (p.c == 0 && !none && a.dh0 != nullptr) {
    const Rsrc r = make_rsrc(a.dh0 + sbase, l.cw * a.n * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) bstore<float>(r, l.state[i], grad[i]);
  }
  const Rsrc rpA = make_rsrc(a.partA + (slot * a.dim + c0) * a.n, l.cw * a.n * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) bstore<float>(rpA, l.state[i], dA[i]);
  const float sD[4] = {dD, dD, dD, dD}, sb[4] = {dbias, dbias, dbias, dbias};
  dD = gather(sD);
  dbias = gather(sb);
  if (l.live && l.q == 0) {
    a.partD[slot * 2 * a.dim + c0 + l.ch] = dD;
    a.partD[(slot * 2 + 1) * a.dim + c0 + l.ch] = dbias;
  }
}

// dB and dC: the sums over the workgroups' blocks.
template <typename T>
__global__ __launch_bounds__(256) void scan_back_sum_kernel(PromptScanArgs a, int wide, int64_t tokens) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x;
  const int64_t per = tokens * 2 * a.n;
  if (i >= per) return;
  const int64_t tok = i / (2 * a.n);
  const int col = static_cast<int>(i - tok * 2 * a.n);
  if (a.q.off != nullptr && tok >= clamped(a.q.off[a.q.nseq], a.q.L)) return;
  float s = 0.0f;
  for (int g = 0; g < wide; ++g) s += a.partBC[g * per + i];
  T *out = static_cast<T *>(col < a.n ? a.dB : a.dC);
  out[tok * a.n + (col < a.n ? col : col - a.n)] = from_f32<T>(s);
}

template <typename T>
hipError_t launch_back(const PromptScanArgs &a, hipStream_t s) {
  const int wide = scan_wide(a.dim);
  const dim3 grid(static_cast<uint32_t>(a.q.slots * wide));
  const int64_t tokens = a.q.L * (a.q.off != nullptr ? 1 : a.q.nseq);
  if (a.ends != nullptr) scan_local_kernel<T><<<grid, 64 * kScanWaves, 0, s>>>(a, wide);
  if (a.z != nullptr)
    scan_back_kernel<T, true><<<grid, 64 * kScanWaves, 0, s>>>(a, wide);
  else
    scan_back_kernel<T, false><<<grid, 64 * kScanWaves, 0, s>>>(a, wide);
  scan_back_sum_kernel<T><<<static_cast<uint32_t>((tokens * 2 * a.n + 255) / 256), 256, 0, s>>>(a, wide, tokens);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prompt_scan_back(const PromptScanArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? launch_back<bf16_t>(a, s) : launch_back<float>(a, s);
}

}  // namespace vmk
