// Gradients of the selective scan over rows of tokens.  With g_t the gradient of
// h_t, a_t = exp(dt A) and p_t = a_t g_t (the gradient of h_{t-1}):
//   dy = dout SiLU(z);   g_t = C_t dy_t + p_{t+1}
//   dC_t = sum_d dy h_t;  dB_t = sum_d dt u g_t;  w_t = sum_n g_t B_t
//   du = dt w + D dy;    ddt = u w + sum_n A p_t h_{t-1};  ddelta = ddt softplus'
//   dA = sum_t dt p_t h_{t-1};  dD = sum_t u dy;  dz = dout y SiLU'(z)
//
// The lane layout is the forward pass's (prompt_device.h).  A first launch walks every
// chunk forward and leaves the states at the starts of its tiles of 8 tokens in memory.
// The second walks back over the tiles, a workgroup over one chunk of four blocks of 16
// channels: a tile's states and decays are formed again and held in registers.  Where
// sequences have several chunks, the first launch starts each of them from a zero state
// and gathers the gradient of the state before it besides; with P_t the product of the
// decays from the chunk's start to t,
//   end state = sum over the chunk as forward,  gradient before it = sum P_t C_t dy_t,
// and the second launch joins what a chunk needs from those on either side of it.
// Sums over channels: 32 products of a group of 4 tokens are folded over the 16
// lanes of a row, halving the values at each step, then over the workgroup's waves
// in LDS; sums over blocks and chunks in a fixed order by launches of their own.
// Bound by vector instructions: 88 a wave and token in the second launch (92 with chunks to
// join), 38 in the first with the gathered gradients and 20 without.  128 x 197 tokens of 384
// channels, fp32: 40 and 135 us; 2 x 4097 of 2048, bf16, in chunks: 106 and 236 us.
// A tile of 8 tokens has places for 16 states of 16 channels.  What fills them up is 0, which
// adds nothing as long as what it meets is finite: tiles with other values, and those that a
// chunk's tokens do not fill, are walked with every sum restricted to what there is.
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
  f32x4 r;
  update<S>(e, b, du, h, r);
  h = r;
#pragma unroll
  for (int i = 0; i < 4; ++i) decay[i] *= e[i];
  f32x4 o = decay;                      // decay C dy: summed over the chunk
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= dy;
  add_each<S>(c, o, grad);
}

// The state after a token, r, from the one before it, and its decays.
template <int S>
__device__ __forceinline__ void again(const float (&A2)[4], float dt, float b, float du, const f32x4 &h, f32x4 &r, f32x4 &decay) {
#pragma unroll
  for (int i = 0; i < 4; ++i) decay[i] = dt * A2[i];
  f32x4 to;
  update<S>(decay, b, du, h, to);
  r = to;
}

// What a tile's tokens bring, as loaded.
struct Raw {
  float u[kGroups], d[kGroups], b[kGroups], c[kGroups], o[kGroups], z[kGroups];
};
template <typename T, bool ALL, bool GATE>
__device__ __forceinline__ void load_tile(const PromptScanArgs &a, const Lane &l, int64_t t, int left, int c0, Raw &r) {
  const int m = left < kBackTile ? left : kBackTile;
  const Rsrc ru = rows<T>(a.u, a.us, t, c0, m, l.cw), rd = rows<T>(a.delta, a.ds, t, c0, m, l.cw),
             rb = rows<T>(a.B, a.bs, t, 0, m, a.n);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    r.u[g] = bload<T>(ru, l.u + g * static_cast<uint32_t>(4 * a.us * sizeof(T)));
    r.d[g] = bload<T>(rd, l.d + g * static_cast<uint32_t>(4 * a.ds * sizeof(T)));
    r.b[g] = bload<T>(rb, l.b + g * static_cast<uint32_t>(4 * a.bs * sizeof(T)));
  }
  if (!ALL) return;
  const Rsrc rc = rows<T>(a.C, a.cs, t, 0, m, a.n), ro = rows<T>(a.dout, a.dim, t, c0, m, l.cw),
             rz = rows<T>(a.z, a.zs, t, c0, GATE ? m : 0, l.cw);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    r.c[g] = bload<T>(rc, l.c + g * static_cast<uint32_t>(4 * a.cs * sizeof(T)));
    r.o[g] = bload<T>(ro, l.dense + g * static_cast<uint32_t>(4 * a.dim * sizeof(T)));
    if (GATE) r.z[g] = bload<T>(rz, l.z + g * static_cast<uint32_t>(4 * a.zs * sizeof(T)));
  }
}

// Walks a chunk forward from state h.  MANY: one of several of its sequence, from zero.
template <typename T, bool GATE, bool MANY>
__device__ __forceinline__ void mark_chunk(const PromptScanArgs &a, const Lane &l, const Piece &p, int64_t slot, int blk,
                                           int lane, const float (&A2)[4], float bias, f32x4 h, float (*meet)[16][12]) {
  const int blocks = (a.dim + 15) / 16, c0 = blk * 16;
  const int64_t first = (p.t0 / kBackTile + p.id) * blocks + blk;
  float *mark = a.marks + first * 256 + lane * 4, *before = a.before + first * 16 + l.ch;
  const int64_t mstep = static_cast<int64_t>(blocks) * 256;
  f32x4 decay = {1, 1, 1, 1}, grad = {0, 0, 0, 0};
  float steps = 0.0f;
  Raw next;
  load_tile<T, MANY, GATE>(a, l, p.t0, p.len, c0, next);
  // (nobody asks for the state after a sequence's last tile)
  const int end = MANY ? p.len : p.len - kBackTile;
  for (int at = 0; at < end; at += kBackTile) {
    const Raw r = next;
    const int m = p.len - at;
    load_tile<T, MANY, GATE>(a, l, p.t0 + at + kBackTile, m - kBackTile, c0, next);
    *reinterpret_cast<f32x4 *>(mark) = h;
    mark += mstep;
    if (MANY) {
      if (l.q == 0) *before = steps;
      before += blocks * 16;
    }
    float mine = 0.0f, size = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float dt = step_of(a, r.d[g] + bias, 4 * g + l.q < m);
      meet[g][l.ch][2 * l.q] = dt;
      meet[g][l.ch][2 * l.q + 1] = dt * r.u[g];
      if (MANY) {
        const float dy = GATE ? r.o[g] * silu_f(r.z[g]) : r.o[g];
        meet[g][l.ch][8 + l.q] = dy;
        size += __builtin_fabsf(dy);
        mine += dt;
      }
    }
    wave_lds_fence();
    if (MANY && uniform(__ballot(!finite(size)) != 0) != 0) {
      // an infinite gradient stays one, though the decays before it may have rounded to 0
      bool all = true;
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int s = 0; s < 4; ++s) all = all && finite(meet[g][l.ch][8 + s]);
#pragma unroll
      for (int i = 0; i < 4; ++i) decay[i] = all ? decay[i] : 1.0f;
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const auto &w = meet[g][l.ch];
      if (MANY) {
        local_token<0>(A2, w[0], r.b[g], w[1], r.c[g], w[8], h, decay, grad);
        local_token<1>(A2, w[2], r.b[g], w[3], r.c[g], w[9], h, decay, grad);
        local_token<2>(A2, w[4], r.b[g], w[5], r.c[g], w[10], h, decay, grad);
        local_token<3>(A2, w[6], r.b[g], w[7], r.c[g], w[11], h, decay, grad);
      } else {
        f32x4 e;
        again<0>(A2, w[0], r.b[g], w[1], h, h, e);
        again<1>(A2, w[2], r.b[g], w[3], h, h, e);
        again<2>(A2, w[4], r.b[g], w[5], h, h, e);
        again<3>(A2, w[6], r.b[g], w[7], h, h, e);
      }
    }
    wave_lds_fence();
    if (MANY) {
      const float s[4] = {mine, mine, mine, mine};
      steps += gather(s);
    }
  }
  if (!MANY) *reinterpret_cast<f32x4 *>(mark) = h;
  if (MANY) {
    const int64_t block = slot * blocks + blk;
    *reinterpret_cast<f32x4 *>(a.ends + block * 256 + lane * 4) = h;
    *reinterpret_cast<f32x4 *>(a.starts + block * 256 + lane * 4) = grad;
    if (l.q == 0) a.steps[block * 16 + l.ch] = steps;
  }
}

template <typename T, bool GATE>
__global__ __launch_bounds__(64 * kScanWaves) void scan_marks_kernel(PromptScanArgs a, int wide) {
  __shared__ __align__(16) float meets[kScanWaves][kGroups][16][12];
  const int lane = threadIdx.x % 64, blocks = (a.dim + 15) / 16;
  const int64_t slot = blockIdx.x / wide;
  if (slot >= a.q.slots) {
    for (void *rows : {a.du, a.ddelta, a.dz}) clear_rest<T>(a.q, rows, a.dim, blockIdx.x - a.q.slots * wide);
    return;
  }
  const int blk = uniform(static_cast<int>(blockIdx.x % wide) * kScanWaves + threadIdx.x / 64);
  if (blk >= blocks) return;
  const Piece p = piece_by_length(a.q, slot);
  if (p.len <= 0) return;
  const int c0 = blk * 16;
  const Lane l = lane_of<T>(a, c0, lane);
  float A2[4];
  const Rsrc rA = make_rsrc(a.A + static_cast<int64_t>(c0) * a.n, l.cw * a.n * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = rate2(bload<float>(rA, l.state[i]));
  const float bias = channel_value(a.bias, c0, l);
  f32x4 h = {0, 0, 0, 0};
  if (p.count > 1) {
    mark_chunk<T, GATE, true>(a, l, p, slot, blk, lane, A2, bias, h, meets[threadIdx.x / 64]);
    return;
  }
  if (a.h0 != nullptr) {
    const Rsrc r = make_rsrc(a.h0 + (static_cast<int64_t>(p.seq) * a.dim + c0) * a.n, l.cw * a.n * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = bload<float>(r, l.state[i]);
  }
  mark_chunk<T, GATE, false>(a, l, p, slot, blk, lane, A2, bias, h, meets[threadIdx.x / 64]);
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
// yy[i] = h[i] dy,  g[i] += c[4 S + i] dy,  w = sum_i b[4 S + i] g[i], and with READ
// y = sum_i c[4 S + i] h[i]  (w and y to be settled; the four products before the first
// DPP operand are its two states, for b and c).
template <int S, bool READ>
__device__ __forceinline__ void back_sums(float dy, float b, float c, const f32x4 &h, f32x4 &g, float (&yy)[4], float &w, float &y);
#define VM_BACK_TEXT(A, B, C, D)                                                                   \
  "v_mul_f32 %[m0], %[h0], %[dy]\n"                                                                \
  "v_mul_f32 %[m1], %[h1], %[dy]\n"                                                                \
  "v_mul_f32 %[m2], %[h2], %[dy]\n"                                                                \
  "v_mul_f32 %[m3], %[h3], %[dy]\n"                                                                \
  "v_fmac_f32_dpp %[g0], %[c], %[dy] row_newbcast:" #A " row_mask:0xf bank_mask:0xf\n"             \
  "v_fmac_f32_dpp %[g1], %[c], %[dy] row_newbcast:" #B " row_mask:0xf bank_mask:0xf\n"             \
  "v_fmac_f32_dpp %[g2], %[c], %[dy] row_newbcast:" #C " row_mask:0xf bank_mask:0xf\n"             \
  "v_fmac_f32_dpp %[g3], %[c], %[dy] row_newbcast:" #D " row_mask:0xf bank_mask:0xf\n"
#define VM_BACK_W(OP, I, L) "v_" OP "_f32_dpp %[w], %[b], %[g" #I "] row_newbcast:" #L " row_mask:0xf bank_mask:0xf\n"
#define VM_BACK_Y(OP, I, L) "v_" OP "_f32_dpp %[y], %[c], %[h" #I "] row_newbcast:" #L " row_mask:0xf bank_mask:0xf\n"
#define VM_BACK_OUT                                                                                \
  [g0] "+&v"(g[0]), [g1] "+&v"(g[1]), [g2] "+&v"(g[2]), [g3] "+&v"(g[3]), [m0] "=&v"(yy[0]),       \
      [m1] "=&v"(yy[1]), [m2] "=&v"(yy[2]), [m3] "=&v"(yy[3]), [w] "=&v"(w)
#define VM_BACK_IN                                                                                 \
  [h0] "v"(h[0]), [h1] "v"(h[1]), [h2] "v"(h[2]), [h3] "v"(h[3]), [b] "v"(b), [c] "v"(c), [dy] "v"(dy)
#define VM_BACK(S, A, B, C, D)                                                                     \
  template <>                                                                                      \
  __device__ __forceinline__ void back_sums<S, false>(float dy, float b, float c, const f32x4 &h, f32x4 &g, \
                                                      float (&yy)[4], float &w, float &) {         \
    asm(VM_BACK_TEXT(A, B, C, D) VM_BACK_W("mul", 0, A) VM_BACK_W("fmac", 1, B)                    \
        VM_BACK_W("fmac", 2, C) VM_BACK_W("fmac", 3, D) : VM_BACK_OUT : VM_BACK_IN);               \
  }                                                                                                \
  template <>                                                                                      \
  __device__ __forceinline__ void back_sums<S, true>(float dy, float b, float c, const f32x4 &h, f32x4 &g, \
                                                     float (&yy)[4], float &w, float &y) {         \
    asm(VM_BACK_TEXT(A, B, C, D) VM_BACK_W("mul", 0, A) VM_BACK_Y("mul", 0, A) VM_BACK_W("fmac", 1, B) \
        VM_BACK_Y("fmac", 1, B) VM_BACK_W("fmac", 2, C) VM_BACK_Y("fmac", 2, C) VM_BACK_W("fmac", 3, D) \
        VM_BACK_Y("fmac", 3, D) : VM_BACK_OUT, [y] "=&v"(y) : VM_BACK_IN);                         \
  }
VM_BACK(0, 0, 1, 2, 3) VM_BACK(1, 4, 5, 6, 7) VM_BACK(2, 8, 9, 10, 11) VM_BACK(3, 12, 13, 14, 15)
#undef VM_BACK
#undef VM_BACK_TEXT
#undef VM_BACK_W
#undef VM_BACK_Y
#undef VM_BACK_OUT
#undef VM_BACK_IN

template <int S, bool GATE>
__device__ __forceinline__ void back_token(const float (&A)[4], float dts, float dus, float dys, float b, float c,
                                           const f32x4 &decay, const f32x4 &h, const f32x4 &before, f32x4 &p,
                                           float (&dA)[4], float (&x)[4], float (&yy)[4], float &w, float &through,
                                           float &y) {
  back_sums<S, GATE>(dys, b, c, h, p, yy, w, y);
  through = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = p[i] * dus;
    p[i] *= decay[i];
    const float m = p[i] * before[i];
    dA[i] = __builtin_fmaf(m, dts, dA[i]);
    through = i == 0 ? m * A[0] : __builtin_fmaf(m, A[i], through);
  }
}

// The same where a product that the formulas do not have may not be finite.  in: the token is one
// of the chunk.  The steps of 0 behind them add nothing to dA: 0 times the last token's state,
// which they would add, is no number where that state is infinite.  PLACES: nor do places without
// a state or channel add to any sum.
template <int S, bool PLACES>
__device__ __forceinline__ void back_token_of(const Lane &l, bool in, const float (&A)[4], float dts, float dus, float dys, float b,
                                              float c, const f32x4 &decay, const f32x4 &h, const f32x4 &before, f32x4 &p,
                                              float (&dA)[4], float (&x)[4], float (&yy)[4], float &w, float &through,
                                              float &y) {
  const float bs[4] = {row_bcast<4 * S>(b), row_bcast<4 * S + 1>(b), row_bcast<4 * S + 2>(b), row_bcast<4 * S + 3>(b)};
  const float cs[4] = {row_bcast<4 * S>(c), row_bcast<4 * S + 1>(c), row_bcast<4 * S + 2>(c), row_bcast<4 * S + 3>(c)};
  w = y = through = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool has = !PLACES || l.has(i);
    const auto only = [&](float v, float other) { return has ? v : other; };
    const float g = only(__builtin_fmaf(cs[i], dys, p[i]), 0.0f);
    w = only(__builtin_fmaf(bs[i], g, w), w);
    y = only(__builtin_fmaf(cs[i], h[i], y), y);
    yy[i] = only(h[i] * dys, 0.0f);
    x[i] = only(g * dus, 0.0f);
    p[i] = only(g * decay[i], 0.0f);
    const float m = p[i] * before[i];
    dA[i] = in ? __builtin_fmaf(m, dts, dA[i]) : dA[i];
    through = only(__builtin_fmaf(m, A[i], through), through);
  }
}

// PLACES: there are fewer than 16 states, or waves with lanes of no channel.  (A kernel of its
// own: the test of each tile costs 3%, 128 x 197 tokens of 8 states 175 -> 180 us.)
template <typename T, bool GATE, bool PLACES>
__global__ __launch_bounds__(64 * kScanWaves, 3) void scan_back_kernel(PromptScanArgs a, int wide) {
  __shared__ __align__(16) float sums[2][kScanWaves][kBackTile * 32];
  __shared__ __align__(16) float meets[kScanWaves][kGroups][16][12];
  const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), blocks = (a.dim + 15) / 16;
  const int64_t slot = blockIdx.x / wide;
  const int group = blockIdx.x % wide, blk = group * kScanWaves + wave;
  float(*meet)[16][12] = meets[wave];
  Piece p = piece_by_length(a.q, slot);
  const bool none = p.len < 0;         // a slot without a chunk: its partial sums are 0
  if (none) {
    p.seq = p.c = p.len = 0;
    p.id = 0;
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
    const float x = bload<float>(rA, l.state[i]);
    A[i] = rate(x);
    A2[i] = rate2(x);
  }
  const float bias = channel_value(a.bias, c0, l), D = channel_value(a.D, c0, l);
  const uint32_t dstep = 4 * static_cast<uint32_t>(a.dim) * sizeof(T);

  // the gradient of the state after the chunk, and of several chunks the state before it
  f32x4 init = {0, 0, 0, 0}, grad = {0, 0, 0, 0};
  const int64_t sbase = (static_cast<int64_t>(p.seq) * a.dim + c0) * a.n;
  if (a.dstate != nullptr) {
    const Rsrc r = make_rsrc(a.dstate + sbase, l.cw * a.n * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) grad[i] = bload<float>(r, l.state[i]);
  }
  if (p.count > 1 && blk < blocks) {
    if (a.h0 != nullptr) {
      const Rsrc r = make_rsrc(a.h0 + sbase, l.cw * a.n * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) init[i] = bload<float>(r, l.state[i]);
    }
    const int64_t first = (slot - p.c) * blocks + blk;
    join_chunks(a.ends, a.steps, first, blocks, p.c, lane, A2, init);
    join_chunks(a.starts, a.steps, first + static_cast<int64_t>(p.count - 1) * blocks, -blocks, p.count - 1 - p.c, lane, A2,
                grad);
    if (PLACES) {
      clear_places(l, init);
      clear_places(l, grad);
    }
  }

  const int64_t mark = (p.t0 / kBackTile + p.id) * blocks + blk;
  const int64_t tokens = a.q.L * (a.q.off != nullptr ? 1 : a.q.nseq);
  float dD = 0.0f, dbias = 0.0f;
  // One tile.  WHOLE: of kBackTile tokens; else it is the chunk's last.
  const auto walk_tile = [&](int tile, auto whole) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(whole)::value;
    const int64_t t = p.t0 + tile * kBackTile, at = mark + static_cast<int64_t>(tile) * blocks;
    const int m = WHOLE ? kBackTile : p.len - tile * kBackTile;
    Raw r;
    load_tile<T, true, GATE>(a, l, t, m, c0, r);
    f32x4 begin = {0, 0, 0, 0};
    if (blk < blocks) {
      begin = *reinterpret_cast<const f32x4 *>(a.marks + at * 256 + lane * 4);
      if (p.count > 1) {
        const float before = a.before[at * 16 + l.ch];
#pragma unroll
        for (int i = 0; i < 4; ++i) begin[i] = carry(hw_exp2(A2[i] * before), init[i], begin[i]);
      }
      if (PLACES) clear_places(l, begin);
    }
    float slope[kGroups] = {};
    float size = 0.0f;                       // of what places without a state or channel multiply by 0
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float dt = step_of(a, r.d[g] + bias, WHOLE || 4 * g + l.q < m), du = dt * r.u[g];
      float dy = r.o[g];
      if (GATE) dy *= silu_both(r.z[g], slope[g]);
      meet[g][l.ch][2 * l.q] = dt;
      meet[g][l.ch][2 * l.q + 1] = du;
      meet[g][l.ch][8 + l.q] = dy;
      if (PLACES && WHOLE)
        size += __builtin_fabsf(du) + __builtin_fabsf(dy) + __builtin_fabsf(r.b[g]) + __builtin_fabsf(r.c[g]);
    }
    wave_lds_fence();
    float *mine = sums[tile & 1][wave];
    const Rsrc rdu = rows<T>(a.du, a.dim, t, c0, m, l.cw), rdd = rows<T>(a.ddelta, a.dim, t, c0, m, l.cw),
               rdz = rows<T>(a.dz, a.dim, t, c0, GATE ? m : 0, l.cw);
    // what a group's tokens give, from their products and sums over a lane's states
    const auto finish = [&](int g, float(&along4)[4], const float(&th)[4], float(&y)[4], const float(&x)[4][4],
                            const float(&yy)[4][4]) __attribute__((always_inline)) {
      settle(along4);
      if (GATE) settle(y);
      const float along = gather(along4), through = gather(th);
      const float dt = meet[g][l.ch][2 * l.q], dy = meet[g][l.ch][8 + l.q];
      if (GATE) {
        const float yt = __builtin_fmaf(D, r.u[g], gather(y));
        put<T>(rdz, l.dense + g * dstep, r.o[g] * yt * slope[g]);
      }
      put<T>(rdu, l.dense + g * dstep, __builtin_fmaf(along, dt, D * dy));
      float dd = __builtin_fmaf(along, r.u[g], through);
      const float slope2 = hw_rcp(1.0f + hw_exp2((r.d[g] + bias) * -kLog2e));
      dd *= a.softplus ? slope2 : 1.0f;
      put<T>(rdd, l.dense + g * dstep, dd);
      dD = __builtin_fmaf(dy, r.u[g], dD);
      dbias += WHOLE || 4 * g + l.q < m ? dd : 0.0f;
      float s[2];
      fold(x, yy, lane, s);
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const int to = (4 * g + ((lane >> 1) & 3)) * 32 + (lane & 8) * 2 + 4 * l.q + 2 * (lane & 1);
      *reinterpret_cast<f32x2 *>(mine + to) = f32x2{s[0], s[1]};
    };
    if (!WHOLE || (PLACES && uniform(__ballot(!finite(size)) != 0) != 0)) {
      // one group at a time, its states walked to from the tile's start
#pragma unroll
      for (int g = kGroups - 1; g >= 0; --g) {
        if (4 * g >= m) continue;
        f32x4 hs[4], es[4], first = begin;
#pragma unroll
        for (int k = 0; k <= g; ++k) {
          if (k > 0) first = hs[3];
          const auto &w = meet[k][l.ch];
          again<0>(A2, w[0], r.b[k], w[1], first, hs[0], es[0]);
          again<1>(A2, w[2], r.b[k], w[3], hs[0], hs[1], es[1]);
          again<2>(A2, w[4], r.b[k], w[5], hs[1], hs[2], es[2]);
          again<3>(A2, w[6], r.b[k], w[7], hs[2], hs[3], es[3]);
        }
        const auto &w = meet[g][l.ch];
        float x[4][4], yy[4][4], along4[4], th[4], y[4];
        back_token_of<3, PLACES>(l, 4 * g + 3 < m, A, w[6], w[7], w[11], r.b[g], r.c[g], es[3], hs[3], hs[2], grad, dA,
                                 x[3], yy[3], along4[3], th[3], y[3]);
        back_token_of<2, PLACES>(l, 4 * g + 2 < m, A, w[4], w[5], w[10], r.b[g], r.c[g], es[2], hs[2], hs[1], grad, dA,
                                 x[2], yy[2], along4[2], th[2], y[2]);
        back_token_of<1, PLACES>(l, 4 * g + 1 < m, A, w[2], w[3], w[9], r.b[g], r.c[g], es[1], hs[1], hs[0], grad, dA,
                                 x[1], yy[1], along4[1], th[1], y[1]);
        back_token_of<0, PLACES>(l, true, A, w[0], w[1], w[8], r.b[g], r.c[g], es[0], hs[0], first, grad, dA, x[0], yy[0],
                                 along4[0], th[0], y[0]);
        finish(g, along4, th, y, x, yy);
      }
    } else if constexpr (WHOLE) {
      f32x4 hs[kBackTile], es[kBackTile];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const auto &w = meet[g][l.ch];
        again<0>(A2, w[0], r.b[g], w[1], g > 0 ? hs[g > 0 ? 4 * g - 1 : 0] : begin, hs[4 * g], es[4 * g]);
        again<1>(A2, w[2], r.b[g], w[3], hs[4 * g], hs[4 * g + 1], es[4 * g + 1]);
        again<2>(A2, w[4], r.b[g], w[5], hs[4 * g + 1], hs[4 * g + 2], es[4 * g + 2]);
        again<3>(A2, w[6], r.b[g], w[7], hs[4 * g + 2], hs[4 * g + 3], es[4 * g + 3]);
      }
#pragma unroll
      for (int g = kGroups - 1; g >= 0; --g) {
        const auto &w = meet[g][l.ch];
        float x[4][4], yy[4][4], along4[4], th[4], y[4];
        back_token<3, GATE>(A, w[6], w[7], w[11], r.b[g], r.c[g], es[4 * g + 3], hs[4 * g + 3], hs[4 * g + 2], grad, dA, x[3],
                            yy[3], along4[3], th[3], y[3]);
        back_token<2, GATE>(A, w[4], w[5], w[10], r.b[g], r.c[g], es[4 * g + 2], hs[4 * g + 2], hs[4 * g + 1], grad, dA, x[2],
                            yy[2], along4[2], th[2], y[2]);
        back_token<1, GATE>(A, w[2], w[3], w[9], r.b[g], r.c[g], es[4 * g + 1], hs[4 * g + 1], hs[4 * g], grad, dA, x[1], yy[1],
                            along4[1], th[1], y[1]);
        back_token<0, GATE>(A, w[0], w[1], w[8], r.b[g], r.c[g], es[4 * g], hs[4 * g], g > 0 ? hs[g > 0 ? 4 * g - 1 : 0] : begin,
                            grad, dA, x[0], yy[0], along4[0], th[0], y[0]);
        finish(g, along4, th, y, x, yy);
      }
    }
    // (the other tile's sums may still be read by waves behind this barrier)
    __syncthreads();
    for (int i = threadIdx.x; i < kBackTile * 32; i += 64 * kScanWaves) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kScanWaves; ++w) s += sums[tile & 1][w][i];
      const int tok = i / 32, which = (i / 16) % 2, n = i % 16;
      if (tok < m && n < a.n) a.partBC[((group * tokens + t + tok) * 2 + which) * a.n + n] = s;
    }
  };
  int tile = p.len / kBackTile;
  if (p.len % kBackTile != 0) walk_tile(tile, std::false_type());
  while (--tile >= 0) walk_tile(tile, std::true_type());

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
  const int64_t per = tokens * 2 * a.n;
  const int64_t end = a.q.off != nullptr ? clamped(a.q.off[a.q.nseq], a.q.L) * 2 * a.n : per, last = a.q.clear > 0 ? per : end;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x; i < last; i += gridDim.x * static_cast<int64_t>(256)) {
    float s = 0.0f;
    int g = i < end ? 0 : wide;              // (rows of no sequence: 0)
    for (; g + 8 <= wide; g += 8) {          // (eight loads under way)
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = a.partBC[(g + k) * per + i];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
    for (; g < wide; ++g) s += a.partBC[g * per + i];
    const int64_t tok = i / (2 * a.n);
    const int col = static_cast<int>(i - tok * 2 * a.n);
    T *out = static_cast<T *>(col < a.n ? a.dB : a.dC);
    out[tok * a.n + (col < a.n ? col : col - a.n)] = from_f32<T>(s);
  }
}

template <typename T>
hipError_t launch_back(const PromptScanArgs &a, hipStream_t s) {
  const int wide = scan_wide(a.dim);
  const dim3 grid(static_cast<uint32_t>(a.q.slots * wide));
  const int64_t tokens = a.q.L * (a.q.off != nullptr ? 1 : a.q.nseq);
  const bool places = a.n < 16 || a.dim % (16 * kScanWaves) != 0;
  const auto both = [&](auto gate) {
    constexpr bool GATE = decltype(gate)::value;
    scan_marks_kernel<T, GATE><<<grid.x + a.q.clear, 64 * kScanWaves, 0, s>>>(a, wide);
    if (places)
      scan_back_kernel<T, GATE, true><<<grid, 64 * kScanWaves, 0, s>>>(a, wide);
    else
      scan_back_kernel<T, GATE, false><<<grid, 64 * kScanWaves, 0, s>>>(a, wide);
  };
  if (a.z != nullptr)
    both(std::true_type());
  else
    both(std::false_type());
  const int64_t sums = (tokens * 2 * a.n + 255) / 256, most = 1 << 16;
  scan_back_sum_kernel<T><<<static_cast<uint32_t>(sums < most ? sums : most), 256, 0, s>>>(a, wide, tokens);
  return hipGetLastError();
}

}  // namespace

// Chunks of a backward pass.  In cycles a token: a workgroup of the second launch takes
// some 680 alone on its compute unit, two 900 and k more 415 k; the first launch some 120
// a wave and SIMD, 200 where it gathers gradients besides (230 and more alone).
int64_t scan_back_chunk(int64_t tokens, int64_t nseq, int64_t L, int dim, bool packed) {
  const int64_t wide = scan_wide(dim);
  if (packed) {
    // The lengths are not known here.  A cut sequence costs the first launch's gathered
    // gradients, one that is too long its chain: a third of a SIMD's tokens where it has many
    // waves, else a fifth.  (Lengths of 1 to 1369, 8145 in all, us: 4096 channels, 10 waves,
    // 1040 tokens 684, 528 621; 2048, 5 waves, 528 393, 208 350; 768, 208 164, 96 152.)
    const int64_t all = tokens * scan_blocks(dim) / 1024, cut = all / (nseq * scan_blocks(dim) >= 8 * 1024 ? 3 : 5);
    const int64_t chunk = cut / kBackTile * kBackTile + kBackTile;
    return chunk < 64 ? (L < 64 ? L : 64) : chunk < L ? chunk : L;
  }
  int64_t best = L;
  double least = 0;
  for (int64_t parts = 1; parts <= 128; ++parts) {
    const int64_t chunk = parts == 1 ? L : ((L + parts - 1) / parts + kBackTile - 1) / kBackTile * kBackTile;
    if (chunk < 32 && parts > 1) break;
    if (chunk >= L && parts > 1) continue;
    const int64_t groups = wide * nseq * ((L + chunk - 1) / chunk), k = (groups + 255) / 256;
    const double waves = groups * 4 / 1024.0, first = waves * (parts > 1 ? 200 : 120);
    const double cost = chunk * ((k > 2 ? k * 415.0 : k > 1 ? 900.0 : 680.0) + (first > 230 ? first : 230)) + parts * 300.0;
    if (parts == 1 || cost < least) {
      least = cost;
      best = chunk;
    }
  }
  return best;
}

hipError_t launch_prompt_scan_back(const PromptScanArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? launch_back<bf16_t>(a, s) : launch_back<float>(a, s);
}

}  // namespace vmk
