// The selective scan over rows of tokens, as a language model's prompts come:
//   dt = softplus(delta + bias);  h_t = exp(dt A) h_{t-1} + dt B_t u_t;
//   y_t = C_t h_t + D u_t;  out_t = y_t SiLU(z_t)
// dense or packed, from given or zero states, the last states kept.
//
// A wave walks over the tokens of 16 channels, 4 states to a lane (the layout in
// prompt_device.h).  A state update is five vector instructions, one of them an
// exponential, and these bound it: 28.6 a wave and token, the SIMD busy with them all
// the while at 4.8 cycles each.  A sequence is cut in chunks where there are too few channels to fill the
// card.  Then one launch walks every chunk but a sequence's last from a zero state
// (its first, whose state is known, in full) and notes its end state and the sum of
// its steps T; a second one forms each later chunk's first state from the chunks
// before it, h <- exp(A T) h + end, and walks it in full.
// 40 packed prompts of 1 to 1500 tokens, 4096 channels, bf16 (1.8 TB/s): 158 us; one prompt of
// 4097 tokens: 119 us in two launches over 13 chunks.  Fewer states leave places empty and take
// the time of 16.
#include <hip/hip_runtime.h>

#include <cmath>

#include "prompt_device.h"

namespace vmk {
namespace {

constexpr int kGroups = 4;            // groups of 4 tokens to a tile
constexpr int kTile = 4 * kGroups;

// One tile's values as they were loaded.
struct Raw {
  float u[kGroups], d[kGroups], z[kGroups], b[kGroups], c[kGroups];
};

template <typename T, bool FULL, bool GATE>
__device__ __forceinline__ void load_tile(const PromptScanArgs &a, const Lane &l, int64_t token, int left, int c0, Raw &r) {
  const int m = left < kTile ? left : kTile;
  const Rsrc ru = rows<T>(a.u, a.us, token, c0, m, l.cw), rd = rows<T>(a.delta, a.ds, token, c0, m, l.cw),
             rb = rows<T>(a.B, a.bs, token, 0, m, a.n);
  const uint32_t su = 4 * a.us * sizeof(T), sd = 4 * a.ds * sizeof(T), sb = 4 * a.bs * sizeof(T);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    r.u[g] = bload<T>(ru, l.u + g * su);
    r.d[g] = bload<T>(rd, l.d + g * sd);
    r.b[g] = bload<T>(rb, l.b + g * sb);
  }
  if (FULL) {
    const Rsrc rc = rows<T>(a.C, a.cs, token, 0, m, a.n);
    const uint32_t sc = 4 * a.cs * sizeof(T);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) r.c[g] = bload<T>(rc, l.c + g * sc);
    if (GATE) {
      const Rsrc rz = rows<T>(a.z, a.zs, token, c0, m, l.cw);
      const uint32_t sz = 4 * a.zs * sizeof(T);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) r.z[g] = bload<T>(rz, l.z + g * sz);
    }
  }
}

// CLEAR: places without a state are cleared before they are read.
template <int S, bool FULL, bool CLEAR>
__device__ __forceinline__ void token(const Lane &l, const float (&A2)[4], float dt, float b, float du, float c, f32x4 &h,
                                      float &y) {
  f32x4 e;
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = dt * A2[i];
  f32x4 r;
  if (FULL && !CLEAR)
    y = update_read<S>(e, b, du, c, h, r);
  else
    update<S>(e, b, du, h, r);
  if (CLEAR) {
    clear_places(l, r);
    y = read_out<S>(c, r);
  }
  h = r;
}

// The tokens of a tile, whose dt and dt u are in `meet`.
template <typename T, bool FULL, bool GATE, bool ALL, bool CLEAR>
__device__ __forceinline__ void tokens(const PromptScanArgs &a, const Lane &l, const Raw &r, Rsrc ro, uint32_t oo, int m,
                                       const float (&A2)[4], float D, f32x4 &h, float (*meet)[16][8]) {
  const uint32_t so = 4 * a.dim * sizeof(T);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (!ALL && 4 * g >= m) break;
    float dts[4], dus[4], y[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      dts[s] = meet[g][l.ch][2 * s];
      dus[s] = meet[g][l.ch][2 * s + 1];
    }
    token<0, FULL, CLEAR>(l, A2, dts[0], r.b[g], dus[0], r.c[g], h, y[0]);
    token<1, FULL, CLEAR>(l, A2, dts[1], r.b[g], dus[1], r.c[g], h, y[1]);
    token<2, FULL, CLEAR>(l, A2, dts[2], r.b[g], dus[2], r.c[g], h, y[2]);
    token<3, FULL, CLEAR>(l, A2, dts[3], r.b[g], dus[3], r.c[g], h, y[3]);
    if (FULL) {
      settle(y);
      float o = __builtin_fmaf(D, r.u[g], gather(y));
      if (GATE) o *= silu_f(r.z[g]);
      put<T>(ro, oo + g * so, o);
    }
  }
}

// One tile of m tokens (ALL: a whole one) from (token, c0) on.
template <typename T, bool FULL, bool GATE, bool PLACES, bool ALL>
__device__ __forceinline__ void tile(const PromptScanArgs &a, const Lane &l, const Raw &r, int64_t at, int m, int c0,
                                     const float (&A2)[4], float bias, float D, f32x4 &h, float &steps,
                                     float (*meet)[16][8]) {
  const Rsrc ro = rows<T>(a.out, a.dim, at, c0, FULL ? m : 0, l.cw);
  const uint32_t oo = l.live ? (l.q * static_cast<uint32_t>(a.dim) + l.ch) * sizeof(T) : kOob;
  // every lane gets its channel's dt and dt u of all tokens by way of LDS
  bool odd = false;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const float dt = step_of(a, r.d[g] + bias, ALL || 4 * g + l.q < m), du = dt * r.u[g];
    steps += dt;
    meet[g][l.ch][2 * l.q] = dt;
    meet[g][l.ch][2 * l.q + 1] = du;
    if (FULL && PLACES) odd |= !finite(du);  // (so is it where dt is not)
  }
  wave_lds_fence();
  if (FULL && PLACES && __any(odd))
    tokens<T, FULL, GATE, ALL, true>(a, l, r, ro, oo, m, A2, D, h, meet);
  else
    tokens<T, FULL, GATE, ALL, false>(a, l, r, ro, oo, m, A2, D, h, meet);
  wave_lds_fence();
}

// Walks a chunk from state h; returns the sum of this lane's steps.
template <typename T, bool FULL, bool GATE, bool PLACES>
__device__ __forceinline__ float walk(const PromptScanArgs &a, const Lane &l, const Piece &p, int c0, const float (&A2)[4],
                                      float bias, float D, f32x4 &h, float (*meet)[16][8]) {
  float steps = 0.0f;
  Raw next;
  load_tile<T, FULL, GATE>(a, l, p.t0, p.len, c0, next);
  int at = 0;
  for (; at + kTile <= p.len; at += kTile) {
    const Raw r = next;
    load_tile<T, FULL, GATE>(a, l, p.t0 + at + kTile, p.len - at - kTile, c0, next);
    tile<T, FULL, GATE, PLACES, true>(a, l, r, p.t0 + at, kTile, c0, A2, bias, D, h, steps, meet);
  }
  if (at < p.len) tile<T, FULL, GATE, PLACES, false>(a, l, next, p.t0 + at, p.len - at, c0, A2, bias, D, h, steps, meet);
  return steps;
}

// PLACES: there are fewer than 16 states.  (A kernel of its own, since the test of each tile
// costs the scan of 16 states 2.7%: 163 -> 168 us for 40 packed prompts.  Four waves a SIMD: with
// three, which the compiler would take, 8 states need 154 us, with four 150.)
template <typename T, bool GATE, bool PLACES, bool SECOND>
__global__ __launch_bounds__(64 * kScanWaves, PLACES ? 4 : 1) void prompt_scan_kernel(PromptScanArgs a, int64_t slots) {
  __shared__ __align__(16) float meets[kScanWaves][kGroups][16][8];
  float(*meet)[16][8] = meets[threadIdx.x / 64];
  const int lane = threadIdx.x % 64;
  const int blocks = (a.dim + 15) / 16, waves = blockDim.x / 64;
  const int wide = (blocks + waves - 1) / waves;
  int64_t slot = blockIdx.x / wide;
  if (!SECOND && slot >= slots) {
    clear_rest<T>(a.q, a.out, a.dim, blockIdx.x - slots * wide);
    return;
  }
  if (a.q.off != nullptr) {
    // by falling length: every other round of workgroups over the 256 compute units backwards, so
    // that the longest sequence of one round shares its units with the shortest of the next
    const int each = 256 / wide, round = each > 1 ? static_cast<int>(slot) / each : 0;
    if ((round & 1) != 0) {
      const int64_t next = (round + int64_t{1}) * each, end = next < slots ? next : slots;
      slot = end - 1 - (slot - static_cast<int64_t>(round) * each);
    }
  }
  if (a.q.off == nullptr && a.ends != nullptr) {   // all chunks of a sequence but its last or first
    const uint32_t per = (static_cast<uint32_t>(a.q.L) + static_cast<uint32_t>(a.q.chunk) - 1) / static_cast<uint32_t>(a.q.chunk),
                   seq = static_cast<uint32_t>(slot) / (per - 1);
    slot += seq + (SECOND ? 1 : 0);
  }
  const int blk = uniform(static_cast<int>(blockIdx.x % wide) * waves + threadIdx.x / 64);
  if (blk >= blocks) return;
  const Piece p = piece_by_length<SECOND ? 2 : 1>(a.q, slot);
  if (p.len < 0 || (SECOND ? p.c == 0 : p.c > 0 && p.c == p.count - 1)) return;
  // a long chunk goes on at its own pace beside short ones
  if (a.q.off != nullptr) {
    const int64_t whole = a.q.chunk < a.q.L ? a.q.chunk : a.q.L, four = int64_t{4} * p.len;
    if (four >= 3 * whole)
      __builtin_amdgcn_s_setprio(3);
    else if (four >= 2 * whole)
      __builtin_amdgcn_s_setprio(2);
    else if (four >= whole)
      __builtin_amdgcn_s_setprio(1);
  }
  const int c0 = blk * 16;
  const Lane l = lane_of<T>(a, c0, lane);
  float A2[4];
  const Rsrc rA = make_rsrc(a.A + static_cast<int64_t>(c0) * a.n, l.cw * a.n * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = rate2(bload<float>(rA, l.state[i]));
  const float D = channel_value(a.D, c0, l), bias = channel_value(a.bias, c0, l);

  const int64_t kept = kept_at(a.q, p.seq);
  const int64_t block = p.id * blocks + blk;
  f32x4 h = {0, 0, 0, 0};
  if (!SECOND) {
    if (p.c == 0 && a.h0 != nullptr && kept >= 0 && starts_kept(a.q, p.seq)) {
      const Rsrc rh = make_rsrc(a.h0 + (kept * a.dim + c0) * a.n, l.cw * a.n * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = bload<float>(rh, l.state[i]);
    }
  } else {
    join_chunks(a.ends, a.steps, block - static_cast<int64_t>(p.c) * blocks, blocks, p.c, lane, A2, h);
    if (PLACES) clear_places(l, h);
  }
  float steps;
  if (SECOND || p.c == 0)
    steps = walk<T, true, GATE, PLACES>(a, l, p, c0, A2, bias, D, h, meet);
  else
    steps = walk<T, false, false, PLACES>(a, l, p, c0, A2, bias, D, h, meet);
  if (p.c == p.count - 1) {
    if (a.state != nullptr && kept >= 0) {
      const Rsrc rh = make_rsrc(a.state + (kept * a.dim + c0) * a.n, l.cw * a.n * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) bstore<float>(rh, l.state[i], h[i]);
    }
  } else if (!SECOND) {                    // (the second launch's other workgroups read these)
    float s[4] = {steps, steps, steps, steps};
    steps = gather(s);
    *reinterpret_cast<f32x4 *>(a.ends + block * 256 + lane * 4) = h;
    if (l.q == 0) a.steps[block * 16 + l.ch] = steps;
  }
}

template <typename T, bool GATE, bool PLACES>
hipError_t launch_scan(const PromptScanArgs &a, hipStream_t s) {
  const int blocks = (a.dim + 15) / 16, waves = blocks < kScanWaves ? blocks : kScanWaves;
  const int64_t wide = (blocks + waves - 1) / waves;
  const bool packed = a.q.off != nullptr, many = a.ends != nullptr;
  const int64_t first = !packed && many ? a.q.slots - a.q.nseq : a.q.slots;
  prompt_scan_kernel<T, GATE, PLACES, false><<<static_cast<uint32_t>(first * wide + a.q.clear), 64 * waves, 0, s>>>(a, first);
  if (many) {
    // (40 packed prompts of one chunk each: 16 us to find nothing to do in all slots, 5 in these)
    const int64_t second = packed && a.q.nseq <= 64 ? a.q.L / a.q.chunk : first;
    prompt_scan_kernel<T, GATE, PLACES, true><<<static_cast<uint32_t>(second * wide), 64 * waves, 0, s>>>(a, second);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch_type(const PromptScanArgs &a, hipStream_t s) {
  if (a.n < 16) return a.z != nullptr ? launch_scan<T, true, true>(a, s) : launch_scan<T, false, true>(a, s);
  return a.z != nullptr ? launch_scan<T, true, false>(a, s) : launch_scan<T, false, false>(a, s);
}

}  // namespace

int64_t seq_slots(int64_t nseq, int64_t L, int64_t chunk, bool packed) {
  return packed ? L / chunk + nseq : nseq * ((L + chunk - 1) / chunk);
}

// Chunks of a forward pass.  In cycles a token: a wave takes some 205 alone on its SIMD,
// k together 60 + 131 k; without read-out three quarters (but the first chunk is walked in
// full in the first launch, which shows where waves are alone).  A second launch costs some
// 25000, and a chunk 900 for the joining of all before it.
int64_t scan_chunk(int64_t tokens, int64_t nseq, int64_t L, int dim, bool packed) {
  const int64_t blocks = scan_blocks(dim);
  if (packed) {
    // The lengths are not known here.  Many waves to a SIMD share it whatever the lengths,
    // and a second walk costs them most: only what is longer than most of a SIMD's tokens is
    // cut.  With fewer the longest sequence sets the time: chunks of a quarter of a SIMD's
    // tokens, but not so many to a sequence that joining them costs more.  (Lengths of 1 to
    // 1369, 8145 in all, us: 4096 channels, 10 waves, 1632 tokens 160, 528 175; 2048, 5 waves,
    // 912 136, 272 112; 768, 384 77, 144 65.)
    const double all = static_cast<double>(tokens * blocks) / 1024.0, few = all / 4, join = 1.5 * sqrt(static_cast<double>(tokens));
    const bool full = nseq * blocks >= 8 * 1024;
    const int64_t chunk = static_cast<int64_t>(full ? 0.8 * all : few > join ? few : join) / kTile * kTile + kTile;
    return chunk < 64 ? (L < 64 ? L : 64) : chunk < L ? chunk : L;
  }
  const auto pace = [](double k) { return k <= 1 ? 205 : 60 + 131 * (k < 4 ? ceil(k) : k); };
  const double all = static_cast<double>(nseq * blocks) / 1024.0;
  int64_t best = L;
  double least = L * pace(all);
  for (int64_t parts = 2; parts <= 128; ++parts) {
    const int64_t chunk = ((L + parts - 1) / parts + kTile - 1) / kTile * kTile;
    if (chunk < 32) break;
    if (chunk >= L) continue;
    const double k = all * (parts - 1), full = pace(k);
    const double cost = chunk * full * (parts == 2 || k <= 1 ? 2.0 : 1.75) + 25000 + parts * 900;
    if (cost < least) {
      least = cost;
      best = chunk;
    }
  }
  return best;
}

hipError_t launch_prompt_scan(const PromptScanArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? launch_type<bf16_t>(a, s) : launch_type<float>(a, s);
}

}  // namespace vmk
