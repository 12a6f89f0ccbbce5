// The short causal convolution of a block over rows of tokens, with SiLU:
//   v_t = bias + sum_k w_k x_{t-W+1+k},  out_t = SiLU(v_t),
// the inputs before a sequence's first token from a kept window (or 0), the last
// ones left in it; over single tokens; and its gradients
//   dv = dout SiLU'(v),  dx_t = sum_k w_k dv_{t+W-1-k},  dw_k = sum_t dv_t x_{t-W+1+k}.
//
// Bound by memory.  A lane holds V neighbouring channels (16 bytes where rows are
// whole pieces of that) and walks over a chunk of a sequence's tokens with the
// window in registers, so x is read once but for the W - 1 tokens before a chunk.
// The windows are written by the lane that reads them, from the sequence's last
// tokens, so that they may be the same memory.  40 packed prompts of 1 to 1500 tokens, 4096
// channels, bf16: 33 us, 4.1 TB/s where a copy of 4 GB runs at 4.6; backward, 128 x 197
// tokens of 384 channels, fp32: 31 us and 4 for the sums.  The backward pass in bf16 is bound by
// vector instructions: 8 channels a lane take 231 registers and two waves a SIMD, as many
// instructions as fp32 for half the bytes (4 x 4097 tokens of 4096 channels: fp32 199 us, 4.1
// TB/s, bf16 141, 2.9).
#include <hip/hip_runtime.h>

#include "prompt_device.h"

namespace vmk {
namespace {

constexpr int kThreads = 256;

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_raw(const void *base, int64_t at) {
  return *reinterpret_cast<const Vec<T, V> *>(static_cast<const T *>(base) + at);
}
template <typename T, int V>
__device__ __forceinline__ void store_raw(void *base, int64_t at, const Vec<T, V> &x) {
  *reinterpret_cast<Vec<T, V> *>(static_cast<T *>(base) + at) = x;
}
template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V> &x, float (&y)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) y[e] = to_f32(x.v[e]);
}
template <typename T, int V>
__device__ __forceinline__ void load(const void *base, int64_t at, float (&y)[V]) {
  widen<T, V>(load_raw<T, V>(base, at), y);
}
template <typename T, int V>
__device__ __forceinline__ void store(void *base, int64_t at, const float (&y)[V]) {
  Vec<T, V> x;
#pragma unroll
  for (int e = 0; e < V; ++e)
    if constexpr (sizeof(T) == 2)
      x.v[e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(y[e]));   // (to nearest even)
    else
      x.v[e] = y[e];
  store_raw<T, V>(base, at, x);
}

template <int W, int V>
struct Taps {
  float w[W][V], bias[V];
};
template <int W, int V>
__device__ __forceinline__ Taps<W, V> load_taps(const float *w, const float *bias, int c) {
  Taps<W, V> t;
  float all[W * V];                        // (one run of memory: the compiler widens the loads)
#pragma unroll
  for (int i = 0; i < W * V; ++i) all[i] = w[static_cast<int64_t>(c) * W + i];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    t.bias[e] = bias != nullptr ? bias[c + e] : 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) t.w[k][e] = all[e * W + k];
  }
  return t;
}

// v of the window x[0 .. W-1], oldest first.
template <int W, int V>
__device__ __forceinline__ void convolve(const Taps<W, V> &t, const float (&x)[W][V], float (&v)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    v[e] = t.bias[e];
#pragma unroll
    for (int k = 0; k < W; ++k) v[e] = __builtin_fmaf(t.w[k][e], x[k][e], v[e]);
  }
}
template <int W, int V>
__device__ __forceinline__ void push(float (&x)[W][V]) {
#pragma unroll
  for (int k = 0; k + 1 < W; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) x[k][e] = x[k + 1][e];
}

// The W - 1 inputs before token t of a sequence, in x[1 .. W-1] (they move down by
// one before the next token enters).  old: its kept window, nullptr = 0.
template <typename T, int W, int V>
__device__ __forceinline__ void window_before(const void *in, int64_t xs, int c, const T *old, int dim, int64_t lo, int64_t t,
                                              float (&x)[W][V]) {
#pragma unroll
  for (int k = 1; k < W; ++k) {
    const int64_t at = t - W + k;
    if (at >= lo)
      load<T, V>(in, at * xs + c, x[k]);
    else if (old != nullptr)
      load<T, V>(old, (W - 1 + at - lo) * dim + c, x[k]);
    else
#pragma unroll
      for (int e = 0; e < V; ++e) x[k][e] = 0.0f;
  }
}

template <typename T, int W, int V>
__global__ __launch_bounds__(kThreads) void prompt_conv_kernel(PromptConvArgs a, uint32_t wide) {
  const int64_t slot = blockIdx.x / wide;
  if (slot >= a.q.slots) {
    clear_rest<T>(a.q, a.out, a.dim, blockIdx.x - a.q.slots * wide);
    return;
  }
  const int c = static_cast<int>((blockIdx.x % wide) * blockDim.x + threadIdx.x) * V;
  const Piece p = piece_of(a.q, slot);
  if (p.len < 0 || c >= a.dim) return;
  const int64_t kept = kept_at(a.q, p.seq), window = static_cast<int64_t>(W - 1) * a.dim;
  const T *old = a.h0 != nullptr && kept >= 0 && starts_kept(a.q, p.seq) ? static_cast<const T *>(a.h0) + kept * window : nullptr;
  const Taps<W, V> taps = load_taps<W, V>(a.w, a.bias, c);
  float x[W][V];
  window_before<T, W, V>(a.x, a.xs, c, old, a.dim, p.lo, p.t0, x);
  if (p.c == 0 && a.state != nullptr && kept >= 0) {
    Vec<T, V> last[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t at = p.hi - (W - 1) + j;
      if (at >= p.lo)
        last[j] = load_raw<T, V>(a.x, at * a.xs + c);
      else if (old != nullptr)
        last[j] = load_raw<T, V>(old, (W - 1 + at - p.lo) * a.dim + c);
      else
        last[j] = Vec<T, V>{};
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_raw<T, V>(static_cast<T *>(a.state) + kept * window, static_cast<int64_t>(j) * a.dim + c, last[j]);
  }
  constexpr int kAhead = 4;
  Vec<T, V> next[kAhead];
  const int64_t end = p.t0 + p.len;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (p.t0 + i < end) next[i] = load_raw<T, V>(a.x, (p.t0 + i) * a.xs + c);
  for (int64_t t = p.t0; t < end; t += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i >= end) break;
      push<W, V>(x);
      widen<T, V>(next[i], x[W - 1]);
      if (t + i + kAhead < end) next[i] = load_raw<T, V>(a.x, (t + i + kAhead) * a.xs + c);
      float v[V];
      convolve<W, V>(taps, x, v);
      if (a.silu)
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = silu_f(v[e]);
      store<T, V>(a.out, (t + i) * a.dim + c, v);
    }
  }
}

// A worker walks every workers-th chunk and keeps its sums of dw and dbias.
template <typename T, int W, int V>
__global__ __launch_bounds__(kThreads) void prompt_conv_back_kernel(PromptConvArgs a, uint32_t wide) {
  const int64_t worker = blockIdx.x / wide;
  if (worker >= a.workers) {
    clear_rest<T>(a.q, a.dx, a.dim, blockIdx.x - static_cast<int64_t>(a.workers) * wide);
    return;
  }
  const int at0 = static_cast<int>((blockIdx.x % wide) * blockDim.x + threadIdx.x) * V;
  const bool live = at0 < a.dim;
  const int c = live ? at0 : 0;               // (lanes past the channels stay for the search, and do no work)
  const Taps<W, V> taps = load_taps<W, V>(a.w, a.bias, c);
  const int64_t window = static_cast<int64_t>(W - 1) * a.dim;
  float dw[W][V] = {}, db[V] = {};
  for (int64_t slot = worker; slot < a.q.slots; slot += a.workers) {
    const Piece p = piece_of(a.q, slot);
    if (p.len < 0 || !live) continue;
    const T *old = a.h0 != nullptr ? static_cast<const T *>(a.h0) + p.seq * window : nullptr;
    const T *dlast = a.dstate != nullptr ? static_cast<const T *>(a.dstate) + p.seq * window : nullptr;
    float x[W][V], dv[W][V] = {};
    window_before<T, W, V>(a.x, a.xs, c, old, a.dim, p.lo, p.t0, x);
    const int64_t end = p.t0 + p.len;
    // dv of the chunk's tokens and of the W - 1 after them; a token's dx is whole when
    // the last of the outputs that read it has passed, and so is the window's gradient
    // (places before the sequence's first token) in its first chunk
    constexpr int kAhead = 4;
    Vec<T, V> nx[kAhead], nd[kAhead];       // the next tokens, under way
    const int64_t last = end + W - 1 < p.hi ? end + W - 1 : p.hi;
    const auto fetch = [&](int64_t t, int i) {
      if (t >= last) return;
      nx[i] = load_raw<T, V>(a.x, t * a.xs + c);
      nd[i] = load_raw<T, V>(a.dout, t * a.dim + c);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(p.t0 + i, i);
    for (int64_t t0 = p.t0; t0 < end + W - 1; t0 += kAhead)
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t t = t0 + i;
        if (t >= end + W - 1) break;
        push<W, V>(x);
        push<W, V>(dv);
#pragma unroll
        for (int e = 0; e < V; ++e) dv[W - 1][e] = 0.0f;
        if (t < last) {
          widen<T, V>(nx[i], x[W - 1]);
          widen<T, V>(nd[i], dv[W - 1]);
          fetch(t + kAhead, i);
          if (a.silu) {
            float v[V];
            convolve<W, V>(taps, x, v);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float s = hw_rcp(1.0f + hw_exp2(-v[e] * kLog2e));
              dv[W - 1][e] *= s * __builtin_fmaf(v[e], 1.0f - s, 1.0f);
            }
          }
          if (t < end)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              db[e] += dv[W - 1][e];
#pragma unroll
              for (int k = 0; k < W; ++k) dw[k][e] = __builtin_fmaf(dv[W - 1][e], x[k][e], dw[k][e]);
            }
        }
        const int64_t at = t - (W - 1);
        if (at >= p.t0 ? at >= end : p.c > 0 || a.dh0 == nullptr) continue;
        float d[V] = {};
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) d[e] = __builtin_fmaf(taps.w[W - 1 - k][e], dv[k][e], d[e]);
        if (dlast != nullptr && at >= p.hi - (W - 1)) {
          float more[V];
          load<T, V>(dlast, (at - p.hi + W - 1) * a.dim + c, more);
#pragma unroll
          for (int e = 0; e < V; ++e) d[e] += more[e];
        }
        if (at >= p.t0)
          store<T, V>(a.dx, at * a.dim + c, d);
        else
          store<T, V>(static_cast<T *>(a.dh0) + p.seq * window, (at - p.lo + W - 1) * a.dim + c, d);
      }
  }
  if (!live) return;
  float *part = a.partial + worker * (W + 1) * a.dim + c;
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) part[e * W + k + static_cast<int64_t>(c) * (W - 1)] = dw[k][e];
    part[static_cast<int64_t>(W) * a.dim + e] = db[e];
  }
}

template <typename T, int W, int V>
__global__ __launch_bounds__(kThreads) void token_conv_kernel(TokenConvArgs a) {
  const int nv = a.dim / V;
  const int64_t id = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x, row = id / nv;
  if (row >= a.batch) return;
  const int c = static_cast<int>(id - row * nv) * V;
  const int64_t slot = a.where != nullptr ? a.where[row] : row;
  float v[V] = {};
  if (slot >= 0 && slot < a.kept) {
    T *state = static_cast<T *>(a.state) + slot * (W - 1) * a.dim;
    Vec<T, V> in[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k] = load_raw<T, V>(state, static_cast<int64_t>(k) * a.dim + c);
    in[W - 1] = load_raw<T, V>(a.x, row * a.xs + c);
    const Taps<W, V> taps = load_taps<W, V>(a.w, a.bias, c);
    float x[W][V];
#pragma unroll
    for (int k = 0; k < W; ++k) widen<T, V>(in[k], x[k]);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_raw<T, V>(state, static_cast<int64_t>(k) * a.dim + c, in[k + 1]);
    convolve<W, V>(taps, x, v);
    if (a.silu)
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = silu_f(v[e]);
  }
  store<T, V>(a.out, row * a.dim + c, v);
}

template <typename T, int V, typename F>
hipError_t by_width(int width, F &&f) {
  switch (width) {
    case 2: f(std::integral_constant<int, 2>()); break;
    case 3: f(std::integral_constant<int, 3>()); break;
    default: f(std::integral_constant<int, 4>()); break;
  }
  return hipGetLastError();
}

uint32_t blocks_of(int64_t threads) { return static_cast<uint32_t>((threads + kThreads - 1) / kThreads); }

// Workgroups to a row of `lanes` lanes, and threads of each (whole waves).
struct Cut {
  uint32_t wide, threads;
};
Cut cut(int lanes) {
  const int waves = (lanes + 63) / 64, wide = (waves + kThreads / 64 - 1) / (kThreads / 64);
  return {static_cast<uint32_t>(wide), static_cast<uint32_t>((waves + wide - 1) / wide * 64)};
}

template <typename T, int V>
hipError_t launch_fwd(const PromptConvArgs &a, hipStream_t s) {
  const Cut z = cut(a.dim / V);
  return by_width<T, V>(a.width, [&](auto w) {
    prompt_conv_kernel<T, decltype(w)::value, V><<<static_cast<uint32_t>(a.q.slots * z.wide + a.q.clear), z.threads, 0, s>>>(a, z.wide);
  });
}
template <typename T, int V>
hipError_t launch_bwd(const PromptConvArgs &a, hipStream_t s) {
  const Cut z = cut(a.dim / V);
  return by_width<T, V>(a.width, [&](auto w) {
    prompt_conv_back_kernel<T, decltype(w)::value, V><<<static_cast<uint32_t>(a.workers) * z.wide + a.q.clear, z.threads, 0, s>>>(a, z.wide);
  });
}
template <typename T, int V>
hipError_t launch_step(const TokenConvArgs &a, hipStream_t s) {
  return by_width<T, V>(a.width, [&](auto w) {
    token_conv_kernel<T, decltype(w)::value, V><<<blocks_of(static_cast<int64_t>(a.batch) * (a.dim / V)), kThreads, 0, s>>>(a);
  });
}

// Whether rows of all these are whole pieces of `bytes`.
bool pieces(std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> strides, int es, int bytes) {
  for (const void *p : ptrs)
    if ((reinterpret_cast<uintptr_t>(p) % bytes) != 0) return false;
  for (int64_t st : strides)
    if (st * es % bytes != 0) return false;
  return true;
}
bool whole(const PromptConvArgs &a, int es) {
  return pieces({a.x, a.h0, a.state, a.out, a.dout, a.dstate, a.dx, a.dh0}, {a.xs, a.dim}, es, 16);
}

}  // namespace

int conv_workers(const PromptConvArgs &a, bool bf16) {
  // (a worker is at least a wave)
  const int es = bf16 ? 2 : 4, nv = whole(a, es) ? a.dim * es / 16 : a.dim;
  const int64_t most = (int64_t{1} << 18) / (nv > 64 ? nv : 64) + 1;
  return static_cast<int>(a.q.slots < most ? a.q.slots : most);
}

hipError_t launch_prompt_conv(const PromptConvArgs &a, bool bf16, hipStream_t s) {
  if (bf16) return whole(a, 2) ? launch_fwd<bf16_t, 8>(a, s) : launch_fwd<bf16_t, 1>(a, s);
  return whole(a, 4) ? launch_fwd<float, 4>(a, s) : launch_fwd<float, 1>(a, s);
}
hipError_t launch_prompt_conv_back(const PromptConvArgs &a, bool bf16, hipStream_t s) {
  if (bf16) return whole(a, 2) ? launch_bwd<bf16_t, 8>(a, s) : launch_bwd<bf16_t, 1>(a, s);
  return whole(a, 4) ? launch_bwd<float, 4>(a, s) : launch_bwd<float, 1>(a, s);
}
hipError_t launch_token_conv(const TokenConvArgs &a, bool bf16, hipStream_t s) {
  const bool v = pieces({a.x, a.state, a.out}, {a.xs, a.dim}, bf16 ? 2 : 4, 16);
  if (bf16) return v ? launch_step<bf16_t, 8>(a, s) : launch_step<bf16_t, 1>(a, s);
  return v ? launch_step<float, 4>(a, s) : launch_step<float, 1>(a, s);
}

}  // namespace vmk
