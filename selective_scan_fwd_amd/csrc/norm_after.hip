// The norm of a block's output by groups of channels, gated and added to the residual,
// and its gradients:
//   y = n(x) w SiLU(z)  or (gate first)  n(x SiLU(z)) w,  out = residual + factor scale y,
//   n(v) = v s, s = 1 / sqrt(mean v^2 + eps) over a group
//   back: d the gradient of n w:  dv = s (w d - n mean(w d n)),  dw = sum d n
// Bound by memory: every input is read once and every output written once.  4 x 4097 rows of
// 16 heads of 128, bf16 (201 MB): 39 us, 5.1 TB/s; backward of 128 x 197 rows of 384, fp32 (194
// MB): 48 us, of which 39 this kernel with the next row's loads under way and 6 the sums.
// The backward pass holds four arrays of columns and two rows in registers, which groups above
// 2048 channels (two pieces a lane) are too wide for: one wave a SIMD to 4096 channels, spills
// through memory above.  Whole rows, gated, bf16: 16384 rows of 2048 128 us (2.6 TB/s), 8192 of
// 4096 209 (1.6), 8192 of 8192 789 (0.9), 4096 of 16384 1896 (0.4); forward 41, 42, 82 and 91.
#include <hip/hip_runtime.h>

#include "block_norm.h"

namespace vmk {
namespace {

// ----------------------------------------------------------------- after
template <typename T, typename R, int LANES, int P, bool VEC>
__global__ __launch_bounds__(threads_of(LANES)) void after_kernel(BlockNormArgs a) {
  __shared__ float meet[kMeet][1];
  const Unit u = unit_of<LANES>(a, a.dim / a.group);
  const int64_t row = u.live ? u.row : 0;
  const int col = u.grp * a.group;
  float x[P][8], z[P][8], t[P][8];
  load<LANES, P, VEC>(static_cast<const T *>(a.x) + row * a.xs + col, a.group, u.lane, x);
  if (a.z != nullptr) {
    load<LANES, P, VEC>(static_cast<const T *>(a.z) + row * a.zs + col, a.group, u.lane, z);
    VM_EACH z[i][e] = silu_f(z[i][e]);
    if (a.gate_first) VM_EACH x[i][e] *= z[i][e];
  }
  float s[1] = {0.0f};
  VM_EACH s[0] = __builtin_fmaf(x[i][e], x[i][e], s[0]);
  sum_lanes<LANES, 1>(s, meet);
  const float size = inverse_root(s[0] / static_cast<float>(a.group) + a.eps);
  load_columns<LANES, P, VEC>(a.w != nullptr && a.wide ? a.w + col : a.w, a.group, u.lane, 1.0f, t);
  VM_EACH x[i][e] = x[i][e] * size * t[i][e];
  if (a.z != nullptr && !a.gate_first) VM_EACH x[i][e] *= z[i][e];
  if (a.scale != nullptr) {
    load<LANES, P, VEC>(a.scale + col, a.group, u.lane, t);
    VM_EACH x[i][e] *= t[i][e];
  }
  if (a.factor != 1.0f) VM_EACH x[i][e] *= a.factor;
  if (a.residual != nullptr) {
    load<LANES, P, VEC>(static_cast<const R *>(a.residual) + row * a.dim + col, a.group, u.lane, t);
    VM_EACH x[i][e] += t[i][e];
  }
  if (u.live) store<LANES, P, VEC>(static_cast<R *>(a.y) + row * a.dim + col, a.group, u.lane, x);
}

template <typename T, typename R, int LANES, int P, bool VEC>
__global__ __launch_bounds__(threads_of(LANES)) void after_back_kernel(BlockNormArgs a) {
  __shared__ float meet[kMeet][2];
  const Unit u = unit_of<LANES>(a, a.dim / a.group);
  const int col = u.grp * a.group;
  float w[P][8], scale[P][8], dw[P][8], ds[P][8];
  load_columns<LANES, P, VEC>(a.w != nullptr && a.wide ? a.w + col : a.w, a.group, u.lane, 1.0f, w);
  load_columns<LANES, P, VEC>(a.scale != nullptr ? a.scale + col : nullptr, a.group, u.lane, 1.0f, scale);
  VM_EACH {
    scale[i][e] *= a.factor;
    dw[i][e] = ds[i][e] = 0.0f;
  }
  const float over = 1.0f / static_cast<float>(a.group);
  float nx[P][8], nz[P][8], nd[P][8];       // the next row, under way
  const auto fetch = [&](int64_t row) {
    load<LANES, P, VEC>(static_cast<const T *>(a.x) + row * a.xs + col, a.group, u.lane, nx);
    load<LANES, P, VEC>(static_cast<const R *>(a.dy) + row * a.dim + col, a.group, u.lane, nd);
    if (a.z != nullptr) load<LANES, P, VEC>(static_cast<const T *>(a.z) + row * a.zs + col, a.group, u.lane, nz);
  };
  if (u.live && u.row < a.rows) fetch(u.row);
  for (int64_t row = u.row; row < a.rows && u.live; row += a.workers) {
    // d: the gradient of n w; what is normed is x, or (gate first) x times the gate
    float x[P][8], gate[P][8], slope[P][8], d[P][8];
    VM_EACH {
      x[i][e] = nx[i][e];
      d[i][e] = nd[i][e];
      slope[i][e] = 0.0f;
      gate[i][e] = a.z != nullptr ? silu_both(nz[i][e], slope[i][e]) : 1.0f;
    }
    if (row + a.workers < a.rows) fetch(row + a.workers);
    float s[2] = {0.0f, 0.0f};
    VM_EACH {
      const float v = a.gate_first ? rounded(x[i][e] * gate[i][e]) : x[i][e];
      const float g = rounded(d[i][e] * scale[i][e] * (a.gate_first ? 1.0f : gate[i][e]) * w[i][e]);
      s[0] = __builtin_fmaf(v, v, s[0]);
      s[1] = __builtin_fmaf(g, v, s[1]);
    }
    sum_lanes<LANES, 2>(s, meet);
    const float size = inverse_root(s[0] * over + a.eps);
    VM_EACH {
      const float v = a.gate_first ? rounded(x[i][e] * gate[i][e]) : x[i][e];
      const float n = v * size, after = a.gate_first ? 1.0f : gate[i][e];
      if (a.want_scale) ds[i][e] = __builtin_fmaf(d[i][e] * a.factor, n * w[i][e] * after, ds[i][e]);
      const float dout = d[i][e] * scale[i][e], dn = dout * after;
      dw[i][e] = __builtin_fmaf(dn, n, dw[i][e]);
      const float dv = norm_back(rounded(dn * w[i][e]), v, size, s[0], s[1], over, a.eps);
      d[i][e] = a.gate_first ? dv * gate[i][e] : dv;
      slope[i][e] *= a.gate_first ? dv * x[i][e] : dout * n * w[i][e];
    }
    store<LANES, P, VEC>(static_cast<T *>(a.dx) + row * a.dim + col, a.group, u.lane, d);
    if (a.dz != nullptr) store<LANES, P, VEC>(static_cast<T *>(a.dz) + row * a.dim + col, a.group, u.lane, slope);
  }
  int which = 0;
  if (a.want_w) keep_sums<LANES, P, VEC>(a, u, which++, dw);
  if (a.want_scale) keep_sums<LANES, P, VEC>(a, u, which++, ds);
}

}  // namespace

hipError_t launch_norm_after(const BlockNormArgs &a, bool bf16, bool rf32, bool back, hipStream_t s) {
  return dispatch(a, bf16, rf32, [&](auto t, auto r, auto vec, auto z) {
    constexpr int L = decltype(z)::lanes, P = decltype(z)::pieces;
    const uint32_t grid = norm_grid(a, L);
    if (back)
      after_back_kernel<decltype(t), decltype(r), L, P, decltype(vec)::value><<<grid, threads_of(L), 0, s>>>(a);
    else
      after_kernel<decltype(t), decltype(r), L, P, decltype(vec)::value><<<grid, threads_of(L), 0, s>>>(a);
  });
}

}  // namespace vmk
