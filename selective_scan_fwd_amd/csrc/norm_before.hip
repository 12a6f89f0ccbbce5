// The norm before a block of a language model, and its gradients:
//   r = residual + factor scale x,   y = (r - mean) s w + b,
//   s = 1 / sqrt(mean (r - mean)^2 + eps); without `center` the mean counts as 0.
//   back: n = (r - mean) s, e = w dy,
//         dr += s (e - mean(e) - n mean(e n)),  dx = factor scale dr,
//         dw = sum dy n, db = sum dy, dscale = factor sum dr x
// Bound by memory: every input is read once and every output written once.  Backward of
// 4 x 4097 rows of 2048, bf16 beside an fp32 residual, with a scale (604 MB): 124 us, 4.9 TB/s.
// (The next row's loads ahead in registers took it to 137: they cost the fourth wave.)  Above 8192
// channels the backward pass spills: bf16, without a scale, 8192 rows of 8192 179 us (3.0 TB/s),
// 4096 of 16384 378 (1.4); forward 98 both.
#include <hip/hip_runtime.h>

#include "block_norm.h"

namespace vmk {
namespace {

// ---------------------------------------------------------------- before
template <typename T, typename R, int LANES, int P, bool VEC>
__global__ __launch_bounds__(threads_of(LANES)) void before_kernel(BlockNormArgs a) {
  __shared__ float meet[kMeet][1], meet2[kMeet][1];
  const Unit u = unit_of<LANES>(a, 1);
  const int64_t row = u.live ? u.row : 0;
  float r[P][8], t[P][8];
  load<LANES, P, VEC>(static_cast<const T *>(a.x) + row * a.xs, a.dim, u.lane, r);
  if (a.scale != nullptr) {
    load<LANES, P, VEC>(a.scale, a.dim, u.lane, t);
    VM_EACH r[i][e] *= t[i][e];
  }
  if (a.factor != 1.0f) VM_EACH r[i][e] *= a.factor;
  if (a.residual != nullptr) {
    load<LANES, P, VEC>(static_cast<const R *>(a.residual) + row * a.dim, a.dim, u.lane, t);
    VM_EACH r[i][e] += t[i][e];
  }
  if (a.r != nullptr && u.live) store<LANES, P, VEC>(static_cast<R *>(a.r) + row * a.dim, a.dim, u.lane, r);
  if (a.center) {
    float m[1] = {0.0f};
    VM_EACH m[0] += r[i][e];
    sum_lanes<LANES, 1>(m, meet2);
    m[0] /= static_cast<float>(a.dim);
    VM_EACH r[i][e] = place<LANES, VEC>(i, e, u.lane) < a.dim ? r[i][e] - m[0] : 0.0f;
  }
  float s[1] = {0.0f};
  VM_EACH s[0] = __builtin_fmaf(r[i][e], r[i][e], s[0]);
  sum_lanes<LANES, 1>(s, meet);
  const float size = inverse_root(s[0] / static_cast<float>(a.dim) + a.eps);
  load_columns<LANES, P, VEC>(a.w, a.dim, u.lane, 1.0f, t);
  VM_EACH r[i][e] = r[i][e] * size * t[i][e];
  if (a.b != nullptr) {
    load<LANES, P, VEC>(a.b, a.dim, u.lane, t);
    VM_EACH r[i][e] += t[i][e];
  }
  if (u.live) store<LANES, P, VEC>(static_cast<T *>(a.y) + row * a.dim, a.dim, u.lane, r);
}

template <typename T, typename R, int LANES, int P, bool VEC>
__global__ __launch_bounds__(threads_of(LANES)) void before_back_kernel(BlockNormArgs a) {
  __shared__ float meet[kMeet][1], meet2[kMeet][3];
  const Unit u = unit_of<LANES>(a, 1);
  float w[P][8], scale[P][8], dw[P][8], db[P][8], ds[P][8];
  load_columns<LANES, P, VEC>(a.w, a.dim, u.lane, 1.0f, w);
  load_columns<LANES, P, VEC>(a.scale, a.dim, u.lane, 1.0f, scale);
  VM_EACH {
    scale[i][e] *= a.factor;
    dw[i][e] = db[i][e] = ds[i][e] = 0.0f;
  }
  const float over = 1.0f / static_cast<float>(a.dim);
  // (LANES = 256: every thread of the workgroup has the same rows)
  for (int64_t row = u.row; row < a.rows && u.live; row += a.workers) {
    float r[P][8], d[P][8];
    load<LANES, P, VEC>(static_cast<const R *>(a.r) + row * a.dim, a.dim, u.lane, r);
    load<LANES, P, VEC>(static_cast<const T *>(a.dy) + row * a.dim, a.dim, u.lane, d);
    if (a.center) {
      float m[1] = {0.0f};
      VM_EACH m[0] += r[i][e];
      sum_lanes<LANES, 1>(m, meet);
      VM_EACH r[i][e] = place<LANES, VEC>(i, e, u.lane) < a.dim ? r[i][e] - m[0] * over : 0.0f;
    }
    float s[3] = {0.0f, 0.0f, 0.0f};           // squares, e n / size, e
    VM_EACH {
      s[0] = __builtin_fmaf(r[i][e], r[i][e], s[0]);
      const float g = rounded(d[i][e] * w[i][e]);
      s[1] = __builtin_fmaf(g, r[i][e], s[1]);
      s[2] += g;
    }
    sum_lanes<LANES, 3>(s, meet2);
    const float size = inverse_root(s[0] * over + a.eps);
    const float mean = a.center ? s[2] * over : 0.0f;
    VM_EACH {
      const float n = r[i][e] * size;
      dw[i][e] = __builtin_fmaf(d[i][e], n, dw[i][e]);
      db[i][e] += d[i][e];
      d[i][e] = norm_back(rounded(d[i][e] * w[i][e]) - mean, r[i][e], size, s[0], s[1], over, a.eps);
    }
    if (a.dr != nullptr) {
      load<LANES, P, VEC>(static_cast<const R *>(a.dr) + row * a.dim, a.dim, u.lane, r);
      VM_EACH d[i][e] += r[i][e];
    }
    if (a.dres != nullptr) store<LANES, P, VEC>(static_cast<R *>(a.dres) + row * a.dim, a.dim, u.lane, d);
    if (a.want_scale) {
      load<LANES, P, VEC>(static_cast<const T *>(a.x) + row * a.xs, a.dim, u.lane, r);
      VM_EACH ds[i][e] = __builtin_fmaf(d[i][e] * a.factor, r[i][e], ds[i][e]);
    }
    if (a.dx != nullptr) {
      VM_EACH d[i][e] *= scale[i][e];
      store<LANES, P, VEC>(static_cast<T *>(a.dx) + row * a.dim, a.dim, u.lane, d);
    }
  }
  int which = 0;
  if (a.want_w) keep_sums<LANES, P, VEC>(a, u, which++, dw);
  if (a.want_b) keep_sums<LANES, P, VEC>(a, u, which++, db);
  if (a.want_scale) keep_sums<LANES, P, VEC>(a, u, which++, ds);
}

}  // namespace

int norm_workers(const BlockNormArgs &a) {
  // rows in flight: about 2048 waves' worth (128 x 197 rows of 384 after a block: 49 us, half as
  // many 50, with 4 x 4097 rows of 2048 before one 124 and 190; twice as many 84 and 124)
  const Shape z = shape_of(a.group);
  const int64_t units = 2048 * 64 / z.lanes, groups = a.dim / a.group;
  const int64_t most = units / groups > 0 ? units / groups : 1;
  return static_cast<int>(a.rows < most ? a.rows : most);
}

hipError_t launch_norm_before(const BlockNormArgs &a, bool bf16, bool rf32, bool back, hipStream_t s) {
  return dispatch(a, bf16, rf32, [&](auto t, auto r, auto vec, auto z) {
    constexpr int L = decltype(z)::lanes, P = decltype(z)::pieces;
    const uint32_t grid = norm_grid(a, L);
    if (back)
      before_back_kernel<decltype(t), decltype(r), L, P, decltype(vec)::value><<<grid, threads_of(L), 0, s>>>(a);
    else
      before_kernel<decltype(t), decltype(r), L, P, decltype(vec)::value><<<grid, threads_of(L), 0, s>>>(a);
  });
}

}  // namespace vmk
