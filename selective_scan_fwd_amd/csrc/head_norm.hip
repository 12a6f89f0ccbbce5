// Per-head normalisation of queries and keys with gains and the rotation by
// position, and its gradients.
//
//   n = r x, r = 1 / sqrt(c sum x^2 + eps), c = 1/dim or 1;  y = rotate(w n)
//   back:  d = rotate^T(dy);  dw = sum d n;  e = w d;
//          dx_i = r (e_i - n_i c sum(e n))
//               = r^3 (eps e_i + c (e_i (sum x^2 - x_i^2) - x_i (sum(e x) - e_i x_i)))
// The second form of dx is computed: a value's own terms leave both sums before
// the difference is taken, so a head whose other values are 0 (a head of one value
// always) keeps its eps term, which the first form loses to cancellation.  Beside
// other values they leave the sums to within a rounding of the sums, 2^-24 of x^2
// for a value that dominates: there both forms are alike.
//
// Bound by memory: x is read once and y written once (back: x and dy read, dx
// written).  A head is held by a group of lanes, 8 values to a lane as two
// pieces of 4: values that the rotation pairs up, (i, i + rot/2) or (2i, 2i+1),
// meet in one lane, so the rotation needs no exchange and only the sum over
// the head crosses lanes.  A group keeps one token's angles in registers and
// walks over the token's heads, queries first, then keys.  4 x 4097 tokens, 24
// heads of 128, bf16 (206 MB): 59 us; backward, 128 x 197 tokens, 12 heads of 64,
// fp32 (233 MB): 58 us and 6 for the gains' sums.
#include <hip/hip_runtime.h>

#include "mixer_internal.h"
#include "vm_internal.h"

namespace vmk {
namespace {

constexpr int kThreads = 256;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// LAST: what is loaded is not used again soon.
template <bool LAST, typename V>
__device__ __forceinline__ V load_as(const V *p) {
  return LAST ? __builtin_nontemporal_load(p) : *p;
}
template <bool LAST = false>
__device__ __forceinline__ f32x4 load4(const float *p) {
  return load_as<LAST>(reinterpret_cast<const f32x4 *>(p));
}
template <bool LAST = false>
__device__ __forceinline__ f32x4 load4(const bf16_t *p) {
  const u16x4 r = load_as<LAST>(reinterpret_cast<const u16x4 *>(p));
  return f32x4{to_f32(r[0]), to_f32(r[1]), to_f32(r[2]), to_f32(r[3])};
}
__device__ __forceinline__ void store4(float *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }
__device__ __forceinline__ void store4(bf16_t *p, f32x4 v) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<bf16x4 *>(p) = __builtin_convertvector(v, bf16x4);   // (to nearest even)
}

// Where a lane's two pieces of 4 values lie in the head, and which angles turn
// them.  VEC: pieces are whole and aligned, so they move as one access; else
// each value is placed by itself and may be absent (dim not a multiple of 8).
struct Place {
  int at[2][4];     // index in the head, -1 = absent
  int angle[4];     // column of the tables, -1 = not rotated
};

// Pair number p of a head: below rot/2 the rotation's pairs, above it the
// remaining values two by two (an odd last one alone).
__device__ __forceinline__ void place_pair(int p, int dim, int rot, bool inter, int &i, int &j, int &angle) {
  const int half = rot >> 1;
  angle = -1;
  if (p < half) {
    i = inter ? 2 * p : p;
    j = inter ? 2 * p + 1 : p + half;
    angle = p;
  } else {
    const int rest = dim - rot, first = (rest + 1) >> 1, k = p - half;
    i = k < first ? rot + k : -1;
    j = k < first && first + k < rest ? rot + first + k : -1;
  }
}

template <bool VEC, bool LAST, typename T>
__device__ __forceinline__ void load_head(const T *x, const Place &pl, bool inter_piece, f32x4 &a, f32x4 &b) {
  if (VEC) {
    if (pl.at[0][0] < 0) {
      a = b = f32x4{0, 0, 0, 0};
    } else if (inter_piece) {
      const f32x4 u = load4<LAST>(x + pl.at[0][0]), v = load4<LAST>(x + pl.at[0][0] + 4);
      a = f32x4{u[0], u[2], v[0], v[2]};
      b = f32x4{u[1], u[3], v[1], v[3]};
    } else {
      a = load4<LAST>(x + pl.at[0][0]);
      b = load4<LAST>(x + pl.at[1][0]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = pl.at[0][e] >= 0 ? to_f32(x[pl.at[0][e]]) : 0.0f;
      b[e] = pl.at[1][e] >= 0 ? to_f32(x[pl.at[1][e]]) : 0.0f;
    }
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_head(T *y, const Place &pl, bool inter_piece, f32x4 a, f32x4 b) {
  if (VEC) {
    if (pl.at[0][0] < 0) return;
    if (inter_piece) {
      store4(y + pl.at[0][0], f32x4{a[0], b[0], a[1], b[1]});
      store4(y + pl.at[0][0] + 4, f32x4{a[2], b[2], a[3], b[3]});
    } else {
      store4(y + pl.at[0][0], a);
      store4(y + pl.at[1][0], b);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (pl.at[0][e] >= 0) y[pl.at[0][e]] = from_f32<T>(a[e]);
      if (pl.at[1][e] >= 0) y[pl.at[1][e]] = from_f32<T>(b[e]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
  return __builtin_fmaf(a[0], b[0], __builtin_fmaf(a[1], b[1], __builtin_fmaf(a[2], b[2], a[3] * b[3])));
}

// One value of dx (see above).  The squares and products are rounded by
// themselves: that is what a sum is in which all other terms are 0, and such a sum
// they leave exactly.  (A sum of more terms took some of them unrounded, and was
// rounded on the way.)
__device__ __forceinline__ float own_term(float e, float x, float squares, float along, float over, float eps, float r) {
#pragma clang fp contract(off)
  const float rest = e * (squares - x * x) - x * (along - e * x);
  return r * (r * r * __builtin_fmaf(over, rest, eps * e));
}

// LPR lanes hold one head.
template <typename T, int LPR, bool VEC, bool BACK>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs A) {
  constexpr int kGroups = kThreads / LPR;
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const bool inter_piece = VEC && A.interleaved && 4 * lane < (A.rot >> 1);
  Place pl;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    place_pair(4 * lane + e, A.dim, A.rot, A.interleaved != 0, pl.at[0][e], pl.at[1][e], pl.angle[e]);
  f32x4 w[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[m][h][e] = A.w[m] != nullptr && pl.at[h][e] >= 0 ? A.w[m][pl.at[h][e]] : 1.0f;
  f32x4 dw[2][2] = {};
  const int heads = A.heads[0] + A.heads[1];
  const int64_t items = A.tokens * A.splits;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kGroups + group; it < items;
       it += static_cast<int64_t>(gridDim.x) * kGroups) {
    const int64_t t = A.splits == 1 ? it : it / A.splits;
    const int first = A.splits == 1 ? 0 : static_cast<int>(it - t * A.splits);
    // The next head is on its way while one is worked on (4097 tokens of 4 rows:
    // 67 -> 63 us; two ahead gain nothing and cost the gradients 30 us), past its
    // last use forward (60 us; the gradients, with twice the loads, lose 3 us).
    f32x4 next_a, next_b, next_p, next_q;
    auto fetch = [&](int h) {
      const int m = h >= A.heads[0], hh = m ? h - A.heads[0] : h;
      load_head<VEC, !BACK>(static_cast<const T *>(A.x[m]) + t * A.xs[m] + static_cast<int64_t>(hh) * A.dim, pl, inter_piece,
                     next_a, next_b);
      if (BACK)
        load_head<VEC, !BACK>(static_cast<const T *>(A.dy[m]) + (t * A.heads[m] + hh) * A.dim, pl, inter_piece, next_p, next_q);
    };
    if (first < heads) fetch(first);
    f32x4 co = {1, 1, 1, 1}, si = {0, 0, 0, 0};
    bool live = true;
    if (A.rot > 0) {
      const int64_t p = A.pos != nullptr ? A.pos[t] : t % A.seqlen;
      live = p >= 0 && p < A.table;
      if (live) {
        const int64_t row = p * (A.rot >> 1);
        if (VEC) {                         // (rot is a multiple of 8, the tables 16-byte aligned)
          if (pl.angle[0] >= 0) {
            co = load4(A.cos + row + pl.angle[0]);
            si = load4(A.sin + row + pl.angle[0]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (pl.angle[e] >= 0) {
              co[e] = A.cos[row + pl.angle[e]];
              si[e] = A.sin[row + pl.angle[e]];
            }
        }
      }
    }
    for (int h = first; h < heads; h += A.splits) {
      const int m = h >= A.heads[0], hh = m ? h - A.heads[0] : h;
      T *y = static_cast<T *>(A.y[m]) + (t * A.heads[m] + hh) * A.dim;
      if (!live) {
        store_head<VEC>(y, pl, inter_piece, f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0});
        continue;
      }
      const f32x4 a = next_a, b = next_b, p = next_p, q = next_q;
      if (h + A.splits < heads) fetch(h + A.splits);
      const float squares = group_sum<LPR>(dot4(a, a) + dot4(b, b));
      const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(squares, A.over, A.eps));
      const f32x4 na = a * r, nb = b * r;
      const f32x4 wa = m ? w[1][0] : w[0][0], wb = m ? w[1][1] : w[0][1];
      if (!BACK) {
        const f32x4 ua = na * wa, ub = nb * wb;
        store_head<VEC>(y, pl, inter_piece, ua * co - ub * si, ub * co + ua * si);
      } else {
        const f32x4 da = p * co + q * si, db = q * co - p * si;
        if (m) {
          dw[1][0] += da * na;
          dw[1][1] += db * nb;
        } else {
          dw[0][0] += da * na;
          dw[0][1] += db * nb;
        }
        const f32x4 ea = da * wa, eb = db * wb;
        const float along = group_sum<LPR>(dot4(ea, a) + dot4(eb, b));
        f32x4 ga, gb;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ga[e] = own_term(ea[e], a[e], squares, along, A.over, A.eps, r);
          gb[e] = own_term(eb[e], b[e], squares, along, A.over, A.eps, r);
        }
        store_head<VEC>(y, pl, inter_piece, ga, gb);
      }
    }
  }
  if (BACK && A.partial != nullptr) {
    // the block's sums, in the order of its groups
    __shared__ float sums[kGroups][LPR * 8];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sums[group][lane * 8 + e] = dw[m][0][e];
        sums[group][lane * 8 + 4 + e] = dw[m][1][e];
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float s = 0;
            for (int k = 0; k < kGroups; ++k) s += sums[k][lane * 8 + 4 * h + e];
            if (pl.at[h][e] >= 0)
              A.partial[(static_cast<int64_t>(blockIdx.x) * 2 + m) * A.dim + pl.at[h][e]] = s;
          }
      }
      __syncthreads();
    }
  }
}

// dw[m][i] = sum over blocks, 64 lanes to a value.
__global__ __launch_bounds__(kThreads) void norm_dw_kernel(NormArgs A, int blocks) {
  const int i = blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
  if (i >= 2 * A.dim) return;
  const int m = i >= A.dim;
  if (A.dw[m] == nullptr) return;
  float s = 0;
  constexpr int kAhead = 8;                 // loads under way
  for (int b = threadIdx.x % 64; b < blocks; b += 64 * kAhead) {
    float x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      x[j] = b + 64 * j < blocks ? A.partial[static_cast<int64_t>(b + 64 * j) * 2 * A.dim + i] : 0.0f;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) s += x[j];
  }
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (threadIdx.x % 64 == 0) A.dw[m][i - m * A.dim] = s;
}

int lanes_per_head(int dim) {
  int l = 1;
  while (8 * l < dim) l *= 2;
  return l < 4 ? 4 : l;
}

bool aligned(const void *p, int64_t bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }

template <typename T, int LPR, bool VEC>
hipError_t launch_one(const NormArgs &a, int blocks, bool back, hipStream_t s) {
  if (back)
    hipLaunchKernelGGL((norm_kernel<T, LPR, VEC, true>), dim3(blocks), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((norm_kernel<T, LPR, VEC, false>), dim3(blocks), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t launch_dim(const NormArgs &a, int blocks, bool back, hipStream_t s) {
  switch (lanes_per_head(a.dim)) {
    case 4: return launch_one<T, 4, VEC>(a, blocks, back, s);
    case 8: return launch_one<T, 8, VEC>(a, blocks, back, s);
    case 16: return launch_one<T, 16, VEC>(a, blocks, back, s);
    case 32: return launch_one<T, 32, VEC>(a, blocks, back, s);
    case 64: return launch_one<T, 64, VEC>(a, blocks, back, s);
    default: return hipErrorInvalidValue;
  }
}

// Groups that share one token: one where the tokens alone give the card 16
// workgroups a compute unit, else up to a group per head.  (4097 tokens of 4
// rows, 24 heads of 128 in bf16, inputs not in the caches: 60 us, with 4
// workgroups 71, with 64 75.)
int head_splits(const NormArgs &a) {
  const int64_t want = 256 * 16 * (kThreads / lanes_per_head(a.dim));
  const int heads = a.heads[0] + a.heads[1];
  int64_t s = (want + a.tokens - 1) / a.tokens;
  return static_cast<int>(s < 1 ? 1 : s > heads ? heads : s);
}

}  // namespace

int norm_blocks(const NormArgs &a, bool back) {
  const int groups = kThreads / lanes_per_head(a.dim);
  const int64_t items = a.tokens * head_splits(a);
  const int64_t blocks = (items + groups - 1) / groups;
  const int64_t most = back ? kNormMaxBlocks : 4096;
  return static_cast<int>(blocks < most ? blocks : most);
}

hipError_t launch_norm(NormArgs a, bool bf16, bool back, hipStream_t s) {
  a.splits = head_splits(a);
  const int blocks = norm_blocks(a, back);
  // whole pieces of 4 values, 4 values aligned
  const int64_t piece = bf16 ? 8 : 16;
  bool vec = a.dim % 8 == 0 && a.rot % 8 == 0 && aligned(a.cos, 16) && aligned(a.sin, 16);
  for (int m = 0; m < 2; ++m)
    vec = vec && (a.heads[m] == 0 || (aligned(a.x[m], piece) && aligned(a.y[m], piece) && a.xs[m] % 4 == 0 &&
                                      (!back || aligned(a.dy[m], piece))));
  hipError_t e;
  if (bf16)
    e = vec ? launch_dim<bf16_t, true>(a, blocks, back, s) : launch_dim<bf16_t, false>(a, blocks, back, s);
  else
    e = vec ? launch_dim<float, true>(a, blocks, back, s) : launch_dim<float, false>(a, blocks, back, s);
  if (e == hipSuccess && back && a.partial != nullptr) {
    hipLaunchKernelGGL(norm_dw_kernel, dim3((2 * a.dim + 3) / 4), dim3(kThreads), 0, s, a, blocks);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace vmk
