// Device helpers of the norms around a block: a group of channels in the registers of
// 4 to 1024 lanes, in pieces of 8 values of which every lane has P.  Only sums cross
// lanes.  Sums over rows (of gains, biases, scales) are kept by workers, each of which
// walks every workers-th row of one group of columns, and are added up by a launch of
// their own.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "prompt_internal.h"
#include "vm_internal.h"

namespace vmk {
namespace {

// Threads of a workgroup whose groups have LANES lanes.
constexpr int threads_of(int lanes) { return lanes > 256 ? lanes : 256; }

template <typename T>
struct alignas(16) Eight {
  T v[16 / sizeof(T)];
};

// Pieces of 8 values.  VEC: whole, 16-byte aligned; else value by value, neighbouring
// lanes at neighbouring values.
template <int LANES, bool VEC>
__device__ __forceinline__ int place(int piece, int e, int lane) {
  return VEC ? (piece * LANES + lane) * 8 + e : (piece * 8 + e) * LANES + lane;
}

template <int LANES, int P, bool VEC, typename T>
__device__ __forceinline__ void load(const T *p, int size, int lane, float (&x)[P][8]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (VEC) {
      const int at = place<LANES, true>(i, 0, lane);
      if (at < size) {
        constexpr int k = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 8 / k; ++j) {
          const Eight<T> v = *reinterpret_cast<const Eight<T> *>(p + at + j * k);
#pragma unroll
          for (int e = 0; e < k; ++e) x[i][j * k + e] = to_f32(v.v[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = place<LANES, false>(i, e, lane);
        x[i][e] = at < size ? to_f32(p[at]) : 0.0f;
      }
    }
  }
}
template <int LANES, int P, bool VEC, typename T>
__device__ __forceinline__ void store(T *p, int size, int lane, const float (&x)[P][8]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (VEC) {
      const int at = place<LANES, true>(i, 0, lane);
      if (at < size) {
        constexpr int k = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 8 / k; ++j) {
          Eight<T> v;
#pragma unroll
          for (int e = 0; e < k; ++e)
            if constexpr (sizeof(T) == 2)
              v.v[e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[i][j * k + e]));   // (to nearest even)
            else
              v.v[e] = x[i][j * k + e];
          *reinterpret_cast<Eight<T> *>(p + at + j * k) = v;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = place<LANES, false>(i, e, lane);
        if (at < size) p[at] = from_f32<T>(x[i][e]);
      }
    }
  }
}

template <int CTRL>
__device__ __forceinline__ float moved(float x) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
// Sums of N values over the lanes of a group (LANES > 64: the workgroup, whose
// waves meet in `meet`; every thread comes through here equally often).
constexpr int kMeet = 16;
template <int LANES, int N>
__device__ __forceinline__ void sum_lanes(float (&s)[N], float (*meet)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] += moved<0xb1>(s[i]);                          // lane ^ 1
    s[i] += moved<0x4e>(s[i]);                          // lane ^ 2
    if (LANES > 4) {
      s[i] += moved<0x141>(s[i]);                       // the other four of each eight
      s[i] += moved<0x140>(s[i]);                       // the other eight of each row
    }
    if (LANES > 16) {
      auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(s[i]), __float_as_uint(s[i]), false, false);
      s[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
      r = __builtin_amdgcn_permlane32_swap(__float_as_uint(s[i]), __float_as_uint(s[i]), false, false);
      s[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
  }
  if (LANES > 64) {
    __syncthreads();
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) meet[threadIdx.x / 64][i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < LANES / 64; ++w) s[i] += meet[w][i];
    }
  }
}

// 1 / sqrt(x), to the last bit or so (the instruction's result and one step).
__device__ __forceinline__ float inverse_root(float x) {
  const float r = __builtin_amdgcn_rsqf(x);
  const float better = r * __builtin_fmaf(-0.5f * x * r, r, 1.5f);
  return x > 0.0f && x < __builtin_inff() ? better : r;
}

// A product that is rounded before it meets a sum.
__device__ __forceinline__ float rounded(float x) {
  asm("" : "+v"(x));
  return x;
}

// The gradient of a normed value v: with n = v s, S = sum v^2, E = sum e v over the group,
//   s (e - n mean(e n)) = s (e s^2 (eps + mean') - n s (E - e v) / size),
//   mean' = (S - v^2) / size.
// The value's own terms leave both sums before the difference is taken, so that a group
// whose other values are 0 (one of a single value always) keeps its eps term.
__device__ __forceinline__ float norm_back(float e, float v, float s, float S, float E, float over, float eps) {
  const float rest = (S - rounded(v * v)) * s * s, along = (E - rounded(e * v)) * s;
  return s * (e * __builtin_fmaf(over, rest, eps * s * s) - over * (v * s) * along);
}

__device__ __forceinline__ float silu_both(float z, float &slope) {
  const float s = hw_rcp(1.0f + hw_exp2(-z * kLog2e));
  slope = s * __builtin_fmaf(z, 1.0f - s, 1.0f);
  return z * s;
}

// A unit's place: units are (row, group of columns), `rows` units of one group in flight.
struct Unit {
  int64_t row;
  int grp, lane;
  bool live;
};
template <int LANES>
__device__ __forceinline__ Unit unit_of(const BlockNormArgs &a, int groups) {
  constexpr int kUnits = threads_of(LANES) / LANES;
  const int64_t id = blockIdx.x * static_cast<int64_t>(kUnits) + threadIdx.x / LANES;
  Unit u;
  u.row = id / groups;
  u.grp = static_cast<int>(id - u.row * groups);
  u.lane = threadIdx.x % LANES;
  u.live = u.row < a.workers;
  return u;
}

template <int LANES, int P, bool VEC>
__device__ __forceinline__ void keep_sums(const BlockNormArgs &a, const Unit &u, int which, const float (&s)[P][8]) {
  if (!u.live) return;
  float *p = a.partial + (static_cast<int64_t>(which) * a.workers + u.row) * a.dim + u.grp * a.group;
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = place<LANES, VEC>(i, e, u.lane);
      if (at < a.group) p[at] = s[i][e];
    }
}

// Columns' gains, biases and scales, 1 or 0 where there are none.
template <int LANES, int P, bool VEC>
__device__ __forceinline__ void load_columns(const float *p, int size, int lane, float other, float (&x)[P][8]) {
  if (p != nullptr) {
    load<LANES, P, VEC>(p, size, lane, x);
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = other;
  }
}

#define VM_EACH                       \
  _Pragma("unroll") for (int i = 0; i < P; ++i) _Pragma("unroll") for (int e = 0; e < 8; ++e)

// Lanes and pieces of a group: the fewest lanes that hold it in few registers.
struct Shape {
  int lanes, pieces;
};
inline Shape shape_of(int size) {
  if (size <= 32) return {4, 1};
  if (size <= 128) return {16, 1};
  if (size <= 512) return {64, 1};
  if (size <= 1024) return {64, 2};
  if (size <= 2048) return {256, 1};
  if (size <= 4096) return {256, 2};
  if (size <= 8192) return {512, 2};
  return {1024, 2};
}
// f(lanes, pieces) with both as types.
template <int L, int P>
struct ShapeType {
  static constexpr int lanes = L, pieces = P;
};
template <typename F>
hipError_t by_shape(int size, F &&f) {
  const Shape z = shape_of(size);
  if (z.lanes == 4)
    f(ShapeType<4, 1>());
  else if (z.lanes == 16)
    f(ShapeType<16, 1>());
  else if (z.lanes == 64 && z.pieces == 1)
    f(ShapeType<64, 1>());
  else if (z.lanes == 64)
    f(ShapeType<64, 2>());
  else if (z.lanes == 256 && z.pieces == 1)
    f(ShapeType<256, 1>());
  else if (z.lanes == 256)
    f(ShapeType<256, 2>());
  else if (z.lanes == 512)
    f(ShapeType<512, 2>());
  else
    f(ShapeType<1024, 2>());
  return hipGetLastError();
}

// Whether every row is whole 16-byte pieces.
inline bool whole_pieces(const BlockNormArgs &a) {
  if (a.dim % 8 != 0 || a.group % 8 != 0 || a.xs % 8 != 0 || a.zs % 8 != 0) return false;
  for (const void *p : {a.x, a.residual, a.z, static_cast<const void *>(a.w), static_cast<const void *>(a.b),
                        static_cast<const void *>(a.scale), static_cast<const void *>(a.y), static_cast<const void *>(a.r),
                        a.dy, a.dr, static_cast<const void *>(a.dx), static_cast<const void *>(a.dres),
                        static_cast<const void *>(a.dz)})
    if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return false;
  return true;
}

// launch(type of x, type of the residual, whole pieces, shape)
template <bool VEC, typename F>
hipError_t by_types(const BlockNormArgs &a, bool bf16, bool rf32, F &&launch) {
  return by_shape(a.group, [&](auto z) {
    constexpr std::integral_constant<bool, VEC> vec{};
    if (!bf16)
      launch(float{}, float{}, vec, z);
    else if (rf32)
      launch(bf16_t{}, float{}, vec, z);
    else
      launch(bf16_t{}, bf16_t{}, vec, z);
  });
}
template <typename F>
hipError_t dispatch(const BlockNormArgs &a, bool bf16, bool rf32, F &&launch) {
  return whole_pieces(a) ? by_types<true>(a, bf16, rf32, launch) : by_types<false>(a, bf16, rf32, launch);
}

inline uint32_t norm_grid(const BlockNormArgs &a, int lanes) {
  const int64_t units = static_cast<int64_t>(a.workers) * (a.dim / a.group), per = threads_of(lanes) / lanes;
  return static_cast<uint32_t>((units + per - 1) / per);
}

}  // namespace
}  // namespace vmk
