// Sums over the rows of fp32 matrices, in fp64 and a fixed order: the last step of the
// gradients that every token or row adds to.  16 columns to a workgroup and 64 threads
// to a column, so that few columns of many rows fill the card too; several matrices to
// a launch.
#include <hip/hip_runtime.h>

#include "prompt_internal.h"

namespace vmk {
namespace {

constexpr int kCols = 16, kRowsAt = 64;

__global__ __launch_bounds__(kCols * kRowsAt) void column_sums_kernel(ColumnSums all) {
  __shared__ double part[kRowsAt][kCols];
  int k = 0;
  while (k + 1 < all.n && static_cast<int>(blockIdx.x) >= all.first[k + 1]) ++k;
  const ColumnSum &m = all.s[k];
  const int col = (blockIdx.x - all.first[k]) * kCols + threadIdx.x % kCols, row = threadIdx.x / kCols;
  double s = 0.0;
  if (col < m.fold)
    for (int c = col; c < m.cols; c += m.fold) {
      const float *in = m.in + c;
      double t[4] = {0, 0, 0, 0};
      int64_t r = row;
      for (; r + 3 * kRowsAt < m.rows; r += 4 * kRowsAt)
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] += in[(r + i * kRowsAt) * m.pitch];
      for (; r < m.rows; r += kRowsAt) t[0] += in[r * m.pitch];
      s += (t[0] + t[1]) + (t[2] + t[3]);
    }
  part[row][threadIdx.x % kCols] = s;
  __syncthreads();
  if (row < 8) {
    s = 0.0;
#pragma unroll
    for (int i = 0; i < kRowsAt; i += 8) s += part[row + i][threadIdx.x % kCols];
  }
  __syncthreads();
  if (row < 8) part[row][threadIdx.x % kCols] = s;
  __syncthreads();
  if (row == 0 && col < m.fold) {
    s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
    m.out[col] = static_cast<float>(s);
  }
}

}  // namespace

void add_sum(ColumnSums &all, const float *in, float *out, int64_t rows, int64_t pitch, int cols, int fold) {
  if (out == nullptr) return;
  all.s[all.n] = {in, out, rows, pitch, cols, fold};
  all.first[all.n + 1] = all.first[all.n] + (fold + kCols - 1) / kCols;
  ++all.n;
}

hipError_t launch_column_sums(const ColumnSums &all, hipStream_t s) {
  if (all.n == 0) return hipSuccess;
  column_sums_kernel<<<all.first[all.n], kCols * kRowsAt, 0, s>>>(all);
  return hipGetLastError();
}

}  // namespace vmk
