// Helpers shared by the C-ABI files: extents of host-visible arguments and
// temporary device memory.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <vector>

#include "vm_scan.h"

namespace vmk {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxElems = int64_t{1} << 40;

struct Span {
  uintptr_t lo = 0, hi = 0;  // [lo, hi)
};
inline Span span(const void *p, int64_t bytes) {
  Span s;
  if (p != nullptr) {
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + static_cast<uintptr_t>(bytes);
  }
  return s;
}
inline bool overlaps(Span a, Span b) { return a.lo != 0 && b.lo != 0 && a.lo < b.hi && b.lo < a.hi; }

inline bool dims_ok(std::initializer_list<int64_t> dims, int64_t *prod) {
  int64_t p = 1;
  for (int64_t d : dims) {
    if (d <= 0 || d > kMaxDim) return false;
    if (p > kMaxElems / d) return false;
    p *= d;
  }
  *prod = p;
  return true;
}

// The library's memory pool of the current device (created on first use).
hipError_t pool_for_current_device(hipMemPool_t *out);

// Temporary fp32 buffers that live on `stream` for the duration of one call.
// Requests below kChunk bytes are carved, 256-byte aligned, from shared
// chunks of kChunk bytes; larger ones get an allocation of their own.  Each
// pool free costs the host about 5 to 30 microseconds, so a backward call's
// dozen buffers freed one by one took longer on the host than its kernels
// on the GPU.
class Scratch {
 public:
  explicit Scratch(hipStream_t s) : s_(s) {}
  ~Scratch() {
    for (void *p : ptrs_) (void)hipFreeAsync(p, s_);
  }
  void *bytes(int64_t n, int *status) {
    if (*status != VM_OK) return nullptr;
    const size_t need = (static_cast<size_t>(n) + 255) & ~static_cast<size_t>(255);
    if (need >= kChunk) return alloc(need, status);
    if (base_ == nullptr || used_ + need > kChunk) {
      base_ = static_cast<char *>(alloc(kChunk, status));
      used_ = 0;
      if (base_ == nullptr) return nullptr;
    }
    void *p = base_ + used_;
    used_ += need;
    return p;
  }
  float *get(int64_t floats, int *status) { return static_cast<float *>(bytes(floats * 4, status)); }

 private:
  static constexpr size_t kChunk = size_t{64} << 20;
  void *alloc(size_t n, int *status) {
    hipMemPool_t pool;
    void *p = nullptr;
    if (pool_for_current_device(&pool) != hipSuccess ||
        hipMallocFromPoolAsync(&p, n, pool, s_) != hipSuccess) {
      (void)hipGetLastError();
      *status = VM_ERR_ALLOC;
      return nullptr;
    }
    ptrs_.push_back(p);
    return p;
  }
  hipStream_t s_;
  std::vector<void *> ptrs_;
  char *base_ = nullptr;      // the current chunk, and the bytes of it handed out
  size_t used_ = 0;
};

// Extent in elements of [batch, seqlen, heads, dim] with a token stride
// (0 = dense); false if the stride is short or the extent overflows.
inline bool token_extent(int64_t batch, int64_t seqlen, int64_t heads, int64_t dim, int64_t *stride, int64_t *extent) {
  int64_t unused = 0;
  if (!dims_ok({batch, seqlen, heads, dim}, &unused)) return false;
  if (*stride == 0) *stride = heads * dim;
  if (*stride < heads * dim || !dims_ok({batch, seqlen, *stride}, &unused)) return false;
  *extent = (batch * seqlen - 1) * *stride + heads * dim;
  return true;
}

template <int N, int M>
bool any_overlap(const Span (&outs)[N], const Span (&ins)[M]) {
  for (int i = 0; i < N; ++i) {
    for (int j = 0; j < M; ++j)
      if (overlaps(outs[i], ins[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

// Temporary memory of one call in one piece: the parts are laid out first, then
// taken from the caller's workspace or from the pool (where each allocation and
// free costs the host some 10 us).
class Parts {
 public:
  static constexpr int64_t whole(int64_t bytes) { return (bytes + 255) & ~int64_t{255}; }
  template <typename P>
  void add(P **to, int64_t bytes) {
    to_[n_] = reinterpret_cast<void **>(to);
    at_[n_++] = total_;
    total_ += whole(bytes);
  }
  int64_t total() const { return total_; }
  int get(void *workspace, int64_t bytes, Scratch &ws) {
    int st = VM_OK;
    char *base = static_cast<char *>(workspace);
    if (base == nullptr)
      base = static_cast<char *>(ws.bytes(total_, &st));
    else if (bytes < total_ || (reinterpret_cast<uintptr_t>(base) & 255) != 0)
      st = VM_ERR_ALLOC;
    if (st == VM_OK)
      for (int i = 0; i < n_; ++i) *to_[i] = base + at_[i];
    return st;
  }

 private:
  void **to_[12];
  int64_t at_[12], total_ = 0;
  int n_ = 0;
};

inline int hip_status(hipError_t e) { return e == hipSuccess ? VM_OK : VM_ERR_HIP; }

}  // namespace vmk
