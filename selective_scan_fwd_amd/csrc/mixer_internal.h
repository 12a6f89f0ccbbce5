// Internal declarations of the matrix-state mixer kernels (gated delta rule,
// per-head norm and rotation, gradient clipping).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "vm_scan.h"

namespace vmk {

// ------------------------------------------------------ norm and rotation
struct NormArgs {
  const void *x[2];       // q, k: [tokens][heads][dim], token stride xs (elements)
  const float *w[2];      // gains or nullptr
  void *y[2];             // forward: outputs (dense); backward: gradients of x
  const void *dy[2];      // backward: gradients of the outputs (dense)
  float *partial;         // backward: [blocks][2][dim] sums for dw, or nullptr
  float *dw[2];
  const float *cos, *sin;
  const int32_t *pos;
  int64_t xs[2];
  int64_t tokens, seqlen, table;
  int heads[2];
  int dim, rot;
  float eps, over;        // over: 1 / dim, or 1 for the Euclidean norm
  int interleaved;
  int splits;             // lane groups that share one token's heads
};
constexpr int kNormMaxBlocks = 1024;
// Blocks of the launch (the number of partial sums of the backward pass).
int norm_blocks(const NormArgs &a, bool back);
hipError_t launch_norm(NormArgs a, bool bf16, bool back, hipStream_t s);

// ------------------------------------------------------------- clipping
constexpr int kClipTable = 120;        // tensors of one launch (kernel arguments)
constexpr int64_t kClipChunk = 2048;   // elements
constexpr uint32_t kClipRun = 8;       // chunks of a block at a time, at most
constexpr int kClipPartials = 1024;   // blocks of a launch, at most: four of 512 threads fill a compute unit
struct ClipTable {
  const void *in[kClipTable];
  void *out[kClipTable];
  int64_t elems[kClipTable];
  uint32_t first[kClipTable + 1];      // first chunk of each tensor
  uint8_t bf16[kClipTable];
  int n;
};
// Adds to the first `have` partial sums, writes the rest of its blocks'.
hipError_t launch_clip_sums(const ClipTable &t, double *partial, int have, int blocks, hipStream_t s);
hipError_t launch_clip_scale(const ClipTable &t, const double *partial, int partials, float max_norm,
                             float *norm, int blocks, hipStream_t s);
hipError_t launch_clip_norm_only(const double *partial, int partials, float *norm, hipStream_t s);

// ------------------------------------------------------ gated delta rule
constexpr int kDeltaChunk = 64;
struct DeltaArgs {
  const void *q, *k, *v;
  const float *g, *beta, *h0;
  const int32_t *off;
  int64_t qs, ks, vs;      // token strides (elements)
  int64_t L;               // tokens of a batch row
  int64_t slots;           // chunk slots over all sequences
  int nseq, hk, hv, dk, dv;
  int reverse;
  float scale;
  // Per (slot, value head), written by the preparing kernel: T = (I + A)^-1 and
  // the scaled masked products P of queries and keys, in the order in which a
  // wave loads them as the left operand of a matrix instruction, [block of
  // 16 x 32][lane][8], the 6 blocks that are not zero.  For bf16 tokens in bf16
  // terms, which go to LDS as they are; for fp32 tokens in fp32, which passes
  // through registers on its way there and is split into three terms then.
  uint16_t *T;             // forward: T, then P; backward: T
  uint16_t *TT;            // backward: the transposes of T, then of P
  float *eg, *ew;          // [64]: exp(G), exp(G_C - G) of the running log decay G
  double *gam;             // [64]: G (backward)
  // forward
  void *out;
  float *state;
  // backward
  const void *dout;
  const float *dstate;
  // per (slot, value head), rows of dvp = dv rounded up to 16 values, zero past dv
  int dvp;
  float *S;                // [dk][dvp]: state at the chunk's start
  float *V;                // [64][dvp]: the chunk's corrected values
  float *dS;               // [dk][dvp]: gradient of the state at the chunk's end
  float *dR;               // [64][dvp]
  void *dq, *dkey, *dval;
  float *dg, *dbeta, *dh0;
};
// Terms of bf16 that stand for an fp32 value: 8 bits each, so three hold all 24.
// All are kept of every operand, those that enter a bf16 output only among them:
// with two, the parts of an output that cancel (a large state read back and the
// chunk's own values) leave an error past the output's rounding (first states of
// 2000 times the values: 4e-2), and 3e-3 of the outputs round to another side.
constexpr int kTerms = 3;
// What a triangular matrix takes in memory, in units of one term.
inline constexpr int tri_units(bool bf16) { return bf16 ? kTerms : 2; }
constexpr int kTriBlocks = 6;
constexpr int64_t kTriTerm = kTriBlocks * 64 * 8;   // values of one term
// Whether every row of q and k is whole 16-byte pieces, and those of v (the
// backward scan: dout, of token stride os) whole 4-byte ones.
inline bool delta_vec(const DeltaArgs &a, int64_t esize) {
  return a.dk % 8 == 0 && (a.qs * esize) % 16 == 0 && (a.ks * esize) % 16 == 0 &&
         (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && (reinterpret_cast<uintptr_t>(a.k) & 15) == 0;
}
inline bool delta_vec_values(const DeltaArgs &a, const void *v, int64_t stride, int64_t esize, int64_t bytes) {
  return (a.dv * esize) % bytes == 0 && (stride * esize) % bytes == 0 &&
         (reinterpret_cast<uintptr_t>(v) % bytes) == 0;
}
// Chunk slots of `n` sequences over L tokens in all (packed) or each.
int64_t delta_slots(int64_t batch, int64_t L, int64_t n, bool packed);
// backward: TT, PT and gam instead of P.
hipError_t launch_delta_prep(const DeltaArgs &a, bool bf16, bool backward, hipStream_t s);
// Forward: out and state; back: S and V, and dS, dR, dv and dh0.
hipError_t launch_delta_scan(const DeltaArgs &a, bool bf16, bool back, hipStream_t s);
// Work-items of that launch.
int64_t delta_scan_items(const DeltaArgs &a, bool bf16, bool back);
hipError_t launch_delta_grad(const DeltaArgs &a, bool bf16, hipStream_t s);

struct StepArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  float *state;
  const int32_t *slots;
  void *out;
  float scale;
  int64_t n_slots;
  int batch, hk, hv, dk, dv;
};
hipError_t launch_delta_step(const StepArgs &a, bool bf16, hipStream_t s);

}  // namespace vmk
