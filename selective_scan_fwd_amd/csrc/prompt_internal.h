// Internal declarations of the prompt and token kernels (selective scan and its
// short convolution over rows of tokens) and of the norms around a block.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "vm_scan.h"

namespace vmk {

// Sequences of a call and their division in chunks of tokens.  Tokens are
// counted over all batch rows.  A slot is one chunk: dense sequences have
// ceil(L / chunk) slots each; packed sequence i has its slots from
// offsets[i] / chunk + i on, which leaves each sequence as many as it needs.
struct SeqArgs {
  const int32_t *off;        // packed: [nseq + 1], else nullptr
  const int32_t *where;      // slot of each sequence in the kept states, nullptr = its number
  const int32_t *fresh;      // nonzero: starts from zero, nullptr = none does
  int64_t L;                 // tokens of a batch row
  int64_t chunk;             // tokens of a chunk
  int64_t slots;             // chunks of the launch
  int64_t kept;              // number of kept states
  int nseq;
  int clear;                 // workgroups behind a launch's others that clear rows of no sequence
};
// Those workgroups for rows of `dim` values: one to 8192 of them, as no launch of its own is
// wanted for what is mostly little or nothing.  40 packed prompts of 4096 channels, 8187 tokens in
// all: 1 us with nothing to clear; as many rows again cost the convolution 7 us, the scan 27.
constexpr int kMostClear = 256;
inline int clear_blocks(int64_t L, int64_t dim) {
  const int64_t n = L * dim / 8192 + 1;
  return static_cast<int>(n < kMostClear ? n : kMostClear);
}
int64_t seq_slots(int64_t nseq, int64_t L, int64_t chunk, bool packed);

// ---------------------------------------------------- column sums
// out[c % fold] = sum over rows r and over c of in[r * pitch + c], c < cols.
struct ColumnSum {
  const float *in;
  float *out;
  int64_t rows, pitch;
  int cols, fold;
};
constexpr int kMaxSums = 6;
struct ColumnSums {
  ColumnSum s[kMaxSums];
  int first[kMaxSums + 1];   // first block of each
  int n;
};
void add_sum(ColumnSums &all, const float *in, float *out, int64_t rows, int64_t pitch, int cols, int fold);
hipError_t launch_column_sums(const ColumnSums &all, hipStream_t s);

// ---------------------------------------------------- convolution
constexpr int kMaxTaps = 4;
struct PromptConvArgs {
  SeqArgs q;
  const void *x;
  const float *w, *bias;
  const void *h0;            // [kept][width - 1][dim]
  void *state;               // the same, or nullptr
  void *out;
  int64_t xs;                // token stride of x
  int dim, width, silu;
  // backward
  const void *dout, *dstate;
  void *dx, *dh0;
  float *partial;            // [workers][width + 1][dim]
  int workers;
};
// Tokens of a chunk.  Forty prompts of 1 to 1500 tokens, 4096 channels: 24 33 us, 16 and 32
// 37, 64 43; backward, 128 x 197 tokens of 384 channels: 32 35 us, 16 40, 64 50.
constexpr int64_t kConvChunk = 24, kConvBackChunk = 32;
// Workers of the backward pass: each walks every workers-th chunk.
int conv_workers(const PromptConvArgs &a, bool bf16);
hipError_t launch_prompt_conv(const PromptConvArgs &a, bool bf16, hipStream_t s);
hipError_t launch_prompt_conv_back(const PromptConvArgs &a, bool bf16, hipStream_t s);

struct TokenConvArgs {
  const void *x;
  const float *w, *bias;
  void *state;
  const int32_t *where;
  void *out;
  int64_t xs, kept;
  int batch, dim, width, silu;
};
hipError_t launch_token_conv(const TokenConvArgs &a, bool bf16, hipStream_t s);

// ---------------------------------------------------- scan
struct PromptScanArgs {
  SeqArgs q;
  const void *u, *delta, *B, *C, *z;
  const float *A, *D, *bias, *h0;
  float *state;              // [kept][dim][n]
  void *out;
  int64_t us, ds, bs, cs, zs;   // token strides
  int dim, n, softplus;
  // Per (slot, block of 16 channels), [64 lanes][4 states] and [16]: a chunk's
  // states from zero (nullptr: every sequence is one chunk) and its steps' sum.
  float *ends, *steps;
  // backward
  const void *dout;          // dense
  const float *dstate;
  void *du, *ddelta, *dB, *dC, *dz;   // dense
  float *dh0;
  float *starts;             // as ends: gradients of the states before a chunk
  // [tile][block][64][4]: states at the tiles' starts (with several chunks from zero at
  // the chunk's, and then [tile][block][16]: the sum of the chunk's steps before them).
  // A chunk's tiles have the numbers from (first token) / kBackTile + (its slot in the
  // tokens' order) on.
  float *marks, *before;
  float *partA, *partD;      // [slot][dim][n], [slot][2][dim]
  float *partBC;             // [workgroup's blocks][token][2 n]
};
// Blocks of 16 channels, and as many as whole workgroups hold.
inline int scan_blocks(int dim) { return (dim + 15) / 16; }
inline int scan_wide(int dim) { return (scan_blocks(dim) + 3) / 4; }
constexpr int kBackTile = 8;     // tokens of a tile of the backward pass
constexpr int kScanWaves = 4;     // blocks of 16 channels to a workgroup
int64_t scan_chunk(int64_t tokens, int64_t nseq, int64_t L, int dim, bool packed);
int64_t scan_back_chunk(int64_t tokens, int64_t nseq, int64_t L, int dim, bool packed);
hipError_t launch_prompt_scan(const PromptScanArgs &a, bool bf16, hipStream_t s);
hipError_t launch_prompt_scan_back(const PromptScanArgs &a, bool bf16, hipStream_t s);

struct TokenScanArgs {
  const void *u, *delta, *B, *C, *z;
  const float *A, *D, *bias;
  float *state;
  const int32_t *where;
  void *out;
  int64_t us, ds, bs, cs, zs, kept;
  int batch, dim, n, softplus;
};
hipError_t launch_token_scan(const TokenScanArgs &a, bool bf16, hipStream_t s);

// ---------------------------------------------------- norms around a block
struct BlockNormArgs {
  const void *x, *residual, *z;
  const float *w, *b, *scale;
  void *y, *r;
  int64_t xs, zs;            // row strides of x and z (the rest is dense)
  int64_t rows;
  int dim, group;
  int wide;                  // w has dim values (else group)
  float eps, factor;
  int center, gate_first;
  // backward
  const void *dy, *dr;
  void *dx, *dres, *dz;
  float *partial;            // [which][workers][dim]: gains, biases, scales
  int workers;               // rows in flight
  int want_w, want_b, want_scale;
};
int norm_workers(const BlockNormArgs &a);
// rf32: the residual is fp32 (else it has the type of x)
hipError_t launch_norm_before(const BlockNormArgs &a, bool bf16, bool rf32, bool back, hipStream_t s);
hipError_t launch_norm_after(const BlockNormArgs &a, bool bf16, bool rf32, bool back, hipStream_t s);

}  // namespace vmk
