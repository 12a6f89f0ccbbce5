// C ABI of the prompt and token operators (declared in include/vm_scan.h):
// argument checks, temporary memory and dispatch of the selective scan and its
// convolution over rows of tokens and single tokens, and of the norms around a
// block.  Every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_util.h"
#include "prompt_internal.h"
#include "vm_scan.h"

namespace {

using vmk::Parts;
using vmk::Scratch;
using vmk::Span;
using vmk::any_overlap;
using vmk::dims_ok;
using vmk::hip_status;
using vmk::span;
using vmk::token_extent;

constexpr int64_t kMaxState = 16, kMaxNorm = 16384;
// Token strides of prompts: a tile's rows are reached with 31-bit byte offsets.
constexpr int64_t kMaxStride = (int64_t{1} << 23) - 1;
// Workgroups of 256 work-items, of which a launch holds less than 2^32.
constexpr int64_t kMaxBlocks = (int64_t{1} << 24) - 1;
constexpr int64_t kMaxDim = int64_t{1} << 22;

bool type_ok(int dtype) { return dtype == VM_F32 || dtype == VM_BF16; }
int size_of(int dtype) { return dtype == VM_BF16 ? 2 : 4; }

// A call's sequences over rows of `dim` values; `kept` elements of all kept states of `each`
// elements.
int check_sequences(const vm_sequences *q, int64_t batch, int64_t seqlen, int64_t dim, bool pool, int64_t each, int clear,
                    vmk::SeqArgs *s, int64_t *kept) {
  int64_t tokens = 0;
  if (!dims_ok({batch, seqlen}, &tokens)) return VM_ERR_SHAPE;
  const int64_t n = q != nullptr ? q->n : batch;
  s->off = q != nullptr ? q->offsets : nullptr;
  s->where = q != nullptr ? q->slots : nullptr;
  s->fresh = q != nullptr ? q->fresh : nullptr;
  if (!pool && (s->where != nullptr || s->fresh != nullptr)) return VM_ERR_FLAG;
  if (s->off != nullptr ? batch != 1 : n != batch) return VM_ERR_SHAPE;
  s->kept = s->where != nullptr ? q->n_slots : n;
  int64_t unused = 0;
  if (!dims_ok({n}, &unused) || !dims_ok({s->kept, each}, kept)) return VM_ERR_SHAPE;
  s->nseq = static_cast<int>(n);
  s->L = seqlen;
  s->clear = clear != 0 && s->off != nullptr ? vmk::clear_blocks(seqlen, dim) : 0;
  return VM_OK;
}
int64_t all_tokens(const vmk::SeqArgs &s) { return s.off != nullptr ? s.L : s.L * s.nseq; }

void divide(vmk::SeqArgs &s, int64_t chunk) {
  s.chunk = chunk;
  s.slots = vmk::seq_slots(s.nseq, s.L, chunk, s.off != nullptr);
}

// What a call's sequences are read from.
struct SeqSpans {
  Span off, where, fresh;
  explicit SeqSpans(const vmk::SeqArgs &s)
      : off(span(s.off, (static_cast<int64_t>(s.nseq) + 1) * 4)), where(span(s.where, static_cast<int64_t>(s.nseq) * 4)),
        fresh(span(s.fresh, static_cast<int64_t>(s.nseq) * 4)) {}
};

// ------------------------------------------------------------ convolution
int check_conv(const vm_sequences *q, bool pool, const void *x, int64_t x_stride, const float *w, int64_t batch, int64_t seqlen,
               int64_t dim, int64_t width, int silu, int dtype, vmk::PromptConvArgs *a, int64_t *ext, int64_t *kept) {
  if (!type_ok(dtype)) return VM_ERR_DTYPE;
  if ((silu & ~(1 | VM_CLEAR_REST)) != 0) return VM_ERR_FLAG;
  if (x == nullptr || w == nullptr) return VM_ERR_NULL;
  a->xs = x_stride;
  int64_t each = 0;
  if (!token_extent(batch, seqlen, 1, dim, &a->xs, ext)) return VM_ERR_SHAPE;
  if (width < 2 || width > vmk::kMaxTaps) return VM_ERR_UNSUPPORTED;
  if (!dims_ok({width - 1, dim}, &each)) return VM_ERR_SHAPE;
  const int st = check_sequences(q, batch, seqlen, dim, pool, each, silu & VM_CLEAR_REST, &a->q, kept);
  if (st != VM_OK) return st;
  if (dim > kMaxDim) return VM_ERR_UNSUPPORTED;
  a->x = x;
  a->w = w;
  a->dim = static_cast<int>(dim);
  a->width = static_cast<int>(width);
  a->silu = silu & 1;
  return VM_OK;
}
// (a lane to each channel and chunk, where rows are not whole pieces, in whole waves)
bool conv_fits(const vmk::SeqArgs &q, int64_t dim) {
  return q.slots <= ((kMaxBlocks - q.clear) * 256) / (((dim + 63) / 64 + 3) * 64);
}

int64_t conv_partial(const vmk::PromptConvArgs &a) {
  return Parts::whole(static_cast<int64_t>(a.workers) * (a.width + 1) * a.dim * 4);
}

// ------------------------------------------------------------------- scan
struct ScanExtents {
  int64_t u, delta, B, C, z, out, kept;
};

int check_rows(const vm_scan_rows *p, int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate, int dtype, int options,
               int allowed, int64_t most_stride, vmk::PromptScanArgs *a, ScanExtents *e) {
  if (!type_ok(dtype)) return VM_ERR_DTYPE;
  if ((options & ~allowed) != 0) return VM_ERR_FLAG;
  if (p == nullptr || p->u == nullptr || p->delta == nullptr || p->A == nullptr || p->B == nullptr || p->C == nullptr)
    return VM_ERR_NULL;
  a->us = p->u_stride;
  a->ds = p->delta_stride;
  a->bs = p->B_stride;
  a->cs = p->C_stride;
  a->zs = p->z != nullptr ? p->z_stride : 0;
  int64_t unused = 0;
  if (!token_extent(batch, seqlen, 1, dim, &a->us, &e->u) || !token_extent(batch, seqlen, 1, dim, &a->ds, &e->delta) ||
      !token_extent(batch, seqlen, 1, dstate, &a->bs, &e->B) || !token_extent(batch, seqlen, 1, dstate, &a->cs, &e->C) ||
      !token_extent(batch, seqlen, 1, dim, &a->zs, &e->z) || !dims_ok({batch, seqlen, dim}, &e->out) ||
      !dims_ok({dim, dstate}, &unused))
    return VM_ERR_SHAPE;
  if (dstate > kMaxState || dim > kMaxDim) return VM_ERR_UNSUPPORTED;
  for (int64_t s : {a->us, a->ds, a->bs, a->cs, a->zs})
    if (s > most_stride) return VM_ERR_UNSUPPORTED;
  a->u = p->u;
  a->delta = p->delta;
  a->A = p->A;
  a->B = p->B;
  a->C = p->C;
  a->D = p->D;
  a->bias = p->delta_bias;
  a->z = p->z;
  a->dim = static_cast<int>(dim);
  a->n = static_cast<int>(dstate);
  a->softplus = (options & VM_DELTA_SOFTPLUS) != 0;
  return VM_OK;
}

bool scan_fits(const vmk::PromptScanArgs &a) { return a.q.slots <= (kMaxBlocks - a.q.clear) / vmk::scan_wide(a.dim); }

// Temporary memory of the forward and of the backward pass.
void scan_parts(vmk::PromptScanArgs &a, bool back, Parts &parts) {
  const int64_t blocks = a.q.slots * vmk::scan_blocks(a.dim), tokens = all_tokens(a.q);
  if (a.q.chunk < a.q.L) {
    parts.add(&a.ends, blocks * 256 * 4);
    parts.add(&a.steps, blocks * 16 * 4);
    if (back) parts.add(&a.starts, blocks * 256 * 4);
  }
  if (back) {
    const int64_t wide = vmk::scan_wide(a.dim);
    const int64_t tiles = (tokens / vmk::kBackTile + a.q.slots + 1) * vmk::scan_blocks(a.dim);
    parts.add(&a.marks, tiles * 256 * 4);
    if (a.q.chunk < a.q.L) parts.add(&a.before, tiles * 16 * 4);
    parts.add(&a.partA, a.q.slots * a.dim * a.n * 4);
    parts.add(&a.partD, a.q.slots * 2 * a.dim * 4);
    parts.add(&a.partBC, wide * tokens * 2 * a.n * 4);
  }
}

// ------------------------------------------------------------------ norms
int check_norm(const vm_block_norm *p, bool after, int64_t rows, int64_t dim, int dtype, int rdtype, vmk::BlockNormArgs *a,
               int64_t *x_ext, int64_t *z_ext) {
  if (!type_ok(dtype) || !type_ok(rdtype)) return VM_ERR_DTYPE;
  if (dtype == VM_F32 && rdtype == VM_BF16) return VM_ERR_DTYPE;
  if (p == nullptr) return VM_ERR_NULL;
  const int allowed = after ? VM_NORM_GATE_FIRST : VM_NORM_CENTER;
  if ((p->options & ~allowed) != 0) return VM_ERR_FLAG;
  a->xs = p->x_stride;
  a->zs = p->z_stride;
  const int64_t group = p->group != 0 ? p->group : dim, gains = p->w_dim != 0 ? p->w_dim : dim;
  if (!token_extent(1, rows, 1, dim, &a->xs, x_ext) || !token_extent(1, rows, 1, dim, &a->zs, z_ext)) return VM_ERR_SHAPE;
  if (group < 1 || dim % group != 0 || (gains != dim && gains != group)) return VM_ERR_SHAPE;
  if (!after && (group != dim || p->z != nullptr)) return VM_ERR_FLAG;
  if (after && p->b != nullptr) return VM_ERR_FLAG;
  if (after && (p->options & VM_NORM_GATE_FIRST) != 0 && p->z == nullptr) return VM_ERR_NULL;
  if (!(p->eps >= 0.0f) || !std::isfinite(p->eps) || !std::isfinite(p->factor) || group > kMaxNorm || dim > kMaxDim)
    return VM_ERR_UNSUPPORTED;
  a->x = p->x;
  a->z = p->z;
  a->w = p->w;
  a->b = p->b;
  a->scale = p->scale;
  a->rows = rows;
  a->dim = static_cast<int>(dim);
  a->group = static_cast<int>(group);
  a->wide = gains == dim;
  a->eps = p->eps;
  a->factor = p->factor;
  a->center = (p->options & VM_NORM_CENTER) != 0;
  a->gate_first = (p->options & VM_NORM_GATE_FIRST) != 0;
  return VM_OK;
}
// (a group has at most 1024 lanes, which hold 16 values each)
bool norm_fits(int64_t rows, int64_t dim, int64_t group) {
  const int64_t lanes = group <= 32 ? 4 : group <= 128 ? 16 : group <= 1024 ? 64 : group <= 4096 ? 256 : group <= 8192 ? 512 : 1024;
  return rows <= (((int64_t{1} << 32) - 1024) / lanes) / (dim / group) && rows < (int64_t{1} << 31);
}

int64_t norm_partial(const vmk::BlockNormArgs &a, int sums) {
  return Parts::whole(static_cast<int64_t>(sums) * a.workers * a.dim * 4);
}

}  // namespace

extern "C" {

int vm_prompt_conv(const vm_sequences *q, const void *x, int64_t x_stride, const float *w, const float *bias, const void *h0,
                   void *state, void *out, int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int silu, int dtype,
                   void *stream) {
  vmk::PromptConvArgs a = {};
  int64_t ext = 0, kept = 0;
  const int st = check_conv(q, true, x, x_stride, w, batch, seqlen, dim, width, silu, dtype, &a, &ext, &kept);
  if (st != VM_OK) return st;
  if (out == nullptr) return VM_ERR_NULL;
  const bool bf16 = dtype == VM_BF16;
  const int es = size_of(dtype);
  divide(a.q, vmk::kConvChunk);
  if (!conv_fits(a.q, dim)) return VM_ERR_UNSUPPORTED;
  const SeqSpans sq(a.q);
  const Span ins[] = {span(x, ext * es), span(w, dim * width * 4), span(bias, dim * 4),
                      state == h0 ? Span{} : span(h0, kept * es), sq.off, sq.where, sq.fresh};
  const Span outs[] = {span(out, batch * seqlen * dim * es), span(state, kept * es)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.bias = bias;
  a.h0 = h0;
  a.state = state;
  a.out = out;
  return hip_status(vmk::launch_prompt_conv(a, bf16, static_cast<hipStream_t>(stream)));
}

int64_t vm_prompt_conv_workspace(int64_t batch, int64_t seqlen, int64_t n, int64_t dim, int64_t width, int dtype, int packed) {
  int64_t unused = 0;
  if (!type_ok(dtype)) return -VM_ERR_DTYPE;
  if (!dims_ok({batch, seqlen, dim}, &unused) || !dims_ok({n}, &unused) || (packed != 0 ? batch != 1 : n != batch))
    return -VM_ERR_SHAPE;
  if (width < 2 || width > vmk::kMaxTaps || dim > kMaxDim) return -VM_ERR_UNSUPPORTED;
  static const int32_t some = 0;
  vmk::PromptConvArgs a = {};
  a.q.off = packed != 0 ? &some : nullptr;
  a.q.nseq = static_cast<int>(n);
  a.q.L = seqlen;
  a.dim = static_cast<int>(dim);
  a.width = static_cast<int>(width);
  a.xs = dim;
  const bool bf16 = dtype == VM_BF16;
  divide(a.q, vmk::kConvBackChunk);
  if (!conv_fits(a.q, dim)) return -VM_ERR_UNSUPPORTED;
  a.workers = vmk::conv_workers(a, bf16);      // (rows of whole pieces have the most)
  return conv_partial(a);
}

int vm_prompt_conv_bwd(const vm_sequences *q, const void *x, int64_t x_stride, const float *w, const float *bias, const void *h0,
                       const void *dout, const void *dstate, const vm_conv_grad *g, int64_t batch, int64_t seqlen, int64_t dim,
                       int64_t width, int silu, int dtype, void *workspace, int64_t workspace_bytes, void *stream) {
  vmk::PromptConvArgs a = {};
  int64_t ext = 0, kept = 0;
  int st = check_conv(q, false, x, x_stride, w, batch, seqlen, dim, width, silu, dtype, &a, &ext, &kept);
  if (st != VM_OK) return st;
  if (dout == nullptr || g == nullptr || g->dx == nullptr || g->dw == nullptr) return VM_ERR_NULL;
  const bool bf16 = dtype == VM_BF16;
  const int es = size_of(dtype);
  divide(a.q, vmk::kConvBackChunk);
  if (!conv_fits(a.q, dim)) return VM_ERR_UNSUPPORTED;
  const SeqSpans sq(a.q);
  const int64_t out = batch * seqlen * dim * es;
  const Span ins[] = {span(x, ext * es), span(w, dim * width * 4), span(bias, dim * 4), span(h0, kept * es),
                      span(dout, out), span(dstate, kept * es), sq.off};
  const Span outs[] = {span(g->dx, out), span(g->dw, dim * width * 4), span(g->dbias, dim * 4), span(g->dh0, kept * es)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.bias = bias;
  a.h0 = h0;
  a.dout = dout;
  a.dstate = dstate;
  a.dx = g->dx;
  a.dh0 = g->dh0;
  a.workers = vmk::conv_workers(a, bf16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  Parts parts;
  parts.add(&a.partial, conv_partial(a));
  st = parts.get(workspace, workspace_bytes, ws);
  if (st != VM_OK) return st;
  st = hip_status(vmk::launch_prompt_conv_back(a, bf16, s));
  if (st != VM_OK) return st;
  vmk::ColumnSums sums = {};
  const int64_t pitch = (a.width + int64_t{1}) * a.dim;
  vmk::add_sum(sums, a.partial, g->dw, a.workers, pitch, a.dim * a.width, a.dim * a.width);
  vmk::add_sum(sums, a.partial + static_cast<int64_t>(a.width) * a.dim, g->dbias, a.workers, pitch, a.dim, a.dim);
  return hip_status(vmk::launch_column_sums(sums, s));
}

int vm_token_conv(const void *x, int64_t x_stride, const float *w, const float *bias, void *state, const int32_t *slots,
                  void *out, int64_t batch, int64_t n_slots, int64_t dim, int64_t width, int silu, int dtype, void *stream) {
  if (!type_ok(dtype)) return VM_ERR_DTYPE;
  if (silu != 0 && silu != 1) return VM_ERR_FLAG;
  if (x == nullptr || w == nullptr || state == nullptr || out == nullptr) return VM_ERR_NULL;
  vmk::TokenConvArgs a = {};
  a.xs = x_stride;
  int64_t ext = 0, kept = 0, all = 0;
  if (!token_extent(batch, 1, 1, dim, &a.xs, &ext) || !dims_ok({batch, dim}, &all)) return VM_ERR_SHAPE;
  if (width < 2 || width > vmk::kMaxTaps) return VM_ERR_UNSUPPORTED;
  if (!dims_ok({n_slots, width - 1, dim}, &kept) || (slots == nullptr && batch > n_slots)) return VM_ERR_SHAPE;
  if (dim > kMaxDim || batch > (kMaxBlocks * 256) / dim) return VM_ERR_UNSUPPORTED;
  const int es = size_of(dtype);
  const Span ins[] = {span(x, ext * es), span(w, dim * width * 4), span(bias, dim * 4), span(slots, batch * 4)};
  const Span outs[] = {span(out, all * es), span(state, kept * es)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.state = state;
  a.where = slots;
  a.out = out;
  a.kept = n_slots;
  a.batch = static_cast<int>(batch);
  a.dim = static_cast<int>(dim);
  a.width = static_cast<int>(width);
  a.silu = silu;
  return hip_status(vmk::launch_token_conv(a, dtype == VM_BF16, static_cast<hipStream_t>(stream)));
}

int vm_prompt_scan(const vm_scan_rows *p, const vm_sequences *q, const float *h0, float *state, void *out, int64_t batch,
                   int64_t seqlen, int64_t dim, int64_t dstate, int dtype, int options, void *workspace,
                   int64_t workspace_bytes, void *stream) {
  vmk::PromptScanArgs a = {};
  ScanExtents e = {};
  int st = check_rows(p, batch, seqlen, dim, dstate, dtype, options, VM_DELTA_SOFTPLUS | VM_CLEAR_REST, kMaxStride, &a, &e);
  if (st == VM_OK)
    st = check_sequences(q, batch, seqlen, dim, true, dim * dstate, options & VM_CLEAR_REST, &a.q, &e.kept);
  if (st != VM_OK) return st;
  if (out == nullptr) return VM_ERR_NULL;
  const int es = size_of(dtype);
  divide(a.q, vmk::scan_chunk(all_tokens(a.q), a.q.nseq, seqlen, a.dim, a.q.off != nullptr));
  if (!scan_fits(a)) return VM_ERR_UNSUPPORTED;
  const SeqSpans sq(a.q);
  const Span ins[] = {span(p->u, e.u * es), span(p->delta, e.delta * es), span(p->B, e.B * es), span(p->C, e.C * es),
                      span(p->z, e.z * es), span(p->A, dim * dstate * 4), span(p->D, dim * 4), span(p->delta_bias, dim * 4),
                      state == h0 ? Span{} : span(h0, e.kept * 4), sq.off, sq.where, sq.fresh};
  const Span outs[] = {span(out, e.out * es), span(state, e.kept * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.h0 = h0;
  a.state = state;
  a.out = out;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  Parts parts;
  scan_parts(a, false, parts);
  if (parts.total() > 0) {
    st = parts.get(workspace, workspace_bytes, ws);
    if (st != VM_OK) return st;
  }
  return hip_status(vmk::launch_prompt_scan(a, dtype == VM_BF16, s));
}

int64_t vm_prompt_scan_workspace(int64_t batch, int64_t seqlen, int64_t n, int64_t dim, int64_t dstate, int packed,
                                 int backward) {
  int64_t unused = 0;
  if (!dims_ok({batch, seqlen, dim}, &unused) || !dims_ok({n, dim, dstate}, &unused) ||
      (packed != 0 ? batch != 1 : n != batch))
    return -VM_ERR_SHAPE;
  if (dstate > kMaxState || dim > kMaxDim) return -VM_ERR_UNSUPPORTED;
  static const int32_t some = 0;
  vmk::PromptScanArgs a = {};
  a.q.off = packed != 0 ? &some : nullptr;
  a.q.nseq = static_cast<int>(n);
  a.q.L = seqlen;
  a.dim = static_cast<int>(dim);
  a.n = static_cast<int>(dstate);
  divide(a.q, backward != 0 ? vmk::scan_back_chunk(all_tokens(a.q), n, seqlen, a.dim, packed != 0)
                            : vmk::scan_chunk(all_tokens(a.q), n, seqlen, a.dim, packed != 0));
  if (!scan_fits(a)) return -VM_ERR_UNSUPPORTED;
  Parts parts;
  scan_parts(a, backward != 0, parts);
  return parts.total();
}

int vm_prompt_scan_bwd(const vm_scan_rows *p, const vm_sequences *q, const float *h0, const void *dout, const float *dstate,
                       const vm_rows_grad *g, int64_t batch, int64_t seqlen, int64_t dim, int64_t N, int dtype, int options,
                       void *workspace, int64_t workspace_bytes, void *stream) {
  vmk::PromptScanArgs a = {};
  ScanExtents e = {};
  int st = check_rows(p, batch, seqlen, dim, N, dtype, options, VM_DELTA_SOFTPLUS | VM_CLEAR_REST, kMaxStride, &a, &e);
  if (st == VM_OK) st = check_sequences(q, batch, seqlen, dim, false, dim * N, options & VM_CLEAR_REST, &a.q, &e.kept);
  if (st != VM_OK) return st;
  if (dout == nullptr || g == nullptr || g->du == nullptr || g->ddelta == nullptr || g->dA == nullptr || g->dB == nullptr ||
      g->dC == nullptr || (g->dz == nullptr) != (p->z == nullptr))
    return VM_ERR_NULL;
  const int es = size_of(dtype);
  divide(a.q, vmk::scan_back_chunk(all_tokens(a.q), a.q.nseq, seqlen, a.dim, a.q.off != nullptr));
  if (!scan_fits(a)) return VM_ERR_UNSUPPORTED;
  const SeqSpans sq(a.q);
  const int64_t bc = batch * seqlen * N * es;
  const Span ins[] = {span(p->u, e.u * es), span(p->delta, e.delta * es), span(p->B, e.B * es), span(p->C, e.C * es),
                      span(p->z, e.z * es), span(p->A, dim * N * 4), span(p->D, dim * 4), span(p->delta_bias, dim * 4),
                      span(h0, e.kept * 4), sq.off, span(dout, e.out * es), span(dstate, e.kept * 4)};
  const Span outs[] = {span(g->du, e.out * es), span(g->ddelta, e.out * es), span(g->dz, e.out * es), span(g->dB, bc),
                       span(g->dC, bc), span(g->dA, dim * N * 4), span(g->dD, dim * 4), span(g->ddelta_bias, dim * 4),
                       span(g->dh0, e.kept * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.h0 = h0;
  a.dout = dout;
  a.dstate = dstate;
  a.du = g->du;
  a.ddelta = g->ddelta;
  a.dB = g->dB;
  a.dC = g->dC;
  a.dz = g->dz;
  a.dh0 = g->dh0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  Parts parts;
  scan_parts(a, true, parts);
  st = parts.get(workspace, workspace_bytes, ws);
  if (st != VM_OK) return st;
  st = hip_status(vmk::launch_prompt_scan_back(a, dtype == VM_BF16, s));
  if (st != VM_OK) return st;
  vmk::ColumnSums sums = {};
  vmk::add_sum(sums, a.partA, g->dA, a.q.slots, static_cast<int64_t>(a.dim) * a.n, a.dim * a.n, a.dim * a.n);
  vmk::add_sum(sums, a.partD, g->dD, a.q.slots, int64_t{2} * a.dim, a.dim, a.dim);
  vmk::add_sum(sums, a.partD + a.dim, g->ddelta_bias, a.q.slots, int64_t{2} * a.dim, a.dim, a.dim);
  return hip_status(vmk::launch_column_sums(sums, s));
}

int vm_token_scan(const vm_scan_rows *p, float *state, const int32_t *slots, void *out, int64_t batch, int64_t n_slots,
                  int64_t dim, int64_t dstate, int dtype, int options, void *stream) {
  vmk::PromptScanArgs r = {};
  ScanExtents e = {};
  const int st = check_rows(p, batch, 1, dim, dstate, dtype, options, VM_DELTA_SOFTPLUS, vmk::kMaxElems, &r, &e);
  if (st != VM_OK) return st;
  if (state == nullptr || out == nullptr) return VM_ERR_NULL;
  if (!dims_ok({n_slots, dim, dstate}, &e.kept) || (slots == nullptr && batch > n_slots)) return VM_ERR_SHAPE;
  if (batch > kMaxBlocks / ((dim + 63) / 64)) return VM_ERR_UNSUPPORTED;
  const int es = size_of(dtype);
  const Span ins[] = {span(p->u, e.u * es), span(p->delta, e.delta * es), span(p->B, e.B * es), span(p->C, e.C * es),
                      span(p->z, e.z * es), span(p->A, dim * dstate * 4), span(p->D, dim * 4), span(p->delta_bias, dim * 4),
                      span(slots, batch * 4)};
  const Span outs[] = {span(out, e.out * es), span(state, e.kept * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  vmk::TokenScanArgs a = {};
  a.u = r.u;
  a.delta = r.delta;
  a.B = r.B;
  a.C = r.C;
  a.z = r.z;
  a.A = r.A;
  a.D = r.D;
  a.bias = r.bias;
  a.state = state;
  a.where = slots;
  a.out = out;
  a.us = r.us;
  a.ds = r.ds;
  a.bs = r.bs;
  a.cs = r.cs;
  a.zs = r.zs;
  a.kept = n_slots;
  a.batch = static_cast<int>(batch);
  a.dim = r.dim;
  a.n = r.n;
  a.softplus = r.softplus;
  return hip_status(vmk::launch_token_scan(a, dtype == VM_BF16, static_cast<hipStream_t>(stream)));
}

int vm_norm_before(const vm_block_norm *p, const void *residual, void *y, void *r, int64_t rows, int64_t dim, int dtype,
                   int rdtype, void *stream) {
  vmk::BlockNormArgs a = {};
  int64_t xe = 0, ze = 0;
  const int st = check_norm(p, false, rows, dim, dtype, rdtype, &a, &xe, &ze);
  if (st != VM_OK) return st;
  if (p->x == nullptr || y == nullptr) return VM_ERR_NULL;
  if (!norm_fits(rows, dim, a.group)) return VM_ERR_UNSUPPORTED;
  const int es = size_of(dtype), rs = size_of(rdtype);
  const int64_t all = rows * dim;
  const Span ins[] = {span(p->x, xe * es), span(p->w, dim * 4), span(p->b, dim * 4), span(p->scale, dim * 4),
                      r == residual ? Span{} : span(residual, all * rs)};
  const Span outs[] = {span(y, all * es), span(r, all * rs)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.residual = residual;
  a.y = y;
  a.r = r;
  a.workers = static_cast<int>(rows);
  return hip_status(vmk::launch_norm_before(a, dtype == VM_BF16, rdtype == VM_F32, false, static_cast<hipStream_t>(stream)));
}

int vm_norm_after(const vm_block_norm *p, const void *residual, void *out, int64_t rows, int64_t dim, int dtype, int rdtype,
                  void *stream) {
  vmk::BlockNormArgs a = {};
  int64_t xe = 0, ze = 0;
  const int st = check_norm(p, true, rows, dim, dtype, rdtype, &a, &xe, &ze);
  if (st != VM_OK) return st;
  if (p->x == nullptr || out == nullptr) return VM_ERR_NULL;
  if (!norm_fits(rows, dim, a.group)) return VM_ERR_UNSUPPORTED;
  const int es = size_of(dtype), rs = size_of(rdtype);
  const int64_t all = rows * dim;
  const Span ins[] = {span(p->x, xe * es), span(p->z, ze * es), span(p->w, (a.wide ? dim : a.group) * 4),
                      span(p->scale, dim * 4), out == residual ? Span{} : span(residual, all * rs)};
  const Span outs[] = {span(out, all * rs)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.residual = residual;
  a.y = out;
  a.workers = static_cast<int>(rows);
  return hip_status(vmk::launch_norm_after(a, dtype == VM_BF16, rdtype == VM_F32, false, static_cast<hipStream_t>(stream)));
}

int64_t vm_block_norm_workspace(int64_t rows, int64_t dim, int64_t group) {
  int64_t unused = 0;
  if (group == 0) group = dim;
  if (!dims_ok({rows, dim}, &unused) || group < 1 || dim % group != 0) return -VM_ERR_SHAPE;
  if (group > kMaxNorm || dim > kMaxDim || !norm_fits(rows, dim, group)) return -VM_ERR_UNSUPPORTED;
  vmk::BlockNormArgs a = {};
  a.rows = rows;
  a.dim = static_cast<int>(dim);
  a.group = static_cast<int>(group);
  a.workers = vmk::norm_workers(a);
  return norm_partial(a, 3);
}

int vm_norm_before_bwd(const vm_block_norm *p, const void *r, const void *dy, const void *dr, const vm_norm_grad *g,
                       int64_t rows, int64_t dim, int dtype, int rdtype, void *workspace, int64_t workspace_bytes,
                       void *stream) {
  vmk::BlockNormArgs a = {};
  int64_t xe = 0, ze = 0;
  int st = check_norm(p, false, rows, dim, dtype, rdtype, &a, &xe, &ze);
  if (st != VM_OK) return st;
  if (r == nullptr || dy == nullptr || g == nullptr || (g->dx == nullptr && g->dresidual == nullptr) || g->dz != nullptr ||
      (g->dw != nullptr && p->w == nullptr) || (g->db != nullptr && p->b == nullptr) ||
      (g->dscale != nullptr && (p->scale == nullptr || p->x == nullptr)))
    return VM_ERR_NULL;
  if (!norm_fits(rows, dim, a.group)) return VM_ERR_UNSUPPORTED;
  const int es = size_of(dtype), rs = size_of(rdtype);
  const int64_t all = rows * dim;
  const Span ins[] = {span(p->x, xe * es), span(p->w, dim * 4), span(p->b, dim * 4), span(p->scale, dim * 4), span(r, all * rs),
                      span(dy, all * es), span(dr, all * rs)};
  const Span outs[] = {span(g->dx, all * es), span(g->dresidual, all * rs), span(g->dw, dim * 4), span(g->db, dim * 4),
                       span(g->dscale, dim * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.r = const_cast<void *>(r);
  a.dy = dy;
  a.dr = dr;
  a.dx = g->dx;
  a.dres = g->dresidual;
  a.want_w = g->dw != nullptr;
  a.want_b = g->db != nullptr;
  a.want_scale = g->dscale != nullptr;
  a.workers = vmk::norm_workers(a);
  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  const int sums = a.want_w + a.want_b + a.want_scale;
  if (sums > 0) {
    Parts parts;
    parts.add(&a.partial, norm_partial(a, sums));
    st = parts.get(workspace, workspace_bytes, ws);
    if (st != VM_OK) return st;
  }
  st = hip_status(vmk::launch_norm_before(a, dtype == VM_BF16, rdtype == VM_F32, true, s));
  if (st != VM_OK) return st;
  vmk::ColumnSums cs = {};
  const float *part = a.partial;
  const int64_t step = static_cast<int64_t>(a.workers) * a.dim;
  for (float *to : {g->dw, g->db, g->dscale})
    if (to != nullptr) {
      vmk::add_sum(cs, part, to, a.workers, a.dim, a.dim, a.dim);
      part += step;
    }
  return hip_status(vmk::launch_column_sums(cs, s));
}

int vm_norm_after_bwd(const vm_block_norm *p, const void *dout, const vm_norm_grad *g, int64_t rows, int64_t dim, int dtype,
                      int rdtype, void *workspace, int64_t workspace_bytes, void *stream) {
  vmk::BlockNormArgs a = {};
  int64_t xe = 0, ze = 0;
  int st = check_norm(p, true, rows, dim, dtype, rdtype, &a, &xe, &ze);
  if (st != VM_OK) return st;
  if (p->x == nullptr || dout == nullptr || g == nullptr || g->dx == nullptr || (g->dz == nullptr) != (p->z == nullptr) ||
      g->db != nullptr || g->dresidual != nullptr || (g->dw != nullptr && p->w == nullptr) ||
      (g->dscale != nullptr && p->scale == nullptr))
    return VM_ERR_NULL;
  if (!norm_fits(rows, dim, a.group)) return VM_ERR_UNSUPPORTED;
  const int es = size_of(dtype), rs = size_of(rdtype);
  const int64_t all = rows * dim, gains = a.wide ? dim : a.group;
  const Span ins[] = {span(p->x, xe * es), span(p->z, ze * es), span(p->w, gains * 4), span(p->scale, dim * 4),
                      span(dout, all * rs)};
  const Span outs[] = {span(g->dx, all * es), span(g->dz, all * es), span(g->dw, gains * 4), span(g->dscale, dim * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.dy = dout;
  a.dx = g->dx;
  a.dz = g->dz;
  a.want_w = g->dw != nullptr;
  a.want_scale = g->dscale != nullptr;
  a.workers = vmk::norm_workers(a);
  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  const int sums = a.want_w + a.want_scale;
  if (sums > 0) {
    Parts parts;
    parts.add(&a.partial, norm_partial(a, sums));
    st = parts.get(workspace, workspace_bytes, ws);
    if (st != VM_OK) return st;
  }
  st = hip_status(vmk::launch_norm_after(a, dtype == VM_BF16, rdtype == VM_F32, true, s));
  if (st != VM_OK) return st;
  vmk::ColumnSums cs = {};
  const float *part = a.partial;
  if (g->dw != nullptr) {
    vmk::add_sum(cs, part, g->dw, a.workers, a.dim, a.dim, static_cast<int>(gains));
    part += static_cast<int64_t>(a.workers) * a.dim;
  }
  vmk::add_sum(cs, part, g->dscale, a.workers, a.dim, a.dim, a.dim);
  return hip_status(vmk::launch_column_sums(cs, s));
}

}  // extern "C"
