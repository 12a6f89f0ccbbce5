// C ABI of the matrix-state mixers (declared in include/vm_scan.h): argument
// checks, temporary memory and dispatch of the gated delta rule, the per-head
// norm with rotation and gradient clipping.  Every check runs before any HIP
// call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_util.h"
#include "mixer_internal.h"
#include "vm_scan.h"

namespace {

using vmk::Scratch;
using vmk::Span;
using vmk::dims_ok;
using vmk::hip_status;
using vmk::overlaps;
using vmk::span;

// Grids put chunk slots and sequences on x with up to 512 work-items each
// (work-items below 2^32) and heads on y.
constexpr int64_t kMaxSlots = (int64_t{1} << 23) - 1;
// Scans put sequences, heads (whole rounds of 8) and blocks of columns on x, and
// the backward pass two scans: how many work-items that makes goes by the variant,
// see sizes_fit().
constexpr int64_t kMaxScans = (int64_t{1} << 21) - 8;
constexpr int64_t kMaxItems = (int64_t{1} << 32) - 1;
constexpr int64_t kMaxHeads = 65535;
constexpr int64_t kMaxDeltaDim = 128, kMaxNormDim = 512, kMaxGrads = 65536;

// Extent in elements of [batch, seqlen, heads, dim] with a token stride
// (0 = dense); false if the stride is short or the extent overflows.
bool token_extent(int64_t batch, int64_t seqlen, int64_t heads, int64_t dim, int64_t *stride, int64_t *extent) {
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

struct DeltaSizes {
  int64_t qs, ks, vs;             // token strides
  int64_t q_ext, k_ext, v_ext;    // elements
  int64_t gates, out, states;     // elements of g, of out and of the states
};

int check_delta(const vm_delta *p, float scale, int64_t batch, int64_t seqlen, int64_t n, int64_t hk, int64_t hv,
                int64_t dk, int64_t dv, int dtype, int reverse, DeltaSizes *z) {
  if (dtype != VM_F32 && dtype != VM_BF16) return VM_ERR_DTYPE;
  if (reverse != 0 && reverse != 1) return VM_ERR_FLAG;
  if (p == nullptr || p->q == nullptr || p->k == nullptr || p->v == nullptr || p->g == nullptr ||
      p->beta == nullptr)
    return VM_ERR_NULL;
  z->qs = p->q_stride;
  z->ks = p->k_stride;
  z->vs = p->v_stride;
  if (hk <= 0 || hv <= 0 || hv % hk != 0) return VM_ERR_SHAPE;
  if (!token_extent(batch, seqlen, hk, dk, &z->qs, &z->q_ext) ||
      !token_extent(batch, seqlen, hk, dk, &z->ks, &z->k_ext) ||
      !token_extent(batch, seqlen, hv, dv, &z->vs, &z->v_ext) ||
      !dims_ok({batch, seqlen, hv}, &z->gates) || !dims_ok({batch, seqlen, hv, dv}, &z->out) ||
      !dims_ok({n, hv, dk, dv}, &z->states))
    return VM_ERR_SHAPE;
  if (p->offsets != nullptr ? batch != 1 : n != batch) return VM_ERR_SHAPE;
  if (!std::isfinite(scale) || dk > kMaxDeltaDim || dv > kMaxDeltaDim) return VM_ERR_UNSUPPORTED;
  // (the kernels reach the 64 tokens of a chunk with 31-bit byte offsets)
  for (int64_t stride : {z->qs, z->ks, z->vs, hv * dv})
    if (stride * 64 * 4 >= (int64_t{1} << 31)) return VM_ERR_UNSUPPORTED;
  return VM_OK;
}

// Whether every launch of a call holds its grid.
bool sizes_fit(const vmk::DeltaArgs &a, int64_t n, bool bf16, bool backward) {
  return a.hv <= kMaxHeads && n * a.hv <= kMaxScans && a.slots <= kMaxSlots &&
         vmk::delta_scan_items(a, bf16, backward) <= kMaxItems;
}

vmk::DeltaArgs delta_args(const vm_delta *p, const DeltaSizes &z, float scale, int64_t batch, int64_t seqlen,
                          int64_t n, int64_t hk, int64_t hv, int64_t dk, int64_t dv, int reverse) {
  vmk::DeltaArgs a = {};
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.g = p->g;
  a.beta = p->beta;
  a.h0 = p->h0;
  a.off = p->offsets;
  a.qs = z.qs;
  a.ks = z.ks;
  a.vs = z.vs;
  a.L = seqlen;
  a.slots = vmk::delta_slots(batch, seqlen, n, p->offsets != nullptr);
  a.nseq = static_cast<int>(n);
  a.hk = static_cast<int>(hk);
  a.hv = static_cast<int>(hv);
  a.dk = static_cast<int>(dk);
  a.dv = static_cast<int>(dv);
  a.reverse = reverse;
  a.scale = scale;
  return a;
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

// The chunks' triangular inverses, masked products and decays, and for the
// backward pass what its kernels hand on.
void delta_parts(vmk::DeltaArgs &a, bool bf16, bool backward, Parts &parts) {
  const int64_t per = a.slots * a.hv, c = vmk::kDeltaChunk, tri = per * vmk::kTriTerm * 2;
  const int units = vmk::tri_units(bf16);
  parts.add(&a.T, tri * units * (backward ? 1 : 2));
  parts.add(&a.eg, per * c * 4);
  parts.add(&a.ew, per * c * 4);
  if (backward) {
    parts.add(&a.TT, tri * units * 2);
    parts.add(&a.gam, per * c * 8);
    a.dvp = (a.dv + 15) / 16 * 16;
    parts.add(&a.S, per * a.dk * a.dvp * 4);
    parts.add(&a.dS, per * a.dk * a.dvp * 4);
    parts.add(&a.V, per * c * a.dvp * 4);
    parts.add(&a.dR, per * c * a.dvp * 4);
  }
}

int check_norm(const vm_head_norm *p, int64_t batch, int64_t seqlen, int64_t hq, int64_t hk, int64_t dim, float eps,
               int norm_options, int dtype, vmk::NormArgs *a, int64_t ext[2], int64_t elems[2]) {
  if (dtype != VM_F32 && dtype != VM_BF16) return VM_ERR_DTYPE;
  if ((norm_options & ~(VM_NORM_L2 | VM_ROPE_INTERLEAVED)) != 0) return VM_ERR_FLAG;
  if (p == nullptr || p->q == nullptr || (p->k == nullptr) != (hk == 0)) return VM_ERR_NULL;
  a->xs[0] = p->q_stride;
  a->xs[1] = p->k_stride;
  int64_t tokens = 0;
  if (!dims_ok({batch, seqlen}, &tokens) || hq <= 0 || hk < 0) return VM_ERR_SHAPE;
  if (!token_extent(batch, seqlen, hq, dim, &a->xs[0], &ext[0]) ||
      (hk > 0 && !token_extent(batch, seqlen, hk, dim, &a->xs[1], &ext[1])))
    return VM_ERR_SHAPE;
  if (p->rot < 0 || p->rot > dim || p->rot % 2 != 0) return VM_ERR_SHAPE;
  if (p->rot > 0) {
    int64_t unused = 0;
    if (p->cos == nullptr || p->sin == nullptr) return VM_ERR_NULL;
    if (!dims_ok({p->table, p->rot}, &unused)) return VM_ERR_SHAPE;
  }
  if (dim > kMaxNormDim || hq > kMaxHeads || hk > kMaxHeads || !(eps >= 0.0f) || !std::isfinite(eps)) return VM_ERR_UNSUPPORTED;
  elems[0] = tokens * hq * dim;
  elems[1] = tokens * hk * dim;
  a->x[0] = p->q;
  a->x[1] = p->k;
  a->w[0] = p->wq;
  a->w[1] = p->wk;
  a->cos = p->cos;
  a->sin = p->sin;
  a->pos = p->positions;
  a->tokens = tokens;
  a->seqlen = seqlen;
  a->table = p->table;
  a->heads[0] = static_cast<int>(hq);
  a->heads[1] = static_cast<int>(hk);
  a->dim = static_cast<int>(dim);
  a->rot = static_cast<int>(p->rot);
  a->eps = eps;
  a->over = (norm_options & VM_NORM_L2) != 0 ? 1.0f : 1.0f / static_cast<float>(dim);
  a->interleaved = (norm_options & VM_ROPE_INTERLEAVED) != 0;
  return VM_OK;
}

}  // namespace

extern "C" {

int64_t vm_gated_delta_workspace(int64_t batch, int64_t seqlen, int64_t n, int64_t hv, int64_t dk, int64_t dv,
                                 int dtype, int packed, int backward) {
  int64_t unused = 0;
  if (!dims_ok({batch, seqlen, hv, dk}, &unused) || !dims_ok({batch, seqlen, hv, dv}, &unused) ||
      !dims_ok({n, hv, dk, dv}, &unused))
    return -VM_ERR_SHAPE;
  if (packed != 0 ? batch != 1 : n != batch) return -VM_ERR_SHAPE;
  if (dk > kMaxDeltaDim || dv > kMaxDeltaDim) return -VM_ERR_UNSUPPORTED;
  static const int32_t some = 0;
  vmk::DeltaArgs a = {};
  a.off = packed != 0 ? &some : nullptr;
  a.slots = vmk::delta_slots(batch, seqlen, n, packed != 0);
  a.nseq = static_cast<int>(n);
  a.hv = static_cast<int>(hv);
  a.dk = static_cast<int>(dk);
  a.dv = static_cast<int>(dv);
  if (!sizes_fit(a, n, dtype == VM_BF16, backward != 0)) return -VM_ERR_UNSUPPORTED;
  Parts parts;
  delta_parts(a, dtype == VM_BF16, backward != 0, parts);
  return parts.total();
}

int64_t vm_head_norm_rope_workspace(int64_t dim) {
  if (dim <= 0) return -VM_ERR_SHAPE;
  if (dim > kMaxNormDim) return -VM_ERR_UNSUPPORTED;
  return Parts::whole(vmk::kNormMaxBlocks * 2 * dim * 4);
}

int64_t vm_clip_grad_workspace(int64_t count) {
  if (count < 0) return -VM_ERR_SHAPE;
  if (count > kMaxGrads) return -VM_ERR_UNSUPPORTED;
  return Parts::whole(vmk::kClipPartials * 8);
}

int vm_gated_delta_fwd(const vm_delta *p, void *out, float *state, float scale, int64_t batch, int64_t seqlen,
                       int64_t n, int64_t hk, int64_t hv, int64_t dk, int64_t dv, int dtype, int reverse,
                       void *workspace, int64_t workspace_bytes, void *stream) {
  DeltaSizes z = {};
  int st = check_delta(p, scale, batch, seqlen, n, hk, hv, dk, dv, dtype, reverse, &z);
  if (st != VM_OK) return st;
  if (out == nullptr) return VM_ERR_NULL;
  const bool bf16 = dtype == VM_BF16;
  const int es = bf16 ? 2 : 4;
  vmk::DeltaArgs a = delta_args(p, z, scale, batch, seqlen, n, hk, hv, dk, dv, reverse);
  a.out = out;
  a.state = state;
  if (!sizes_fit(a, n, bf16, false)) return VM_ERR_UNSUPPORTED;
  const Span ins[] = {span(p->q, z.q_ext * es), span(p->k, z.k_ext * es), span(p->v, z.v_ext * es),
                      span(p->g, z.gates * 4), span(p->beta, z.gates * 4),
                      state == p->h0 ? Span{} : span(p->h0, z.states * 4),
                      p->offsets != nullptr ? span(p->offsets, (n + 1) * 4) : Span{}};
  const Span outs[] = {span(out, z.out * es), span(state, z.states * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;

  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  Parts parts;
  delta_parts(a, bf16, false, parts);
  st = parts.get(workspace, workspace_bytes, ws);
  if (st != VM_OK) return st;
  st = hip_status(vmk::launch_delta_prep(a, bf16, false, s));
  if (st != VM_OK) return st;
  return hip_status(vmk::launch_delta_scan(a, bf16, false, s));
}

int vm_gated_delta_bwd(const vm_delta *p, const void *dout, const float *dstate, const vm_delta_grad *grad, float scale,
                       int64_t batch, int64_t seqlen, int64_t n, int64_t hk, int64_t hv, int64_t dk, int64_t dv,
                       int dtype, int reverse, void *workspace, int64_t workspace_bytes, void *stream) {
  DeltaSizes z = {};
  int st = check_delta(p, scale, batch, seqlen, n, hk, hv, dk, dv, dtype, reverse, &z);
  if (st != VM_OK) return st;
  if (dout == nullptr || grad == nullptr || grad->dq == nullptr || grad->dk == nullptr || grad->dv == nullptr ||
      grad->dg == nullptr || grad->dbeta == nullptr)
    return VM_ERR_NULL;
  const bool bf16 = dtype == VM_BF16;
  const int es = bf16 ? 2 : 4;
  vmk::DeltaArgs a = delta_args(p, z, scale, batch, seqlen, n, hk, hv, dk, dv, reverse);
  a.dout = dout;
  a.dstate = dstate;
  a.dq = grad->dq;
  a.dkey = grad->dk;
  a.dval = grad->dv;
  a.dg = grad->dg;
  a.dbeta = grad->dbeta;
  a.dh0 = grad->dh0;
  if (!sizes_fit(a, n, bf16, true)) return VM_ERR_UNSUPPORTED;
  const int64_t keys = batch * seqlen * hk * dk;
  const Span ins[] = {span(p->q, z.q_ext * es), span(p->k, z.k_ext * es), span(p->v, z.v_ext * es),
                      span(p->g, z.gates * 4), span(p->beta, z.gates * 4), span(p->h0, z.states * 4),
                      p->offsets != nullptr ? span(p->offsets, (n + 1) * 4) : Span{}, span(dout, z.out * es),
                      span(dstate, z.states * 4)};
  const Span outs[] = {span(grad->dq, keys * es), span(grad->dk, keys * es), span(grad->dv, z.out * es),
                       span(grad->dg, z.gates * 4), span(grad->dbeta, z.gates * 4), span(grad->dh0, z.states * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;

  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  Parts parts;
  delta_parts(a, bf16, true, parts);
  st = parts.get(workspace, workspace_bytes, ws);
  if (st != VM_OK) return st;
  st = hip_status(vmk::launch_delta_prep(a, bf16, true, s));
  if (st == VM_OK) st = hip_status(vmk::launch_delta_scan(a, bf16, true, s));
  if (st == VM_OK) st = hip_status(vmk::launch_delta_grad(a, bf16, s));
  return st;
}

int vm_gated_delta_step(const void *q, const void *k, const void *v, const float *g, const float *beta, float *state,
                        const int32_t *slots, void *out, float scale, int64_t batch, int64_t n_slots, int64_t hk,
                        int64_t hv, int64_t dk, int64_t dv, int dtype, void *stream) {
  if (dtype != VM_F32 && dtype != VM_BF16) return VM_ERR_DTYPE;
  if (q == nullptr || k == nullptr || v == nullptr || g == nullptr || beta == nullptr || state == nullptr ||
      out == nullptr)
    return VM_ERR_NULL;
  int64_t keys = 0, values = 0, gates = 0, states = 0;
  if (hk <= 0 || hv <= 0 || hv % hk != 0 || !dims_ok({batch, hk, dk}, &keys) || !dims_ok({batch, hv, dv}, &values) ||
      !dims_ok({batch, hv}, &gates) || !dims_ok({n_slots, hv, dk, dv}, &states))
    return VM_ERR_SHAPE;
  if (slots == nullptr && batch > n_slots) return VM_ERR_SHAPE;
  if (!std::isfinite(scale) || dk > kMaxDeltaDim || dv > kMaxDeltaDim || gates * 4 >= (int64_t{1} << 26)) return VM_ERR_UNSUPPORTED;
  const int es = dtype == VM_BF16 ? 2 : 4;
  const Span ins[] = {span(q, keys * es), span(k, keys * es), span(v, values * es), span(g, gates * 4),
                      span(beta, gates * 4), span(slots, batch * 4)};
  const Span outs[] = {span(out, values * es), span(state, states * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  vmk::StepArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.state = state;
  a.slots = slots;
  a.out = out;
  a.scale = scale;
  a.n_slots = n_slots;
  a.batch = static_cast<int>(batch);
  a.hk = static_cast<int>(hk);
  a.hv = static_cast<int>(hv);
  a.dk = static_cast<int>(dk);
  a.dv = static_cast<int>(dv);
  return hip_status(vmk::launch_delta_step(a, dtype == VM_BF16, static_cast<hipStream_t>(stream)));
}

int vm_head_norm_rope(const vm_head_norm *p, void *q_out, void *k_out, int64_t batch, int64_t seqlen, int64_t hq,
                      int64_t hk, int64_t dim, float eps, int norm_options, int dtype, void *stream) {
  vmk::NormArgs a = {};
  int64_t ext[2] = {0, 0}, elems[2] = {0, 0};
  const int st = check_norm(p, batch, seqlen, hq, hk, dim, eps, norm_options, dtype, &a, ext, elems);
  if (st != VM_OK) return st;
  if (q_out == nullptr || (k_out == nullptr) != (hk == 0)) return VM_ERR_NULL;
  const int es = dtype == VM_BF16 ? 2 : 4;
  const int64_t table = p->rot > 0 ? p->table * (p->rot / 2) * 4 : 0;
  const Span ins[] = {span(p->q, ext[0] * es), span(p->k, ext[1] * es), span(p->wq, dim * 4), span(p->wk, dim * 4),
                      span(p->cos, table), span(p->sin, table), span(p->positions, p->rot > 0 ? a.tokens * 4 : 0)};
  const Span outs[] = {span(q_out, elems[0] * es), span(k_out, elems[1] * es)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.y[0] = q_out;
  a.y[1] = k_out;
  return hip_status(vmk::launch_norm(a, dtype == VM_BF16, false, static_cast<hipStream_t>(stream)));
}

int vm_head_norm_rope_bwd(const vm_head_norm *p, const void *dq_out, const void *dk_out, void *dq, void *dk, float *dwq,
                          float *dwk, int64_t batch, int64_t seqlen, int64_t hq, int64_t hk, int64_t dim, float eps,
                          int norm_options, int dtype, void *workspace, int64_t workspace_bytes, void *stream) {
  vmk::NormArgs a = {};
  int64_t ext[2] = {0, 0}, elems[2] = {0, 0};
  int st = check_norm(p, batch, seqlen, hq, hk, dim, eps, norm_options, dtype, &a, ext, elems);
  if (st != VM_OK) return st;
  if (dq_out == nullptr || dq == nullptr || (dk_out == nullptr) != (hk == 0) || (dk == nullptr) != (hk == 0))
    return VM_ERR_NULL;
  if ((dwq != nullptr && p->wq == nullptr) || (dwk != nullptr && (p->wk == nullptr || hk == 0))) return VM_ERR_NULL;
  const bool bf16 = dtype == VM_BF16;
  const int es = bf16 ? 2 : 4;
  const int64_t table = p->rot > 0 ? p->table * (p->rot / 2) * 4 : 0;
  const Span ins[] = {span(p->q, ext[0] * es), span(p->k, ext[1] * es), span(p->wq, dim * 4), span(p->wk, dim * 4),
                      span(p->cos, table), span(p->sin, table), span(p->positions, p->rot > 0 ? a.tokens * 4 : 0),
                      span(dq_out, elems[0] * es), span(dk_out, elems[1] * es)};
  const Span outs[] = {span(dq, elems[0] * es), span(dk, elems[1] * es), span(dwq, dim * 4), span(dwk, dim * 4)};
  if (any_overlap(outs, ins)) return VM_ERR_ALIAS;
  a.y[0] = dq;
  a.y[1] = dk;
  a.dy[0] = dq_out;
  a.dy[1] = dk_out;
  a.dw[0] = dwq;
  a.dw[1] = dwk;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  if (dwq != nullptr || dwk != nullptr) {
    Parts parts;
    parts.add(&a.partial, vm_head_norm_rope_workspace(dim));
    st = parts.get(workspace, workspace_bytes, ws);
    if (st != VM_OK) return st;
  }
  return hip_status(vmk::launch_norm(a, bf16, true, s));
}

int vm_clip_grad_norm(const vm_grad_tensor *list, int64_t count, float max_norm, float *norm, void *workspace,
                      int64_t workspace_bytes, void *stream) {
  if (norm == nullptr || (list == nullptr && count > 0)) return VM_ERR_NULL;
  if (count < 0) return VM_ERR_SHAPE;
  if (count > kMaxGrads || !(max_norm >= 0.0f)) return VM_ERR_UNSUPPORTED;
  const Span sn = span(norm, 4);
  bool scaled = false;
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    const vm_grad_tensor &t = list[i];
    if (t.elems < 0 || t.elems > vmk::kMaxElems) return VM_ERR_SHAPE;
    if (t.dtype != VM_F32 && t.dtype != VM_BF16) return VM_ERR_DTYPE;
    if (t.elems > 0 && t.in == nullptr) return VM_ERR_NULL;
    const int es = t.dtype == VM_BF16 ? 2 : 4;
    const Span si = span(t.in, t.elems * es), so = span(t.out, t.elems * es);
    if ((t.out != t.in && overlaps(si, so)) || overlaps(si, sn) || overlaps(so, sn)) return VM_ERR_ALIAS;
    scaled = scaled || (t.out != nullptr && t.elems > 0);
    chunks += (t.elems + vmk::kClipChunk - 1) / vmk::kClipChunk;
    if (chunks > vmk::kMaxDim) return VM_ERR_UNSUPPORTED;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  Scratch ws(s);
  int st = VM_OK;
  double *partial = nullptr;
  Parts parts;
  parts.add(&partial, vm_clip_grad_workspace(count));
  st = parts.get(workspace, workspace_bytes, ws);
  if (st != VM_OK) return st;
  int used = 0;
  for (int pass = 0; pass < (scaled ? 2 : 1); ++pass)
    for (int64_t from = 0; from < count; from += vmk::kClipTable) {
      vmk::ClipTable t;
      t.n = 0;
      uint32_t at = 0;
      for (int64_t i = from; i < count && i < from + vmk::kClipTable; ++i) {
        if (list[i].elems == 0) continue;
        t.in[t.n] = list[i].in;
        t.out[t.n] = list[i].out;
        t.elems[t.n] = list[i].elems;
        t.bf16[t.n] = list[i].dtype == VM_BF16;
        t.first[t.n] = at;
        at += static_cast<uint32_t>((list[i].elems + vmk::kClipChunk - 1) / vmk::kClipChunk);
        ++t.n;
      }
      t.first[t.n] = at;
      if (t.n == 0) continue;
      const int blocks = static_cast<int>(at < vmk::kClipPartials ? at : vmk::kClipPartials);
      if (pass == 0) {
        st = hip_status(vmk::launch_clip_sums(t, partial, used, blocks, s));
        used = blocks > used ? blocks : used;
      } else {
        st = hip_status(vmk::launch_clip_scale(t, partial, used, max_norm, norm, blocks, s));
      }
      if (st != VM_OK) return st;
    }
  if (!scaled) st = hip_status(vmk::launch_clip_norm_only(partial, used, norm, s));
  return st;
}

}  // extern "C"
