/*
 * vm_scan.h -- C ABI of the selective-scan hot path for vision Mamba
 * backbones (Vim bidirectional blocks, EfficientVMamba atrous ES2D, FastVim
 * pooled scan, four-direction SS2D) on AMD Instinct MI355X (gfx950).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensors are dense, contiguous, row-major, in the shapes given at each
 *    call, and live in device memory of the current HIP device.  The caller
 *    owns every buffer; the library never frees or keeps a pointer past the
 *    call.  Outputs must not overlap any input (checked: VM_ERR_ALIAS).
 *  - dtype selects the storage of the token tensors (u, delta, z, B, C, x,
 *    streams, out): VM_F32 or VM_BF16.  A, D and delta_bias are always fp32.
 *    Arithmetic is fp32 (bf16 inputs are widened exactly; bf16 outputs are
 *    rounded to nearest even).
 *  - Work is enqueued asynchronously on `stream` (a hipStream_t; NULL = the
 *    default stream).  Argument checks run on the host first and nothing is
 *    launched when they fail.  Kernel-side faults surface at the caller's next
 *    synchronisation; VM_ERR_HIP reports a launch failure.
 *  - No data-dependent checks run on the device: A <= 0, finite inputs and a
 *    non-negative step size are preconditions of the method, and NaN / Inf
 *    propagate by IEEE rules.
 *  - Some calls need temporary device memory (noted at the call); it comes
 *    from a stream-ordered pool owned by the library and is released on the
 *    same stream before the call returns (VM_ERR_ALLOC if unavailable).
 *  - Calls are thread-safe.
 *
 * The pages this follows (cited by title and section):
 *  [Vim]  "Vision Mamba: Bidirectional State Space Models for Images"
 *  [EVM]  "EfficientVMamba: Atrous Selective Scan for Light Weight Visual Mamba"
 *  [FVim] "Fast Vision Mamba: Pooling Spatial Dimensions for Accelerated
 *         Processing"
 *  [NoD]  "Norm or Direction? Decoding Vision Mambas for High-Resolution
 *         Vision"
 */
#ifndef VM_SCAN_H
#define VM_SCAN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Storage type of token tensors. */
enum { VM_F32 = 0, VM_BF16 = 1 };

/* Status codes returned by every entry point. */
enum {
  VM_OK = 0,
  VM_ERR_NULL = 1,        /* a required pointer is NULL                      */
  VM_ERR_SHAPE = 2,       /* a size is <= 0, or an element count overflows   */
  VM_ERR_DTYPE = 3,       /* unknown dtype                                    */
  VM_ERR_FLAG = 4,        /* a flag or pool_axis is not 0/1, or options has
                             unknown bits                                     */
  VM_ERR_ALIAS = 5,       /* the output overlaps an input                     */
  VM_ERR_UNSUPPORTED = 6, /* dstate outside [1, 16], a head size past its
                             limit (see the call), a non-finite scale, or
                             sizes past the kernels' 32-bit offsets or grid
                             limits: 32 rows of seqlen + 16 steps, or one
                             batch row of B or C, must span < 2 GiB; the map
                             calls (atrous, pooled, SS2D) take at most
                             2^24 - 1 planes (batch * channels), the scans
                             at most 2^24 - 1 row blocks of 16 channels
                             (batch * ceil(dim / 16))                         */
  VM_ERR_HIP = 7,         /* a HIP launch or runtime call failed              */
  VM_ERR_ALLOC = 8        /* temporary device memory could not be obtained    */
};

/*
 * Options of the scan entry points (`options`, bitwise OR; any other bit is
 * VM_ERR_FLAG):
 *   VM_DELTA_SOFTPLUS  dt = softplus(delta + bias); without it dt = delta + bias
 *   VM_ZOH             write with the exact zero-order-hold coefficient
 *                      (exp(dt A) - 1) / A in place of dt ([NoD] section 3,
 *                      eq. 2, for diagonal A; [Vim] "A state retains, writes,
 *                      and reads" gives the scalar form and notes that the
 *                      released recurrence uses dt).  Its A -> 0 limit is dt.
 *                      Evaluated in fp32 to within about 5e-7 relative,
 *                      including small dt A, where exp(dt A) - 1 would cancel.
 * The released Vim model is options = VM_DELTA_SOFTPLUS.
 */
enum { VM_DELTA_SOFTPLUS = 1, VM_ZOH = 2 };

/* Human-readable name of a status code (static storage; never NULL). */
const char *vm_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int vm_version(void);

/*
 * One scan direction, in the argument order of the selective-scan function
 * on [Vim] implementation row 4 ("Keep a running state, then read it"):
 *   u           [batch, dim, seqlen]    token content (dtype)
 *   delta       [batch, dim, seqlen]    step-size pre-activation (dtype),
 *                                       before bias and softplus
 *   A           [dim, dstate]  fp32     decay; A = -exp(A_log), so A <= 0
 *   B, C        [batch, dstate, seqlen] input write / output read (dtype),
 *                                       shared by all channels of a batch row
 *   D           [dim]          fp32     direct skip (required)
 *   delta_bias  [dim]          fp32     added to delta before softplus; NULL = 0
 *   bc_stride   storage of B and C:
 *                 0   dense [batch, dstate, seqlen] as written above;
 *                 >0  token-major: element (b, n, t) at (b*seqlen + t)*bc_stride
 *                     + n, i.e. the [batch, dstate, seqlen] tensors are
 *                     transposed views of [batch, seqlen, >= dstate] memory.
 *                     This is how the page's projection produces B and C (it
 *                     splits the projected tokens and passes transposed
 *                     views); both layouts are read in place.
 *                     Requires bc_stride >= dstate.
 *   conv_w      [dim, 4]       fp32     NULL: u is the scan input as given.
 *                                       Non-NULL: u holds the content x before
 *                                       the block's depthwise causal conv, and
 *                                       the scan input is computed on the fly
 *                                       as SiLU(conv(x)) (vm_causal_conv1d_silu,
 *                                       with this direction's reverse sense);
 *                                       the D skip uses that input.  Only
 *                                       vm_selective_scan_fwd and
 *                                       vm_bidir_scan_fwd (both directions or
 *                                       neither) accept it; elsewhere
 *                                       VM_ERR_UNSUPPORTED.
 *   conv_b      [dim]          fp32     conv bias; NULL = 0 (ignored without
 *                                       conv_w)
 * For vm_pool_scan_repeat the shapes differ (see there).
 */
typedef struct vm_scan_dir {
  const void *u;
  const void *delta;
  const float *A;
  const void *B;
  const void *C;
  const float *D;
  const float *delta_bias;
  int64_t bc_stride;
  const float *conv_w;
  const float *conv_b;
} vm_scan_dir;

/*
 * Selective scan, one direction ([Vim] "A state retains, writes, and reads"
 * and implementation row 4).  For every (b, d), from a zero state:
 *   dt_t   = softplus(delta_t + bias_d)   (options & VM_DELTA_SOFTPLUS)
 *          = delta_t + bias_d             (otherwise)
 *   h_t,n  = exp(dt_t A_d,n) h_t-1,n + k_t,n B_b,n,t u_t
 *   k_t,n  = dt_t, or (exp(dt_t A_d,n) - 1) / A_d,n with VM_ZOH
 *   y_t    = sum_n C_b,n,t h_t,n + D_d u_t
 *   out_t  = y_t * SiLU(z_t)   (z != NULL),   y_t otherwise
 * reverse = 1 visits t = seqlen-1 .. 0 instead, which equals reversing every
 * token tensor, scanning forward and reversing the result ([Vim] "Two scans
 * meet at the same token").  All tensors stay in original token order.
 *   z, out: [batch, dim, seqlen] (dtype).  dstate in [1, 16].
 */
int vm_selective_scan_fwd(const vm_scan_dir *p, const void *z, void *out,
                          int64_t batch, int64_t dim, int64_t seqlen,
                          int64_t dstate, int dtype, int options,
                          int reverse, void *stream);

/*
 * Bidirectional scan with the aligned combine and shared gate ([Vim] "Two
 * scans meet at the same token", "Inside the released Vim block",
 * implementation row 5):
 *   out = combine_scale * (y_fwd + y_bwd) * SiLU(z)
 * y_fwd is the forward scan of `fwd`; y_bwd is the reversed-order scan of
 * `bwd` (its own u, delta, A, B, C, D, bias), returned in original order.
 * combine_scale = 0.5 is the released averaging model, 1 the summed form.
 * z may be NULL (no gate).  out: [batch, dim, seqlen] (dtype).
 * Temporary memory: for sequences too long for the on-chip exchange buffer
 * (seqlen above 552; 520 with a fused conv), an fp32 [batch, dim, seqlen rounded up to 32]
 * exchange buffer from the library's stream-ordered pool.  With VM_F32, a
 * seqlen that is a multiple of 32 and a 128-byte aligned `out`, `out` itself
 * serves as the exchange buffer and nothing is allocated.
 */
int vm_bidir_scan_fwd(const vm_scan_dir *fwd, const vm_scan_dir *bwd,
                      const void *z, float combine_scale, void *out,
                      int64_t batch, int64_t dim, int64_t seqlen,
                      int64_t dstate, int dtype, int options,
                      void *stream);

/*
 * vm_bidir_scan_fwd for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, results and checks as vm_bidir_scan_fwd, and
 * the same kernels; it calls no hipMalloc, hipFree or allocating routine.
 * Where vm_bidir_scan_fwd would take its exchange buffer from the pool (a
 * sequence past the on-chip exchange whose `out` cannot serve), this entry
 * uses a library-owned device array of 8 Mi fp32 values (32 MiB; one per
 * GPU the library runs on, held until the process ends):
 *   batch * dim * (seqlen rounded up to 32) must be at most 8388608, else
 *   VM_ERR_UNSUPPORTED (checked on the host before any HIP call).
 * Every call on one GPU shares that array and leaves its contents behind
 * (each exchange row is written before it is read, so nothing needs
 * clearing): calls that overlap in time on one GPU (different streams or
 * host threads) race and must not be issued.
 */
int vm_bidir_scan_fwd_noalloc(const vm_scan_dir *fwd, const vm_scan_dir *bwd,
                              const void *z, float combine_scale, void *out,
                              int64_t batch, int64_t dim, int64_t seqlen,
                              int64_t dstate, int dtype, int options,
                              void *stream);

/*
 * Depthwise causal convolution of width 4 with bias, then SiLU: the step
 * that produces the scan input u from the block's content x ([Vim] "Inside
 * the released Vim block": each branch's content passes through its own
 * kernel-four causal Conv1d, then SiLU; the backward branch reverses the
 * sequence first).  For every row (b, d):
 *   forward      u_t = SiLU(bias_d + sum_k w_d,k x_{t-3+k})
 *   reverse = 1  u_t = SiLU(bias_d + sum_k w_d,k x_{t+3-k})
 * with x = 0 outside [0, seqlen): w_d,3 weights the current token, w_d,0 the
 * token three steps earlier in the direction's visit order, and the
 * convolution does not reach across rows.
 *   x, out [batch, dim, seqlen] (dtype); w [dim, 4] fp32; bias [dim] fp32
 *   (NULL = 0).  The same result feeds the block's projections of delta, B
 *   and C; the scan entry points can recompute it from x (conv_w).
 * Limit: batch * dim * seqlen below 2^33 elements (VM_ERR_UNSUPPORTED).
 */
int vm_causal_conv1d_silu(const void *x, const float *w, const float *bias,
                          void *out, int64_t batch, int64_t dim,
                          int64_t seqlen, int reverse, int dtype,
                          void *stream);

/*
 * Backward of vm_causal_conv1d_silu: the gradients of L = sum(du * u) for
 * the same x, w, bias and direction (the pages pin gradients only as
 * automatic differentiation of the forward loop).  With dv = du SiLU'(v),
 * v the convolution plus bias:
 *   dx_t  = sum_k w_d,k dv_{t+3-k}  (forward; reverse: dv_{t-3+k})
 *   dw_d,k = sum over b, t of dv_t x_{t-3+k}  (reverse: x_{t+3-k})
 *   dbias_d = sum over b, t of dv_t
 *   x [batch, dim, seqlen] (dtype); w [dim, 4], bias [dim] (NULL = 0) fp32;
 *   du [batch, dim, seqlen] fp32 (the scan backward's u gradient);
 *   dx [batch, dim, seqlen], dw [dim, 4] fp32; dbias [dim] fp32 or NULL
 *   (not computed).  Outputs must not overlap the inputs or each other
 *   (VM_ERR_ALIAS).  dw and dbias are summed in a fixed order
 *   (deterministic).
 * Temporary memory: per-chunk partial sums, about 2048 * 5 floats.
 * Limits: dim at most 2^24 - 1, and seqlen times the rows of one chunk below
 * 2^31 (VM_ERR_UNSUPPORTED).
 */
int vm_causal_conv1d_silu_bwd(const void *x, const float *w, const float *bias,
                              const float *du, float *dx, float *dw, float *dbias,
                              int64_t batch, int64_t dim, int64_t seqlen, int reverse,
                              int dtype, void *stream);

/*
 * Number of steps of each p = 2 atrous group: ceil(H/2) * ceil(W/2)
 * ([EVM] implementation row 1).  Returns -VM_ERR_SHAPE for H or W <= 0.
 * Pure host function.
 */
int64_t vm_atrous_group_len(int64_t height, int64_t width);

/*
 * Atrous gather, p = 2 ([EVM] "Four shorter sequences, one dense output",
 * implementation row 1).  x [batch, channels, H, W] -> streams
 * [batch, 4, channels, Lg].  Group k has offset (row, col) = (0,0), (1,0),
 * (0,1), (1,1); groups 0 and 2 walk the half grid row-major, 1 and 3
 * column-major.  The map is padded right/bottom to even size; padded steps
 * hold +0.0.  A bit-exact copy.
 */
int vm_atrous_gather(const void *x, void *streams, int64_t batch,
                     int64_t channels, int64_t height, int64_t width,
                     int dtype, void *stream);

/*
 * Atrous scatter / merge ([EVM] "Merge restores coordinates instead of adding
 * directions", implementation row 3): the inverse routing, then a crop of the
 * padding.  streams [batch, 4, channels, Lg] -> y [batch, channels, H, W];
 * each valid coordinate takes its single owner's value; nothing is summed.
 * A bit-exact copy.
 */
int vm_atrous_scatter(const void *streams, void *y, int64_t batch,
                      int64_t channels, int64_t height, int64_t width,
                      int dtype, void *stream);

/*
 * FastVim pooled scan ([FVim] "Methodology"): mean-pool u over one spatial
 * axis, run the selective scan on the pooled tokens (forward, plus backward
 * when bwd != NULL), repeat the result along the pooled axis, gate with the
 * full-resolution SiLU(z):
 *   out[b,d,i,j] = combine_scale * (y_fwd + y_bwd)[b,d,p] * SiLU(z[b,d,i,j])
 *   p = i, Lp = H for pool_axis = 0 (mean over W)
 *   p = j, Lp = W for pool_axis = 1 (mean over H)
 * Per direction: u [batch, dim, H, W] (full resolution), delta [batch, dim,
 * Lp], B and C [batch, dstate, Lp] (the pooled tokens' projections), A, D,
 * delta_bias as for vm_selective_scan_fwd.  The D skip acts on the pooled u.
 * z, out: [batch, dim, H, W].  z may be NULL.  Temporary memory: fp32
 * [batch, dim, Lp] buffers for the pooled u of each direction and the scan
 * result, and fp32 copies of delta, B and C with VM_BF16.
 */
int vm_pool_scan_repeat(const vm_scan_dir *fwd, const vm_scan_dir *bwd,
                        const void *z, float combine_scale, void *out,
                        int64_t batch, int64_t dim, int64_t height,
                        int64_t width, int64_t dstate, int pool_axis,
                        int dtype, int options, void *stream);

/*
 * Four-direction 2-D selective scan with summed merge ([NoD] section 3,
 * "2D Selective Scan (SS2D)": four traversals of the map, one S6 scan each,
 * outputs restored to the map and merged; the merge of full SS2D adds the
 * four aligned outputs, [EVM] "Merge restores coordinates instead of adding
 * directions"):
 *   traversal 0: row-major, pixel (i, j) at step i*W + j
 *   traversal 1: traversal 0 reversed
 *   traversal 2: column-major, pixel (i, j) at step j*H + i
 *   traversal 3: traversal 2 reversed
 *   out[b,d,i,j] = combine_scale * sum_k y_k[b,d,(i,j)] * SiLU(z[b,d,i,j])
 * u, z, out: [batch, dim, H, W] (dtype); z may be NULL.  dirs[4]: the four
 * traversals' parameters; dirs[k].u is ignored (every traversal reads u).
 * delta [batch, dim, H*W] and B, C [batch, dstate, H*W] (or token-major, see
 * bc_stride) are indexed by traversal step: row-major for traversals 0 and 1,
 * column-major for 2 and 3.  A traversal's D skip adds D * u at each pixel,
 * so the merged skip is (D_0 + D_1 + D_2 + D_3) * u.  The H and W 32-pixel
 * tile counts multiplied must not exceed 65535 (VM_ERR_UNSUPPORTED).
 * Temporary memory: fp32 [batch, dim, H, W] buffers for the transposed u and
 * the column traversals' sum, plus (VM_BF16) the row traversals' sum and fp32
 * copies of u, delta, B and C, plus the exchange buffers of long sequences as
 * in vm_bidir_scan_fwd.
 */
int vm_ss2d_scan_fwd(const vm_scan_dir *dirs, const void *u, const void *z,
                     float combine_scale, void *out, int64_t batch,
                     int64_t dim, int64_t height, int64_t width,
                     int64_t dstate, int dtype, int options,
                     void *stream);

/*
 * Gradients of one scan direction (fp32 device buffers, owned by the
 * caller).  dB and dC are dense [batch, dstate, seqlen] whatever the layout
 * of B and C; ddelta_bias may be NULL (not computed).
 */
typedef struct vm_scan_grad {
  float *du;           /* [batch, dim, seqlen] */
  float *ddelta;       /* [batch, dim, seqlen] */
  float *dA;           /* [dim, dstate]        */
  float *dB;           /* [batch, dstate, seqlen] */
  float *dC;           /* [batch, dstate, seqlen] */
  float *dD;           /* [dim]                */
  float *ddelta_bias;  /* [dim] or NULL        */
  /* With the fused conv (conv_w in the direction, whose u is then the conv
     input x): du receives the gradient with respect to x, and these the
     conv parameters' (dconv_b NULL = not computed).  Unused otherwise. */
  float *dconv_w;      /* [dim, 4]             */
  float *dconv_b;      /* [dim] or NULL        */
} vm_scan_grad;

/*
 * Backward pass of vm_selective_scan_fwd: the gradients of
 * L = sum(dout * out) with respect to every input, for the same arguments
 * (the pages pin the backward pass only as automatic differentiation of the
 * scan loop, [Vim] "A state retains, writes, and reads" and implementation
 * row 4; the adjoint recurrence it implies is g_t = C_t dy_t + a_{t+1} g_{t+1}).
 *   dout [batch, dim, seqlen] (dtype); g: the gradients (see vm_scan_grad);
 *   dz [batch, dim, seqlen] fp32: required exactly when z is given.
 * Gradients are fp32 for either dtype (VM_BF16 inputs are widened exactly
 * and the pass runs in fp32).  Either write (options as the forward call's:
 * with VM_ZOH the derivatives of k = expm1(dt A) / A are included, A = 0
 * among them), with or without the fused conv (see vm_scan_grad).  Gradient buffers must not
 * overlap any input or each other (VM_ERR_ALIAS).  Sums over batch rows (dA,
 * dD, ddelta_bias) and over channels (dB, dC) are formed from per-block
 * partials in a fixed order, so results are deterministic.
 * Temporary memory: state checkpoints ([batch * dim, seqlen / 8, 16] fp32),
 * the partials ([dim / 16, batch, dstate, seqlen] fp32 for each of dB, dC),
 * with z the recomputed forward output and dy, with VM_BF16 fp32 copies of
 * the token tensors, and with the fused conv the conv output, its gradient
 * and the conv backward's partial sums.
 */
int vm_selective_scan_bwd(const vm_scan_dir *p, const void *z,
                          const void *dout, const vm_scan_grad *g, void *dz,
                          int64_t batch, int64_t dim, int64_t seqlen,
                          int64_t dstate, int dtype, int options, int reverse,
                          void *stream);

/*
 * Backward pass of vm_bidir_scan_fwd: gf and gb receive the gradients of the
 * forward and backward directions' inputs, dz (required when z is given) the
 * gate's.  The same limits and temporary memory as vm_selective_scan_bwd,
 * with checkpoints for each direction and, without VM_ZOH, partials for
 * each direction (both directions' backward kernels run as one launch),
 * plus, with z and sequences too long for the on-chip exchange, the
 * recomputation's fp32 exchange rows (as vm_bidir_scan_fwd).  All temporary
 * memory is taken before the first launch.
 */
int vm_bidir_scan_bwd(const vm_scan_dir *fwd, const vm_scan_dir *bwd,
                      const void *z, const void *dout, float combine_scale,
                      const vm_scan_grad *gf, const vm_scan_grad *gb, void *dz,
                      int64_t batch, int64_t dim, int64_t seqlen,
                      int64_t dstate, int dtype, int options, void *stream);

/*
 * Backward pass of vm_pool_scan_repeat ([FVim] "Methodology"), with the same
 * arguments and dout [batch, dim, H, W] (dtype).  gf (and gb when bwd is
 * given) receive their direction's gradients: du at full resolution
 * [batch, dim, H, W] (the mean pool's backward spreads each pooled
 * gradient times 1/w over its line), the others at the pooled length Lp as
 * in vm_selective_scan_bwd; dz [batch, dim, H, W] fp32, required exactly
 * when z is given.  The pooled output's gradient sums the gated dout over
 * the repeated axis in index order (deterministic).  The same options,
 * limits and temporary memory as the scan backward (at length Lp), plus
 * pooled buffers; no fused conv (VM_ERR_UNSUPPORTED).
 */
int vm_pool_scan_repeat_bwd(const vm_scan_dir *fwd, const vm_scan_dir *bwd,
                            const void *z, const void *dout, float combine_scale,
                            const vm_scan_grad *gf, const vm_scan_grad *gb, void *dz,
                            int64_t batch, int64_t dim, int64_t height, int64_t width,
                            int64_t dstate, int pool_axis, int dtype, int options,
                            void *stream);

/*
 * Backward pass of vm_ss2d_scan_fwd ([NoD] section 3, "2D Selective Scan
 * (SS2D)"), with the same arguments and dout [batch, dim, H, W] (dtype).
 *   grads: four gradient sets, one per traversal, for its delta, A, B, C, D
 *   and delta_bias (their du field is ignored); du [batch, dim, H, W] fp32
 *   receives the map's gradient, summed over the four traversals; dz
 *   [batch, dim, H, W] fp32, required exactly when z is given.
 * The same options and limits as the scan backward at length H * W, and
 * as vm_ss2d_scan_fwd.  Temporary memory: the transposed map, with z the
 * recomputed row and column sums, the output gradient in both layouts,
 * four map gradients, and the scan backward's checkpoints and partials for
 * each traversal (the four backward kernels run as one launch).
 */
int vm_ss2d_scan_bwd(const vm_scan_dir *dirs, const void *u, const void *z,
                     const void *dout, float combine_scale, const vm_scan_grad *grads,
                     float *du, void *dz, int64_t batch, int64_t dim, int64_t height,
                     int64_t width, int64_t dstate, int dtype, int options, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Matrix-state mixers: the gated delta rule, the per-head norm and rotation of
 * its queries and keys, and the clipping of gradients by their global norm.
 * Token tensors of these calls are token-major, [batch, seqlen, heads, dim]: a
 * head's values are contiguous, so one projection's output row can be passed
 * as it is.  A token stride (elements from one token to the next; 0 = dense,
 * heads * dim; otherwise >= heads * dim) lets q, k and v be slices of such a
 * row; the stride from one batch row to the next is seqlen token strides.
 * The dtype selects the storage of q, k, v, out and of their gradients;
 * everything else is fp32.
 * Calls that need temporary device memory take a workspace: device memory of
 * at least the bytes that the call's _workspace function returns, 256-byte
 * aligned, free for the call's work on its stream until that work is done.
 * workspace = NULL: the memory comes from the library's stream-ordered pool.
 * With a workspace a call makes no allocation and can be captured in a graph.
 * A workspace that is too small or not aligned is VM_ERR_ALLOC.
 * ---------------------------------------------------------------------------
 */

/*
 * Inputs of the gated delta rule.  Value heads hv are a multiple of key heads
 * hk: value head h reads key head h / (hv / hk).
 *   q, k     [batch, seqlen, hk, dk]   token stride q_stride, k_stride
 *   v        [batch, seqlen, hv, dv]   token stride v_stride
 *   g        [batch, seqlen, hv] fp32  log of the decay, g <= 0 (dense); values
 *                                      below -120, -Inf among them, decay to 0
 *   beta     [batch, seqlen, hv] fp32  write strength (dense)
 *   h0       [n, hv, dk, dv] fp32      initial states; NULL = 0
 *   offsets  [n + 1] int32             NULL: n = batch sequences of seqlen
 *                                      tokens.  Else batch is 1 and sequence i
 *                                      is tokens offsets[i] .. offsets[i+1]-1 of
 *                                      the packed row: non-decreasing from 0 to
 *                                      seqlen (a precondition; the kernels clamp
 *                                      what they read to [0, seqlen], and with
 *                                      other offsets the results are undefined
 *                                      but no access leaves the tensors).  A
 *                                      sequence may be empty.
 */
typedef struct vm_delta {
  const void *q;
  const void *k;
  const void *v;
  const float *g;
  const float *beta;
  const float *h0;
  const int32_t *offsets;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
} vm_delta;

/*
 * The gated delta rule.  For every sequence and value head, from S_0 = h0:
 *   S'_t = exp(g_t) S_{t-1}
 *   S_t  = S'_t + beta_t k_t (v_t - S'_t^T k_t)^T
 *   out_t = scale S_t^T q_t
 * reverse = 1 visits the tokens of each sequence from its last to its first.
 *   out    [batch, seqlen, hv, dv] (dtype), dense; tokens of no sequence are
 *          not written
 *   state  [n, hv, dk, dv] fp32: the last states; NULL = not kept.  An empty
 *          sequence's is its h0.  May be h0 itself (the states then advance in
 *          place), but must not overlap it otherwise.
 *   n      number of sequences (batch without offsets)
 * dk and dv in [1, 128], hv up to 65535, n hv up to 2^21 - 8, up to 2^23 - 1
 * chunks of 64 steps over all sequences, and token strides (hv dv among them)
 * below 2^23 elements: VM_ERR_UNSUPPORTED beyond.  hv % hk != 0 is VM_ERR_SHAPE.
 * Sequences are computed in chunks of 64 steps, within which a NaN or Inf of one
 * token reaches the outputs of earlier tokens too.
 */
int vm_gated_delta_fwd(const vm_delta *p, void *out, float *state, float scale,
                       int64_t batch, int64_t seqlen, int64_t n, int64_t hk,
                       int64_t hv, int64_t dk, int64_t dv, int dtype,
                       int reverse, void *workspace, int64_t workspace_bytes,
                       void *stream);

/*
 * Workspace of vm_gated_delta_fwd (backward = 0) or vm_gated_delta_bwd
 * (backward = 1), with packed = 1 for sequences given by offsets.  About 37 KB
 * (fp32: 25 KB) per 64 tokens and value head, backward 55 KB (37 KB) + 8 dk dv +
 * 512 dv bytes.
 * Returns -VM_ERR_SHAPE or -VM_ERR_UNSUPPORTED for sizes that no call (on rows of
 * whole 16-byte pieces, where the sizes allow them) takes, as the other
 * _workspace functions do.  Pure host function.
 */
int64_t vm_gated_delta_workspace(int64_t batch, int64_t seqlen, int64_t n,
                                 int64_t hv, int64_t dk, int64_t dv, int dtype,
                                 int packed, int backward);

/* Gradients of the gated delta rule (dense; the caller's buffers). */
typedef struct vm_delta_grad {
  void *dq;      /* [batch, seqlen, hk, dk] (dtype), summed over the value heads of a key head */
  void *dk;      /* [batch, seqlen, hk, dk] (dtype) */
  void *dv;      /* [batch, seqlen, hv, dv] (dtype) */
  float *dg;     /* [batch, seqlen, hv] */
  float *dbeta;  /* [batch, seqlen, hv] */
  float *dh0;    /* [n, hv, dk, dv] or NULL (not computed) */
} vm_delta_grad;

/*
 * Backward pass of vm_gated_delta_fwd: the gradients of
 * L = sum(dout * out) + sum(dstate * state) for the same arguments.
 *   dout [batch, seqlen, hv, dv] (dtype), dense; dstate [n, hv, dk, dv] or
 *   NULL (= 0).  Gradients of tokens of no sequence are not written.  A token
 *   whose g is below -120 has dg as if it were -120 (0).
 * Outputs must not overlap any input or each other.  Sums over value heads
 * and over a chunk are formed in a fixed order (deterministic).
 * Sizes as forward; with bf16 rows of whole pieces (dk a multiple of 8, dv even)
 * and dk > 64 also n hv ceil(dv / 32) below 2^22 (n hv in whole eights with
 * offsets): VM_ERR_UNSUPPORTED beyond.
 */
int vm_gated_delta_bwd(const vm_delta *p, const void *dout, const float *dstate,
                       const vm_delta_grad *grad, float scale, int64_t batch,
                       int64_t seqlen, int64_t n, int64_t hk, int64_t hv,
                       int64_t dk, int64_t dv, int dtype, int reverse,
                       void *workspace, int64_t workspace_bytes,
                       void *stream);

/*
 * One token of the gated delta rule for every row of a batch, on states that
 * are kept: q, k [batch, hk, dk], v, out [batch, hv, dv] (dtype), g, beta
 * [batch, hv] fp32, all dense; state [n_slots, hv, dk, dv] fp32 is updated in
 * place.  slots [batch] int32: the state of each row, NULL = row b uses state
 * b (batch <= n_slots, else VM_ERR_SHAPE).  A row whose slot is outside
 * [0, n_slots) is idle: its out is zero and it touches no state.  Two rows
 * must not name the same slot (their updates would race).  No temporary
 * memory, one launch: the call can be captured in a graph.
 */
int vm_gated_delta_step(const void *q, const void *k, const void *v,
                        const float *g, const float *beta, float *state,
                        const int32_t *slots, void *out, float scale,
                        int64_t batch, int64_t n_slots, int64_t hk, int64_t hv,
                        int64_t dk, int64_t dv, int dtype, void *stream);

/*
 * Per-head norm and rotation of queries and keys, options of `norm_options`
 * (bitwise OR; other bits VM_ERR_FLAG):
 *   VM_NORM_L2           divide by sqrt(sum x^2 + eps); without it by
 *                        sqrt(mean x^2 + eps)
 *   VM_ROPE_INTERLEAVED  rotate the pairs (2i, 2i+1); without it (i, i + rot/2)
 */
enum { VM_NORM_L2 = 1, VM_ROPE_INTERLEAVED = 2 };

/*
 *   q [batch, seqlen, hq, dim], k [batch, seqlen, hk, dim] (dtype; k may be
 *   NULL with hk = 0), token strides as above.
 *   wq, wk [dim] fp32: gains after the norm; NULL = 1.
 *   cos, sin [table, rot / 2] fp32: the rotation's table; rot (even, in
 *   [0, dim]) leading values of each head are turned; rot = 0: no rotation,
 *   cos, sin, positions unused.
 *   positions [batch, seqlen] int32: each token's row of the table; NULL =
 *   0 .. seqlen - 1.  A token whose position is outside [0, table) is padding:
 *   its outputs and gradients are zero and it adds nothing to dwq and dwk.
 */
typedef struct vm_head_norm {
  const void *q;
  const void *k;
  const float *wq;
  const float *wk;
  const float *cos;
  const float *sin;
  const int32_t *positions;
  int64_t q_stride;
  int64_t k_stride;
  int64_t table;
  int64_t rot;
} vm_head_norm;

/*
 * q_out, k_out = rotate(gain * normalise(q)), and of k: dense, the shapes of
 * q and k, both in one launch.  dim in [1, 512] (VM_ERR_UNSUPPORTED beyond).
 */
int vm_head_norm_rope(const vm_head_norm *p, void *q_out, void *k_out,
                      int64_t batch, int64_t seqlen, int64_t hq, int64_t hk,
                      int64_t dim, float eps, int norm_options, int dtype,
                      void *stream);

/*
 * Its backward: from dq_out, dk_out (dense, dtype) the gradients dq, dk
 * (dense, dtype) and dwq, dwk [dim] fp32 (NULL = not computed; only with the
 * gain given, else VM_ERR_NULL).  Summed in a fixed order (deterministic).
 * A workspace is needed only for dwq or dwk.
 */
int vm_head_norm_rope_bwd(const vm_head_norm *p, const void *dq_out,
                          const void *dk_out, void *dq, void *dk, float *dwq,
                          float *dwk, int64_t batch, int64_t seqlen, int64_t hq,
                          int64_t hk, int64_t dim, float eps, int norm_options,
                          int dtype, void *workspace,
                          int64_t workspace_bytes, void *stream);

/* Workspace of vm_head_norm_rope_bwd.  Pure host function. */
int64_t vm_head_norm_rope_workspace(int64_t dim);

/* One gradient of vm_clip_grad_norm.  elems may be 0. */
typedef struct vm_grad_tensor {
  const void *in;
  void *out;      /* NULL: only counted in the norm; may be in itself */
  int64_t elems;
  int64_t dtype;  /* VM_F32 or VM_BF16, of in and out */
} vm_grad_tensor;

/*
 * The Euclidean norm over every element of `count` gradients, and each
 * gradient scaled to at most that norm:
 *   norm = sqrt(sum in^2),  out = in * min(1, max_norm / (norm + 1e-6))
 * list is host memory, read before the call returns.  norm [1] fp32 (device)
 * receives the norm (required).  Squares are summed in fp64, in a fixed order
 * (deterministic); a NaN or Inf among the gradients follows the formula by
 * IEEE rules.  max_norm < 0 or NaN is VM_ERR_UNSUPPORTED.  An out must not
 * overlap its in except by being it, nor any other tensor of the list (the
 * latter is not checked).  count in [0, 65536] (VM_ERR_UNSUPPORTED beyond).
 */
int vm_clip_grad_norm(const vm_grad_tensor *list, int64_t count, float max_norm,
                      float *norm, void *workspace, int64_t workspace_bytes,
                      void *stream);

/* Workspace of vm_clip_grad_norm.  Pure host function. */
int64_t vm_clip_grad_workspace(int64_t count);

/*
 * ---------------------------------------------------------------------------
 * Prompts and single tokens: the selective scan and its short convolution over
 * rows of tokens, as a language model's block has them, and the norms around a
 * block.  Token tensors are token-major, [batch, seqlen, dim], with a token stride
 * (elements; 0 = dense, otherwise >= the row's values) that lets them be slices of
 * one projection's row; the stride from one batch row to the next is seqlen token
 * strides.  Strides and workspaces are as in the section above.  The dtype selects
 * the storage of token tensors, of their gradients and of kept windows; parameters,
 * states and their gradients are fp32.
 * ---------------------------------------------------------------------------
 */

/*
 * The sequences of a call; NULL: every batch row is one, and states are numbered
 * as they are.
 *   offsets  [n + 1] int32  NULL: n = batch sequences of seqlen tokens.  Else batch
 *                           is 1 and sequence i is tokens offsets[i] ..
 *                           offsets[i+1]-1 of the packed row: non-decreasing from 0
 *                           to at most seqlen (a precondition; the kernels clamp what
 *                           they read to [0, seqlen], and with other offsets the
 *                           results are undefined but no access leaves the tensors).
 *                           A sequence may be empty; its state stays its first.
 *                           Tokens behind the last sequence are not written (with
 *                           VM_CLEAR_REST: zeros are).
 *   slots    [n] int32      where in h0 and state (both of n_slots states) each
 *                           sequence's state lies; NULL: sequence i has state i, of n.
 *                           A sequence whose slot is outside [0, n_slots) starts from
 *                           zero and its state is not kept.  Two sequences must not
 *                           name the same slot.
 *   fresh    [n] int32      nonzero: the sequence starts from zero though h0 is given;
 *                           NULL: none does
 * The backward calls take offsets only (slots or fresh: VM_ERR_FLAG).
 *
 * VM_CLEAR_REST, beside the other options of a scan over prompts or added to a
 * convolution's silu: the rows behind the last sequence are set to zero in every
 * output of a call that holds rows of tokens.  In buffers that are new to each call
 * they would hold whatever was there, which a sum over all rows takes up.  (The calls
 * on single tokens have no such rows: VM_ERR_FLAG.)
 */
enum { VM_CLEAR_REST = 16 };
typedef struct vm_sequences {
  const int32_t *offsets;
  const int32_t *slots;
  const int32_t *fresh;
  int64_t n;
  int64_t n_slots;
} vm_sequences;

/*
 * Depthwise causal convolution over rows of tokens, with SiLU (silu = 1) or
 * without (0): with x before a sequence's first token from its kept window,
 *   v_t = bias + sum_k w_k x_{t-width+1+k},   out_t = SiLU(v_t) or v_t
 *   x [batch, seqlen, dim] (dtype), token stride x_stride; w [dim, width], bias
 *   [dim] (NULL = 0) fp32; out dense.
 *   h0, state [n or n_slots, width - 1, dim] (dtype): the inputs before the first
 *   token and the last ones, oldest first; NULL = 0 / not kept.  state may be h0
 *   itself, but must not overlap it otherwise.
 * width in [2, 4], dim up to 2^22 (VM_ERR_UNSUPPORTED).  One launch, no temporary
 * memory.
 */
int vm_prompt_conv(const vm_sequences *q, const void *x, int64_t x_stride,
                   const float *w, const float *bias, const void *h0,
                   void *state, void *out, int64_t batch, int64_t seqlen,
                   int64_t dim, int64_t width, int silu, int dtype,
                   void *stream);

/* Gradients of vm_prompt_conv (dense; the caller's buffers). */
typedef struct vm_conv_grad {
  void *dx;      /* [batch, seqlen, dim] (dtype) */
  float *dw;     /* [dim, width] */
  float *dbias;  /* [dim] or NULL (not computed) */
  void *dh0;     /* [n, width - 1, dim] (dtype) or NULL */
} vm_conv_grad;

/*
 * Backward pass of vm_prompt_conv: the gradients of
 * L = sum(dout * out) + sum(dstate * state) for the same arguments.
 *   dout [batch, seqlen, dim] (dtype), dense; dstate [n, width - 1, dim] (dtype) or
 *   NULL (= 0).  Gradients of tokens of no sequence are not written (with
 *   VM_CLEAR_REST: they are 0).  Sums are formed in a fixed order (deterministic).
 */
int vm_prompt_conv_bwd(const vm_sequences *q, const void *x, int64_t x_stride,
                       const float *w, const float *bias, const void *h0,
                       const void *dout, const void *dstate,
                       const vm_conv_grad *grad, int64_t batch, int64_t seqlen,
                       int64_t dim, int64_t width, int silu, int dtype,
                       void *workspace, int64_t workspace_bytes, void *stream);

/* Workspace of vm_prompt_conv_bwd (packed = 1 with offsets).  Pure host function. */
int64_t vm_prompt_conv_workspace(int64_t batch, int64_t seqlen, int64_t n,
                                 int64_t dim, int64_t width, int dtype,
                                 int packed);

/*
 * One token of that convolution for every row of a batch, on kept windows:
 * x [batch, dim] (dtype), row stride x_stride; state [n_slots, width - 1, dim]
 * (dtype) is advanced in place; out [batch, dim], dense.  slots [batch] int32: the
 * window of each row, NULL = row b uses window b (batch <= n_slots, else
 * VM_ERR_SHAPE).  A row whose slot is outside [0, n_slots) is idle: its out is zero
 * and it touches no window.  Two rows must not name the same slot.  One launch, no
 * temporary memory.
 */
int vm_token_conv(const void *x, int64_t x_stride, const float *w,
                  const float *bias, void *state, const int32_t *slots,
                  void *out, int64_t batch, int64_t n_slots, int64_t dim,
                  int64_t width, int silu, int dtype, void *stream);

/*
 * Inputs of the selective scan over rows of tokens (vm_scan_dir's, token-major):
 *   u, delta, z  [batch, seqlen, dim]     z NULL: no gate
 *   B, C         [batch, seqlen, dstate]
 *   A [dim, dstate], D [dim] (NULL = 0), delta_bias [dim] (NULL = 0)  fp32
 * and the token strides of the five token tensors.
 */
typedef struct vm_scan_rows {
  const void *u;
  const void *delta;
  const float *A;
  const void *B;
  const void *C;
  const float *D;
  const float *delta_bias;
  const void *z;
  int64_t u_stride;
  int64_t delta_stride;
  int64_t B_stride;
  int64_t C_stride;
  int64_t z_stride;
} vm_scan_rows;

/*
 * The selective scan over rows of tokens, from given states.  For every sequence
 * and channel, with the recurrence of vm_selective_scan_fwd:
 *   h_t = exp(dt_t A) h_{t-1} + dt_t B_t u_t,  y_t = C_t h_t + D u_t,
 *   out_t = y_t SiLU(z_t)  (z != NULL),  y_t otherwise
 *   h0, state [n or n_slots, dim, dstate] fp32: first and last states; NULL = 0 /
 *   not kept.  state may be h0 itself, but must not overlap it otherwise.
 *   out [batch, seqlen, dim] (dtype), dense.  options: VM_DELTA_SOFTPLUS or 0,
 *   VM_CLEAR_REST (the write is dt; VM_ZOH is VM_ERR_FLAG).
 * dstate in [1, 16], dim up to 2^22, token strides below 2^23 elements
 * (VM_ERR_UNSUPPORTED).  Long sequences of few channels are walked in chunks at
 * once, whose states need a workspace (vm_prompt_scan_workspace; 0 bytes where
 * there is one chunk to a sequence).
 */
int vm_prompt_scan(const vm_scan_rows *p, const vm_sequences *q,
                   const float *h0, float *state, void *out, int64_t batch,
                   int64_t seqlen, int64_t dim, int64_t dstate, int dtype,
                   int options, void *workspace, int64_t workspace_bytes,
                   void *stream);

/*
 * Workspace of vm_prompt_scan (backward = 0) or vm_prompt_scan_bwd (backward = 1),
 * with packed = 1 for sequences given by offsets.  At 16 states the backward pass
 * takes about 8 bytes per token and channel and 270 per chunk and channel, the
 * forward pass 70 per chunk and channel (packed: one chunk or more to each of the
 * n sequences).  Pure host function.
 */
int64_t vm_prompt_scan_workspace(int64_t batch, int64_t seqlen, int64_t n,
                                 int64_t dim, int64_t dstate, int packed,
                                 int backward);

/* Gradients of the selective scan over rows (dense; the caller's buffers). */
typedef struct vm_rows_grad {
  void *du;           /* [batch, seqlen, dim] (dtype) */
  void *ddelta;       /* [batch, seqlen, dim] (dtype) */
  float *dA;          /* [dim, dstate] */
  void *dB;           /* [batch, seqlen, dstate] (dtype) */
  void *dC;           /* [batch, seqlen, dstate] (dtype) */
  float *dD;          /* [dim] or NULL (not computed) */
  float *ddelta_bias; /* [dim] or NULL */
  void *dz;           /* [batch, seqlen, dim] (dtype): required exactly with z */
  float *dh0;         /* [n, dim, dstate] or NULL */
} vm_rows_grad;

/*
 * Backward pass of vm_prompt_scan: the gradients of
 * L = sum(dout * out) + sum(dstate * state) for the same arguments.
 *   dout [batch, seqlen, dim] (dtype), dense; dstate [n, dim, N] or NULL (= 0).
 * Gradients of tokens of no sequence are not written (with VM_CLEAR_REST: they are
 * 0).  Outputs must not overlap any input or each other.  Sums over channels, rows
 * and chunks are formed in a fixed order (deterministic).
 */
int vm_prompt_scan_bwd(const vm_scan_rows *p, const vm_sequences *q,
                       const float *h0, const void *dout, const float *dstate,
                       const vm_rows_grad *grad, int64_t batch, int64_t seqlen,
                       int64_t dim, int64_t N, int dtype, int options,
                       void *workspace, int64_t workspace_bytes, void *stream);

/*
 * One token of the selective scan for every row of a batch, on states that are
 * kept: the rows of p with seqlen 1; state [n_slots, dim, dstate] fp32 is updated
 * in place; out [batch, dim] (dtype), dense; slots as for vm_token_conv.  (Rows may
 * lie as far apart as 2^31 - 1 elements.)  One launch, no temporary memory.
 */
int vm_token_scan(const vm_scan_rows *p, float *state, const int32_t *slots,
                  void *out, int64_t batch, int64_t n_slots, int64_t dim,
                  int64_t dstate, int dtype, int options, void *stream);

/*
 * Options of the norms around a block (others VM_ERR_FLAG):
 *   VM_NORM_CENTER      before: take the mean off first
 *   VM_NORM_GATE_FIRST  after: the norm of x SiLU(z), not SiLU(z) times that of x
 */
enum { VM_NORM_CENTER = 4, VM_NORM_GATE_FIRST = 8 };

/*
 * What a norm around a block is taken of.
 *   x       [rows, dim] (dtype), row stride x_stride (0 = dense)
 *   w       [w_dim] fp32 gains, NULL = 1; w_dim = dim (or 0), or, after a block,
 *           group: the same gains for every group
 *   b       [dim] fp32, NULL = 0; before a block only (else VM_ERR_FLAG)
 *   scale   [dim] fp32: residual scale of each channel, NULL = 1; factor: of all
 *   z       [rows, dim] (dtype), row stride z_stride: the gate after a block, NULL =
 *           none; NULL before one
 *   group   channels that are normed together, a divisor of dim; 0 = dim (before a
 *           block only dim)
 */
typedef struct vm_block_norm {
  const void *x;
  const float *w;
  const float *b;
  const float *scale;
  const void *z;
  int64_t x_stride;
  int64_t z_stride;
  int64_t w_dim;
  int64_t group;
  float eps;
  float factor;
  int32_t options;
} vm_block_norm;

/*
 * The norm before a block, of the residual with the last block's output added:
 *   r = residual + factor scale x,   y = (r - mean) / sqrt(mean (r - mean)^2 + eps)
 *   w + b    (mean = 0 without VM_NORM_CENTER; of r in fp32, before it is rounded)
 *   residual, r [rows, dim] (rdtype: dtype, or VM_F32 beside bf16 rows; else
 *   VM_ERR_DTYPE), dense; residual NULL = 0, r NULL = not kept, r may be residual
 *   itself; y [rows, dim] (dtype), dense.
 * dim up to 16384, rows below 2^31 (VM_ERR_UNSUPPORTED).  One launch.
 */
int vm_norm_before(const vm_block_norm *p, const void *residual, void *y,
                   void *r, int64_t rows, int64_t dim, int dtype, int rdtype,
                   void *stream);

/* Gradients of the norms around a block; NULL = not computed. */
typedef struct vm_norm_grad {
  void *dx;         /* [rows, dim] (dtype); after a block required */
  void *dresidual;  /* [rows, dim] (rdtype); before a block only */
  void *dz;         /* [rows, dim] (dtype): after a block, required exactly with z */
  float *dw;        /* [w_dim] */
  float *db;        /* [dim]; before a block only */
  float *dscale;    /* [dim] */
} vm_norm_grad;

/*
 * Backward pass of vm_norm_before at the residual r that it gave: from dy (dtype)
 * and dr (rdtype; what else arrives at r, NULL = 0), both dense,
 *   dresidual = dr + the norm's gradient,  dx = factor scale dresidual
 * and dw, db, dscale (only where w, b, scale are given, else VM_ERR_NULL; dscale
 * needs x, which is not read otherwise and may be NULL).  At least one of dx and
 * dresidual is given.  Summed in a fixed order (deterministic); a workspace is
 * needed only for dw, db or dscale.
 */
int vm_norm_before_bwd(const vm_block_norm *p, const void *r, const void *dy,
                       const void *dr, const vm_norm_grad *grad, int64_t rows,
                       int64_t dim, int dtype, int rdtype, void *workspace,
                       int64_t workspace_bytes, void *stream);

/*
 * The norm after a block, by groups of channels, gated and added to the residual:
 *   y = n(x) w SiLU(z)  or (VM_NORM_GATE_FIRST)  n(x SiLU(z)) w,
 *   n(v) = v / sqrt(mean v^2 + eps) over a group;  out = residual + factor scale y
 *   residual, out [rows, dim] (rdtype), dense; residual NULL = 0; out may be
 *   residual itself.
 * group up to 16384, dim up to 2^22, rows below 2^31 (VM_ERR_UNSUPPORTED).  One
 * launch.
 */
int vm_norm_after(const vm_block_norm *p, const void *residual, void *out,
                  int64_t rows, int64_t dim, int dtype, int rdtype,
                  void *stream);

/*
 * Its backward: from dout [rows, dim] (rdtype), dense, the gradients dx, dz, dw and
 * dscale (the residual's is dout itself).  Deterministic; a workspace as above.
 */
int vm_norm_after_bwd(const vm_block_norm *p, const void *dout,
                      const vm_norm_grad *grad, int64_t rows, int64_t dim,
                      int dtype, int rdtype, void *workspace,
                      int64_t workspace_bytes, void *stream);

/* Workspace of the norms' backward passes (group 0 = dim).  Pure host function. */
int64_t vm_block_norm_workspace(int64_t rows, int64_t dim, int64_t group);

#ifdef __cplusplus
}
#endif

#endif /* VM_SCAN_H */
