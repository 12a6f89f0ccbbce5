"""Selective-scan hot path for vision Mamba backbones on AMD MI355X (gfx950).

Thin Python binding over the C ABI in include/vm_scan.h (libvmscan.so, built
in-tree by ``selective_scan_fwd_amd.build``).  The functions here only check
tensor shapes / dtypes / devices and marshal pointers; every step of the
computation runs in the library's HIP kernels on the current torch stream.
PyTorch supplies device memory and the stream.  There is no fallback: if the
library is missing or fails to load, every call raises.

Names and argument order follow the C ABI:
  vm_selective_scan_fwd, vm_bidir_scan_fwd, vm_atrous_gather,
  vm_atrous_scatter, vm_pool_scan_repeat, vm_ss2d_scan_fwd,
  vm_causal_conv1d_silu, vm_causal_conv1d_silu_bwd, vm_selective_scan_bwd,
  vm_bidir_scan_bwd, vm_pool_scan_repeat_bwd, vm_ss2d_scan_bwd,
  vm_atrous_group_len; the matrix-state mixers: vm_gated_delta_fwd,
  vm_gated_delta_bwd, vm_gated_delta_step, vm_head_norm_rope,
  vm_head_norm_rope_bwd, vm_clip_grad_norm; and the scan over prompts and single
  tokens with the norms around a block: vm_prompt_conv, vm_prompt_conv_bwd,
  vm_token_conv, vm_prompt_scan, vm_prompt_scan_bwd, vm_token_scan,
  vm_norm_before, vm_norm_before_bwd, vm_norm_after, vm_norm_after_bwd.
"""
from __future__ import annotations

import array
import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvmscan.so")

VM_F32, VM_BF16 = 0, 1
VM_DELTA_SOFTPLUS, VM_ZOH = 1, 2
VM_NORM_L2, VM_ROPE_INTERLEAVED = 1, 2
VM_NORM_CENTER, VM_NORM_GATE_FIRST = 4, 8
VM_CLEAR_REST = 16
VM_OK = 0
STATUS_NAMES = {0: "VM_OK", 1: "VM_ERR_NULL", 2: "VM_ERR_SHAPE", 3: "VM_ERR_DTYPE", 4: "VM_ERR_FLAG",
                5: "VM_ERR_ALIAS", 6: "VM_ERR_UNSUPPORTED", 7: "VM_ERR_HIP", 8: "VM_ERR_ALLOC"}

EXPORTED = ("vm_status_string", "vm_version", "vm_selective_scan_fwd", "vm_bidir_scan_fwd",
            "vm_bidir_scan_fwd_noalloc",
            "vm_atrous_group_len", "vm_atrous_gather", "vm_atrous_scatter", "vm_pool_scan_repeat",
            "vm_ss2d_scan_fwd", "vm_causal_conv1d_silu", "vm_causal_conv1d_silu_bwd",
            "vm_selective_scan_bwd", "vm_bidir_scan_bwd", "vm_pool_scan_repeat_bwd",
            "vm_ss2d_scan_bwd",
            "vm_gated_delta_fwd", "vm_gated_delta_bwd", "vm_gated_delta_step",
            "vm_head_norm_rope", "vm_head_norm_rope_bwd", "vm_clip_grad_norm",
            "vm_gated_delta_workspace", "vm_head_norm_rope_workspace", "vm_clip_grad_workspace",
            "vm_prompt_conv", "vm_prompt_conv_bwd", "vm_token_conv", "vm_prompt_scan", "vm_prompt_scan_bwd",
            "vm_token_scan", "vm_norm_before", "vm_norm_before_bwd", "vm_norm_after", "vm_norm_after_bwd",
            "vm_prompt_conv_workspace", "vm_prompt_scan_workspace", "vm_block_norm_workspace")


class VmScanDir(ctypes.Structure):
    """struct vm_scan_dir (one scan direction's device pointers)."""
    _fields_ = [("u", ctypes.c_void_p), ("delta", ctypes.c_void_p), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("C", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("delta_bias", ctypes.c_void_p), ("bc_stride", ctypes.c_int64),
                ("conv_w", ctypes.c_void_p), ("conv_b", ctypes.c_void_p)]


class VmScanGrad(ctypes.Structure):
    """struct vm_scan_grad (one direction's gradient buffers)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("du", "ddelta", "dA", "dB", "dC", "dD", "ddelta_bias",
                                                "dconv_w", "dconv_b")]


class VmDelta(ctypes.Structure):
    """struct vm_delta (inputs of the gated delta rule)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("q", "k", "v", "g", "beta", "h0", "offsets")] + \
               [(k, ctypes.c_int64) for k in ("q_stride", "k_stride", "v_stride")]


class VmDeltaGrad(ctypes.Structure):
    """struct vm_delta_grad (gradient buffers of the gated delta rule)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("dq", "dk", "dv", "dg", "dbeta", "dh0")]


class VmHeadNorm(ctypes.Structure):
    """struct vm_head_norm (inputs of the per-head norm and rotation)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("q", "k", "wq", "wk", "cos", "sin", "positions")] + \
               [(k, ctypes.c_int64) for k in ("q_stride", "k_stride", "table", "rot")]


class VmGradTensor(ctypes.Structure):
    """struct vm_grad_tensor (one gradient of vm_clip_grad_norm)."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("elems", ctypes.c_int64),
                ("dtype", ctypes.c_int64)]


class VmSequences(ctypes.Structure):
    """struct vm_sequences (the sequences of a call over rows of tokens)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("offsets", "slots", "fresh")] + \
               [(k, ctypes.c_int64) for k in ("n", "n_slots")]


class VmConvGrad(ctypes.Structure):
    """struct vm_conv_grad (gradient buffers of the convolution over rows)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("dx", "dw", "dbias", "dh0")]


class VmScanRows(ctypes.Structure):
    """struct vm_scan_rows (inputs of the selective scan over rows)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("u", "delta", "A", "B", "C", "D", "delta_bias", "z")] + \
               [(k, ctypes.c_int64) for k in ("u_stride", "delta_stride", "B_stride", "C_stride", "z_stride")]


class VmRowsGrad(ctypes.Structure):
    """struct vm_rows_grad (gradient buffers of the selective scan over rows)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("du", "ddelta", "dA", "dB", "dC", "dD", "ddelta_bias", "dz", "dh0")]


class VmBlockNorm(ctypes.Structure):
    """struct vm_block_norm (inputs of the norms around a block)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("x", "w", "b", "scale", "z")] + \
               [(k, ctypes.c_int64) for k in ("x_stride", "z_stride", "w_dim", "group")] + \
               [("eps", ctypes.c_float), ("factor", ctypes.c_float), ("options", ctypes.c_int32)]


class VmNormGrad(ctypes.Structure):
    """struct vm_norm_grad (gradient buffers of the norms around a block)."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("dx", "dresidual", "dz", "dw", "db", "dscale")]


class VmError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(msg)
        self.status = status


_lock = threading.Lock()
_lib = None


def load_library():
    """Load libvmscan.so and declare the C signatures.  Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is not built; run selective_scan_fwd_amd.build.build() "
                                   "first")
            lib = ctypes.CDLL(LIB_PATH)
            P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
            D = ctypes.POINTER(VmScanDir)
            lib.vm_status_string.argtypes = [I]
            lib.vm_status_string.restype = ctypes.c_char_p
            lib.vm_version.argtypes = []
            lib.vm_version.restype = I
            lib.vm_selective_scan_fwd.argtypes = [D, P, P, I64, I64, I64, I64, I, I, I, P]
            lib.vm_bidir_scan_fwd.argtypes = [D, D, P, F, P, I64, I64, I64, I64, I, I, P]
            lib.vm_bidir_scan_fwd_noalloc.argtypes = [D, D, P, F, P, I64, I64, I64, I64, I, I, P]
            lib.vm_atrous_group_len.argtypes = [I64, I64]
            lib.vm_atrous_group_len.restype = I64
            lib.vm_atrous_gather.argtypes = [P, P, I64, I64, I64, I64, I, P]
            lib.vm_atrous_scatter.argtypes = [P, P, I64, I64, I64, I64, I, P]
            lib.vm_pool_scan_repeat.argtypes = [D, D, P, F, P, I64, I64, I64, I64, I64, I, I, I, P]
            lib.vm_ss2d_scan_fwd.argtypes = [D, P, P, F, P, I64, I64, I64, I64, I64, I, I, P]
            lib.vm_causal_conv1d_silu.argtypes = [P, P, P, P, I64, I64, I64, I, I, P]
            lib.vm_causal_conv1d_silu_bwd.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I, I, P]
            G = ctypes.POINTER(VmScanGrad)
            lib.vm_selective_scan_bwd.argtypes = [D, P, P, G, P, I64, I64, I64, I64, I, I, I, P]
            lib.vm_bidir_scan_bwd.argtypes = [D, D, P, P, F, G, G, P, I64, I64, I64, I64, I, I, P]
            lib.vm_pool_scan_repeat_bwd.argtypes = [D, D, P, P, F, G, G, P, I64, I64, I64, I64, I64, I, I, I, P]
            lib.vm_ss2d_scan_bwd.argtypes = [D, P, P, P, F, G, P, P, I64, I64, I64, I64, I64, I, I, P]
            X, Y = ctypes.POINTER(VmDelta), ctypes.POINTER(VmDeltaGrad)
            N = ctypes.POINTER(VmHeadNorm)
            lib.vm_gated_delta_fwd.argtypes = [X, P, P, F, I64, I64, I64, I64, I64, I64, I64, I, I, P, I64, P]
            lib.vm_gated_delta_bwd.argtypes = [X, P, P, Y, F, I64, I64, I64, I64, I64, I64, I64, I, I, P, I64, P]
            lib.vm_gated_delta_step.argtypes = [P, P, P, P, P, P, P, P, F, I64, I64, I64, I64, I64, I64, I, P]
            lib.vm_head_norm_rope.argtypes = [N, P, P, I64, I64, I64, I64, I64, F, I, I, P]
            lib.vm_head_norm_rope_bwd.argtypes = [N, P, P, P, P, P, P, I64, I64, I64, I64, I64, F, I, I, P, I64, P]
            lib.vm_clip_grad_norm.argtypes = [ctypes.POINTER(VmGradTensor), I64, F, P, P, I64, P]
            lib.vm_gated_delta_workspace.argtypes = [I64, I64, I64, I64, I64, I64, I, I, I]
            lib.vm_head_norm_rope_workspace.argtypes = [I64]
            lib.vm_clip_grad_workspace.argtypes = [I64]
            Q, R, B = ctypes.POINTER(VmSequences), ctypes.POINTER(VmScanRows), ctypes.POINTER(VmBlockNorm)
            K = ctypes.POINTER(VmNormGrad)
            lib.vm_prompt_conv.argtypes = [Q, P, I64, P, P, P, P, P, I64, I64, I64, I64, I, I, P]
            lib.vm_prompt_conv_bwd.argtypes = [Q, P, I64, P, P, P, P, P, ctypes.POINTER(VmConvGrad), I64, I64, I64, I64, I, I,
                                               P, I64, P]
            lib.vm_token_conv.argtypes = [P, I64, P, P, P, P, P, I64, I64, I64, I64, I, I, P]
            lib.vm_prompt_scan.argtypes = [R, Q, P, P, P, I64, I64, I64, I64, I, I, P, I64, P]
            lib.vm_prompt_scan_bwd.argtypes = [R, Q, P, P, P, ctypes.POINTER(VmRowsGrad), I64, I64, I64, I64, I, I, P, I64, P]
            lib.vm_token_scan.argtypes = [R, P, P, P, I64, I64, I64, I64, I, I, P]
            lib.vm_norm_before.argtypes = [B, P, P, P, I64, I64, I, I, P]
            lib.vm_norm_before_bwd.argtypes = [B, P, P, P, K, I64, I64, I, I, P, I64, P]
            lib.vm_norm_after.argtypes = [B, P, P, I64, I64, I, I, P]
            lib.vm_norm_after_bwd.argtypes = [B, P, K, I64, I64, I, I, P, I64, P]
            lib.vm_prompt_conv_workspace.argtypes = [I64, I64, I64, I64, I64, I, I]
            lib.vm_prompt_scan_workspace.argtypes = [I64, I64, I64, I64, I64, I, I]
            lib.vm_block_norm_workspace.argtypes = [I64, I64, I64]
            for name in ("vm_gated_delta_workspace", "vm_head_norm_rope_workspace", "vm_clip_grad_workspace",
                         "vm_prompt_conv_workspace", "vm_prompt_scan_workspace", "vm_block_norm_workspace"):
                getattr(lib, name).restype = I64
            for name in ("vm_gated_delta_fwd", "vm_gated_delta_bwd", "vm_gated_delta_step", "vm_head_norm_rope",
                         "vm_head_norm_rope_bwd", "vm_clip_grad_norm",
                         "vm_prompt_conv", "vm_prompt_conv_bwd", "vm_token_conv", "vm_prompt_scan", "vm_prompt_scan_bwd",
                         "vm_token_scan", "vm_norm_before", "vm_norm_before_bwd", "vm_norm_after", "vm_norm_after_bwd",
                         "vm_selective_scan_fwd", "vm_bidir_scan_fwd", "vm_bidir_scan_fwd_noalloc",
                         "vm_atrous_gather",
                         "vm_atrous_scatter", "vm_pool_scan_repeat", "vm_ss2d_scan_fwd",
                         "vm_causal_conv1d_silu", "vm_causal_conv1d_silu_bwd", "vm_selective_scan_bwd",
                         "vm_bidir_scan_bwd", "vm_pool_scan_repeat_bwd", "vm_ss2d_scan_bwd"):
                getattr(lib, name).restype = I
            _lib = lib
    return _lib


def vm_status_string(status: int) -> str:
    return load_library().vm_status_string(int(status)).decode()


def vm_version() -> int:
    return int(load_library().vm_version())


def _check(status, what):
    if status != VM_OK:
        raise VmError(status, f"{what}: {vm_status_string(status)}")


# ---------------------------------------------------------------- marshalling
def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return VM_F32
    if t.dtype == torch.bfloat16:
        return VM_BF16
    raise TypeError(f"token tensors must be float32 or bfloat16, got {t.dtype}")


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _bc(t: torch.Tensor, name: str, dtype, shape, device):
    """B or C [batch, N, L]: dense, or a transposed view of token-major
    [batch, L, >= N] memory.  Returns the C ABI's bc_stride (0 = dense)."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    batch, n, L = shape
    if t.is_contiguous():
        return 0
    sb, sn, st = t.stride()
    if sn == 1 and st >= n and (sb == L * st or batch == 1):
        return st
    raise ValueError(f"{name} must be dense [batch, N, L] or a transposed view of token-major "
                     f"[batch, L, >= N] memory (strides {t.stride()})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _options(delta_softplus, zoh):
    return (VM_DELTA_SOFTPLUS if delta_softplus else 0) | (VM_ZOH if zoh else 0)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _direction(p, batch, dim, u_shape, tok_len, dstate, dt, device, name):
    """Validate one direction dict and return (VmScanDir, keepalive)."""
    u = _dev(p["u"], f"{name}.u", dt, u_shape, device)
    delta = _dev(p["delta"], f"{name}.delta", dt, (batch, dim, tok_len), device)
    A = _dev(p["A"], f"{name}.A", torch.float32, (dim, dstate), device)
    B, C = p["B"], p["C"]
    sB = _bc(B, f"{name}.B", dt, (batch, dstate, tok_len), device)
    sC = _bc(C, f"{name}.C", dt, (batch, dstate, tok_len), device)
    if sB != sC:
        raise ValueError(f"{name}.B and {name}.C must share one layout (bc strides {sB} vs {sC})")
    D = _dev(p["D"], f"{name}.D", torch.float32, (dim,), device)
    bias = p.get("delta_bias")
    if bias is not None:
        bias = _dev(bias, f"{name}.delta_bias", torch.float32, (dim,), device)
    cw, cb = p.get("conv_w"), p.get("conv_b")
    if cw is not None:
        cw = _dev(cw, f"{name}.conv_w", torch.float32, (dim, 4), device)
        if cb is not None:
            cb = _dev(cb, f"{name}.conv_b", torch.float32, (dim,), device)
    else:
        cb = None
    ptr = lambda t: t.data_ptr() if t is not None else None
    s = VmScanDir(u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
                  D.data_ptr(), ptr(bias), sB, ptr(cw), ptr(cb))
    return s, (u, delta, A, B, C, D, bias, cw, cb)


# ---------------------------------------------------------------- entry points
def vm_selective_scan_fwd(u, delta, A, B, C, D, z=None, delta_bias=None, delta_softplus=True,
                          reverse=False, out=None, zoh=False, conv_w=None, conv_b=None):
    """One-direction selective scan; returns out shaped like u.
    u, delta, z: [batch, dim, L]; A: [dim, N] fp32; B, C: [batch, N, L]
    (dense, or transposed views of token-major [batch, L, N] memory, which
    the kernels read directly); D, delta_bias: [dim] fp32.
    reverse=True visits t = L-1 .. 0.  zoh=True writes with the zero-order-hold
    coefficient (exp(dt A) - 1) / A instead of dt (every scan entry point
    takes delta_softplus and zoh).  conv_w [dim, 4] (and conv_b [dim]): u is
    the content before the block's causal conv and the scan runs on
    SiLU(conv(u)) computed in the kernel (vm_scan_dir.conv_w; direction dicts
    of vm_bidir_scan_fwd take the same keys)."""
    dt = u.dtype
    batch, dim, L = u.shape
    N = A.shape[-1]
    d, keep = _direction(dict(u=u, delta=delta, A=A, B=B, C=C, D=D, delta_bias=delta_bias,
                              conv_w=conv_w, conv_b=conv_b),
                         batch, dim, (batch, dim, L), L, N, dt, u.device, "p")
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)
    out = torch.empty_like(u) if out is None else _dev(out, "out", dt, u.shape, u.device)
    with torch.cuda.device(u.device):
        st = load_library().vm_selective_scan_fwd(ctypes.byref(d), _ptr(z), _ptr(out), batch, dim, L, N,
                                                  _dtype_code(u), _options(delta_softplus, zoh),
                                                  int(bool(reverse)), _stream(u.device))
    _check(st, "vm_selective_scan_fwd")
    return out


def vm_bidir_scan_fwd(fwd, bwd, z=None, combine_scale=1.0, delta_softplus=True, out=None, zoh=False):
    """Bidirectional scan: combine_scale * (y_fwd + y_bwd) * SiLU(z).
    fwd / bwd: dicts with u, delta, A, B, C, D, delta_bias (original token order)."""
    u = fwd["u"]
    dt = u.dtype
    batch, dim, L = u.shape
    N = fwd["A"].shape[-1]
    df, kf = _direction(fwd, batch, dim, (batch, dim, L), L, N, dt, u.device, "fwd")
    db, kb = _direction(bwd, batch, dim, (batch, dim, L), L, N, dt, u.device, "bwd")
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)
    out = torch.empty_like(u) if out is None else _dev(out, "out", dt, u.shape, u.device)
    with torch.cuda.device(u.device):
        st = load_library().vm_bidir_scan_fwd(ctypes.byref(df), ctypes.byref(db), _ptr(z),
                                              float(combine_scale), _ptr(out), batch, dim, L, N,
                                              _dtype_code(u), _options(delta_softplus, zoh),
                                              _stream(u.device))
    _check(st, "vm_bidir_scan_fwd")
    return out


def vm_bidir_scan_fwd_noalloc(fwd, bwd, out, z=None, combine_scale=1.0, delta_softplus=True, zoh=False):
    """vm_bidir_scan_fwd for callers that cannot allocate device memory: the
    same result, written into the caller's `out`; the exchange buffer of long
    sequences comes from a library-owned device array (batch * dim * (L
    rounded up to 32) <= 8388608, else VmError).  Calls on one GPU share that
    array: calls that overlap in time on one GPU must not be issued."""
    u = fwd["u"]
    dt = u.dtype
    batch, dim, L = u.shape
    N = fwd["A"].shape[-1]
    df, kf = _direction(fwd, batch, dim, (batch, dim, L), L, N, dt, u.device, "fwd")
    db, kb = _direction(bwd, batch, dim, (batch, dim, L), L, N, dt, u.device, "bwd")
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)
    _dev(out, "out", dt, u.shape, u.device)
    with torch.cuda.device(u.device):
        st = load_library().vm_bidir_scan_fwd_noalloc(ctypes.byref(df), ctypes.byref(db), _ptr(z),
                                                      float(combine_scale), _ptr(out), batch, dim, L, N,
                                                      _dtype_code(u), _options(delta_softplus, zoh),
                                                      _stream(u.device))
    _check(st, "vm_bidir_scan_fwd_noalloc")
    return out


def vm_causal_conv1d_silu(x, w, bias=None, reverse=False, out=None):
    """u = SiLU(depthwise causal conv of width 4 (+ bias)) per row of
    x [batch, dim, L]; w [dim, 4] fp32 (w[:, 3] on the current token);
    reverse=True convolves in reversed order (the backward branch)."""
    _dev(x, "x")
    dim = x.shape[1]
    _dev(w, "w", torch.float32, (dim, 4), x.device)
    if bias is not None:
        _dev(bias, "bias", torch.float32, (dim,), x.device)
    out = torch.empty_like(x) if out is None else _dev(out, "out", x.dtype, x.shape, x.device)
    batch, dim, L = x.shape
    with torch.cuda.device(x.device):
        st = load_library().vm_causal_conv1d_silu(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), batch, dim,
                                                  L, int(bool(reverse)), _dtype_code(x),
                                                  _stream(x.device))
    _check(st, "vm_causal_conv1d_silu")
    return out


def vm_causal_conv1d_silu_bwd(x, w, du, bias=None, reverse=False, with_dbias=None):
    """Gradients of sum(du * vm_causal_conv1d_silu(x, w, bias, reverse)):
    returns (dx, dw, dbias), fp32; du fp32 [batch, dim, L].  dbias is None
    when with_dbias is false (default: computed when bias is given)."""
    _dev(x, "x")
    batch, dim, L = x.shape
    _dev(w, "w", torch.float32, (dim, 4), x.device)
    _dev(du, "du", torch.float32, x.shape, x.device)
    if bias is not None:
        _dev(bias, "bias", torch.float32, (dim,), x.device)
    if with_dbias is None:
        with_dbias = bias is not None
    dx = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    dw = torch.empty((dim, 4), dtype=torch.float32, device=x.device)
    db = torch.empty((dim,), dtype=torch.float32, device=x.device) if with_dbias else None
    with torch.cuda.device(x.device):
        st = load_library().vm_causal_conv1d_silu_bwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(du), _ptr(dx),
                                                      _ptr(dw), _ptr(db), batch, dim, L,
                                                      int(bool(reverse)), _dtype_code(x), _stream(x.device))
    _check(st, "vm_causal_conv1d_silu_bwd")
    return dx, dw, db


def _grad_set(p, batch, dim, L, N, device, with_bias):
    """Gradient buffers of one direction; with the fused conv (p["conv_w"])
    also conv_w (and conv_b when p has one), and u is then the conv input's."""
    f = lambda *shape: torch.empty(shape, dtype=torch.float32, device=device)
    conv = p.get("conv_w") is not None
    g = dict(u=f(batch, dim, L), delta=f(batch, dim, L), A=f(dim, N), B=f(batch, N, L),
             C=f(batch, N, L), D=f(dim), delta_bias=f(dim) if with_bias else None)
    if conv:
        g["conv_w"] = f(dim, 4)
        g["conv_b"] = f(dim) if p.get("conv_b") is not None else None
    ptr = lambda k: g[k].data_ptr() if g.get(k) is not None else None
    s = VmScanGrad(*(ptr(k) for k in ("u", "delta", "A", "B", "C", "D", "delta_bias", "conv_w", "conv_b")))
    return s, g


def vm_selective_scan_bwd(p, dout, z=None, delta_softplus=True, reverse=False, zoh=False):
    """Gradients of sum(dout * vm_selective_scan_fwd(**p, z=z, ...)).  p: dict
    u, delta, A, B, C, D, delta_bias (token tensors fp32 or bf16, like dout and
    z).  Returns (grads, dz), fp32: grads has the keys of p (dB, dC dense
    [batch, N, L]); dz is None without z."""
    u = p["u"]
    dt = u.dtype
    batch, dim, L = u.shape
    N = p["A"].shape[-1]
    d, keep = _direction(p, batch, dim, (batch, dim, L), L, N, dt, u.device, "p")
    _dev(dout, "dout", dt, u.shape, u.device)
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)
    gs, g = _grad_set(p, batch, dim, L, N, u.device, p.get("delta_bias") is not None)
    dz = torch.empty(u.shape, dtype=torch.float32, device=u.device) if z is not None else None
    with torch.cuda.device(u.device):
        st = load_library().vm_selective_scan_bwd(ctypes.byref(d), _ptr(z), _ptr(dout), ctypes.byref(gs),
                                                  _ptr(dz), batch, dim, L, N, _dtype_code(u),
                                                  _options(delta_softplus, zoh), int(bool(reverse)),
                                                  _stream(u.device))
    _check(st, "vm_selective_scan_bwd")
    return g, dz


def vm_bidir_scan_bwd(fwd, bwd, dout, z=None, combine_scale=1.0, delta_softplus=True, zoh=False):
    """Gradients of sum(dout * vm_bidir_scan_fwd(fwd, bwd, z, combine_scale)).
    Returns (grads of fwd, grads of bwd, dz), fp32 for fp32 or bf16 inputs."""
    u = fwd["u"]
    dt = u.dtype
    batch, dim, L = u.shape
    N = fwd["A"].shape[-1]
    df, kf = _direction(fwd, batch, dim, (batch, dim, L), L, N, dt, u.device, "fwd")
    db, kb = _direction(bwd, batch, dim, (batch, dim, L), L, N, dt, u.device, "bwd")
    _dev(dout, "dout", dt, u.shape, u.device)
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)
    gsf, gf = _grad_set(fwd, batch, dim, L, N, u.device, fwd.get("delta_bias") is not None)
    gsb, gb = _grad_set(bwd, batch, dim, L, N, u.device, bwd.get("delta_bias") is not None)
    dz = torch.empty(u.shape, dtype=torch.float32, device=u.device) if z is not None else None
    with torch.cuda.device(u.device):
        st = load_library().vm_bidir_scan_bwd(ctypes.byref(df), ctypes.byref(db), _ptr(z), _ptr(dout),
                                              float(combine_scale), ctypes.byref(gsf), ctypes.byref(gsb),
                                              _ptr(dz), batch, dim, L, N, _dtype_code(u),
                                              _options(delta_softplus, zoh), _stream(u.device))
    _check(st, "vm_bidir_scan_bwd")
    return gf, gb, dz


def vm_atrous_group_len(height: int, width: int) -> int:
    n = int(load_library().vm_atrous_group_len(int(height), int(width)))
    if n < 0:
        raise VmError(-n, f"vm_atrous_group_len: {vm_status_string(-n)}")
    return n


def vm_atrous_gather(x, out=None):
    """x [batch, ch, H, W] -> streams [batch, 4, ch, ceil(H/2)*ceil(W/2)]."""
    _dev(x, "x")
    batch, ch, H, W = x.shape
    shape = (batch, 4, ch, vm_atrous_group_len(H, W))
    out = torch.empty(shape, dtype=x.dtype, device=x.device) if out is None else \
        _dev(out, "streams", x.dtype, shape, x.device)
    with torch.cuda.device(x.device):
        st = load_library().vm_atrous_gather(_ptr(x), _ptr(out), batch, ch, H, W, _dtype_code(x),
                                             _stream(x.device))
    _check(st, "vm_atrous_gather")
    return out


def vm_atrous_scatter(streams, height, width, out=None):
    """streams [batch, 4, ch, Lg] -> y [batch, ch, height, width]."""
    _dev(streams, "streams")
    batch, four, ch, Lg = streams.shape
    if four != 4 or Lg != vm_atrous_group_len(height, width):
        raise ValueError("streams must be [batch, 4, ch, ceil(H/2)*ceil(W/2)]")
    shape = (batch, ch, height, width)
    out = torch.empty(shape, dtype=streams.dtype, device=streams.device) if out is None else \
        _dev(out, "y", streams.dtype, shape, streams.device)
    with torch.cuda.device(streams.device):
        st = load_library().vm_atrous_scatter(_ptr(streams), _ptr(out), batch, ch, height, width,
                                              _dtype_code(streams), _stream(streams.device))
    _check(st, "vm_atrous_scatter")
    return out


def vm_pool_scan_repeat(fwd, bwd=None, z=None, combine_scale=1.0, pool_axis=0, delta_softplus=True,
                        out=None, zoh=False):
    """FastVim pooled scan.  Per direction: u [batch, dim, H, W], delta
    [batch, dim, Lp], B/C [batch, N, Lp] (Lp = H for pool_axis 0, W for 1).
    Returns [batch, dim, H, W]."""
    u = fwd["u"]
    dt = u.dtype
    batch, dim, H, W = u.shape
    Lp = H if pool_axis == 0 else W
    N = fwd["A"].shape[-1]
    df, kf = _direction(fwd, batch, dim, (batch, dim, H, W), Lp, N, dt, u.device, "fwd")
    pb = None
    if bwd is not None:
        db, kb = _direction(bwd, batch, dim, (batch, dim, H, W), Lp, N, dt, u.device, "bwd")
        pb = ctypes.byref(db)
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)
    out = torch.empty_like(u) if out is None else _dev(out, "out", dt, u.shape, u.device)
    with torch.cuda.device(u.device):
        st = load_library().vm_pool_scan_repeat(ctypes.byref(df), pb, _ptr(z), float(combine_scale),
                                                _ptr(out), batch, dim, H, W, N, int(pool_axis),
                                                _dtype_code(u), _options(delta_softplus, zoh),
                                                _stream(u.device))
    _check(st, "vm_pool_scan_repeat")
    return out


def vm_pool_scan_repeat_bwd(fwd, dout, bwd=None, z=None, combine_scale=1.0, pool_axis=0,
                            delta_softplus=True, zoh=False):
    """Gradients of sum(dout * vm_pool_scan_repeat(fwd, bwd, z, ...)).
    Returns (grads of fwd, grads of bwd or None, dz or None), fp32: u's
    gradient at full resolution, the others at the pooled length."""
    u = fwd["u"]
    dt = u.dtype
    batch, dim, H, W = u.shape
    Lp = H if pool_axis == 0 else W
    N = fwd["A"].shape[-1]
    df, kf = _direction(fwd, batch, dim, (batch, dim, H, W), Lp, N, dt, u.device, "fwd")
    pb, gsb, gb = None, None, None
    if bwd is not None:
        db, kb = _direction(bwd, batch, dim, (batch, dim, H, W), Lp, N, dt, u.device, "bwd")
        pb = ctypes.byref(db)
    _dev(dout, "dout", dt, u.shape, u.device)
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)

    def grad_set(p):
        s_, g_ = _grad_set(p, batch, dim, Lp, N, u.device, p.get("delta_bias") is not None)
        g_["u"] = torch.empty(u.shape, dtype=torch.float32, device=u.device)   # full resolution
        s_.du = g_["u"].data_ptr()
        return s_, g_

    gsf, gf = grad_set(fwd)
    if bwd is not None:
        gsb, gb = grad_set(bwd)
    dz = torch.empty(u.shape, dtype=torch.float32, device=u.device) if z is not None else None
    with torch.cuda.device(u.device):
        st = load_library().vm_pool_scan_repeat_bwd(
            ctypes.byref(df), pb, _ptr(z), _ptr(dout), float(combine_scale), ctypes.byref(gsf),
            ctypes.byref(gsb) if gsb is not None else None, _ptr(dz), batch, dim, H, W, N,
            int(pool_axis), _dtype_code(u), _options(delta_softplus, zoh), _stream(u.device))
    _check(st, "vm_pool_scan_repeat_bwd")
    return gf, gb, dz


def vm_ss2d_scan_fwd(u, dirs, z=None, combine_scale=1.0, delta_softplus=True, out=None, zoh=False):
    """Four-direction 2-D scan with summed merge.  u, z: [batch, dim, H, W].
    dirs: four dicts with delta, A, B, C, D, delta_bias (a "u" key is
    ignored); traversals 0 / 1 are row-major forward / reversed, 2 / 3
    column-major forward / reversed, and each indexes its delta [batch, dim,
    H*W] and B, C [batch, N, H*W] by its own traversal step.
    Returns combine_scale * (sum of the four aligned outputs) * SiLU(z)."""
    _dev(u, "u")
    dt = u.dtype
    batch, dim, H, W = u.shape
    if len(dirs) != 4:
        raise ValueError("dirs must hold four traversals")
    N = dirs[0]["A"].shape[-1]
    arr = (VmScanDir * 4)()
    keep = []
    for k, p in enumerate(dirs):
        d, kp = _direction(dict(p, u=u), batch, dim, (batch, dim, H, W), H * W, N, dt, u.device,
                           f"dirs[{k}]")
        arr[k] = d
        keep.append(kp)
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)
    out = torch.empty_like(u) if out is None else _dev(out, "out", dt, u.shape, u.device)
    with torch.cuda.device(u.device):
        st = load_library().vm_ss2d_scan_fwd(arr, _ptr(u), _ptr(z), float(combine_scale), _ptr(out),
                                             batch, dim, H, W, N, _dtype_code(u),
                                             _options(delta_softplus, zoh), _stream(u.device))
    _check(st, "vm_ss2d_scan_fwd")
    return out


def vm_ss2d_scan_bwd(u, dirs, dout, z=None, combine_scale=1.0, delta_softplus=True, zoh=False):
    """Gradients of sum(dout * vm_ss2d_scan_fwd(u, dirs, z, combine_scale)).
    Returns (du [batch, dim, H, W], per-traversal grads (four dicts with the
    keys of dirs, dB / dC dense [batch, N, H*W]), dz or None), all fp32."""
    _dev(u, "u")
    dt = u.dtype
    batch, dim, H, W = u.shape
    if len(dirs) != 4:
        raise ValueError("dirs must hold four traversals")
    N = dirs[0]["A"].shape[-1]
    arr = (VmScanDir * 4)()
    garr = (VmScanGrad * 4)()
    keep, grads = [], []
    for k, p in enumerate(dirs):
        d, kp = _direction(dict(p, u=u), batch, dim, (batch, dim, H, W), H * W, N, dt, u.device,
                           f"dirs[{k}]")
        arr[k] = d
        keep.append(kp)
        gs, g = _grad_set(dict(p, u=u), batch, dim, H * W, N, u.device, p.get("delta_bias") is not None)
        del g["u"]                  # the map's gradient is the summed du below
        gs.du = None
        garr[k] = gs
        grads.append(g)
    _dev(dout, "dout", dt, u.shape, u.device)
    if z is not None:
        _dev(z, "z", dt, u.shape, u.device)
    du = torch.empty(u.shape, dtype=torch.float32, device=u.device)
    dz = torch.empty(u.shape, dtype=torch.float32, device=u.device) if z is not None else None
    with torch.cuda.device(u.device):
        st = load_library().vm_ss2d_scan_bwd(arr, _ptr(u), _ptr(z), _ptr(dout), float(combine_scale), garr,
                                             _ptr(du), _ptr(dz), batch, dim, H, W, N, _dtype_code(u),
                                             _options(delta_softplus, zoh), _stream(u.device))
    _check(st, "vm_ss2d_scan_bwd")
    return du, grads, dz


# ------------------------------------------------------- matrix-state mixers
def _arg(t, name, dtype, shape, index):
    """Address of a contiguous tensor (None = NULL).  index: the GPU's number.
    The one quick test covers the good case; _dev says what is wrong."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0
            and t.is_contiguous()):
        _dev(t, name, dtype, shape, torch.device("cuda", index) if index >= 0 else None)
    return t.data_ptr()


def _current_stream(index):
    """The raw handle of torch's current stream (a Stream object costs 3 us)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _launch(name, index, *args):
    """Call an entry point on the current stream of GPU `index`."""
    call = getattr(load_library(), name)
    if index == torch.cuda.current_device():
        st = call(*args, _current_stream(index))
    else:
        with torch.cuda.device(index):
            st = call(*args, _current_stream(index))
    if st != VM_OK:
        _check(st, name)


def _workspace(nbytes, device):
    """Temporary memory of one call from torch's allocator, which hands it on in
    stream order.  Returns the tensor (to be kept until the call returns), its
    address and size."""
    if nbytes <= 0:                              # sizes that the call itself refuses
        return None, None, 0
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), nbytes


def _tokens(t, name, dtype, shape, index):
    """q, k or v [batch, seqlen, heads, dim]: each token's heads contiguous,
    tokens evenly spaced.  Returns the address and the C ABI's token stride
    (0 = dense)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} must be on a GPU device{', cuda:%d' % index if index >= 0 else ''} (got {t.device})")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    batch, L, heads, dim = shape
    sb, st, sh, sd = t.stride()
    step = st if L > 1 else sb                   # (one token a row: the batch stride is the token stride)
    if (sd == 1 or dim == 1) and (sh == dim or heads == 1) and step >= heads * dim and \
            (L == 1 or batch == 1 or sb == L * st):
        return t.data_ptr(), step
    raise ValueError(f"{name} must be [batch, seqlen, heads, dim] with contiguous heads and evenly spaced "
                     f"tokens (strides {t.stride()})")


def _delta(q, k, v, g, beta, h0, offsets):
    """Validate the gated delta rule's inputs; returns (VmDelta, GPU, sizes)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a [batch, seqlen, heads, dim] tensor")
    batch, L, hk, dk = q.shape
    hv, dv = v.shape[2:]
    index, dtype = q.get_device(), q.dtype
    pq, sq = _tokens(q, "q", dtype, (batch, L, hk, dk), index)
    pk, sk = _tokens(k, "k", dtype, (batch, L, hk, dk), index)
    pv, sv = _tokens(v, "v", dtype, (batch, L, hv, dv), index)
    pg = _arg(g, "g", torch.float32, (batch, L, hv), index)
    pb = _arg(beta, "beta", torch.float32, (batch, L, hv), index)
    n, po = batch, None
    if offsets is not None:
        if batch != 1:
            raise ValueError("packed sequences (offsets) take batch 1")
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError("offsets must be an int32 tensor [sequences + 1]")
        n = offsets.shape[0] - 1
        po = _arg(offsets, "offsets", torch.int32, (n + 1,), index)
    ph = _arg(h0, "h0", torch.float32, (n, hv, dk, dv), index)
    return VmDelta(pq, pk, pv, pg, pb, ph, po, sq, sk, sv), index, (batch, L, n, hk, hv, dk, dv)


def vm_gated_delta_fwd(q, k, v, g, beta, scale=None, h0=None, want_state=False, reverse=False, offsets=None,
                       out=None, state=None):
    """Gated delta rule over whole sequences; returns (out, state).
    q, k: [batch, L, hk, dk]; v: [batch, L, hv, dv] (hv a multiple of hk; fp32 or
    bf16; slices of a common projection row are read in place); g (log decay,
    <= 0), beta: [batch, L, hv] fp32; h0: [n, hv, dk, dv] fp32 or None;
    scale: dk ** -0.5 by default.  offsets (int32 [n + 1], batch 1): sequence i
    is tokens offsets[i] .. offsets[i + 1] - 1.  reverse=True visits each
    sequence from its last token.  out is [batch, L, hv, dv]; state (the last
    states, [n, hv, dk, dv] fp32) is None unless want_state or a state buffer
    (which may be h0) is given.  Rows behind the last packed sequence are not
    written: those of a new out hold what memory held."""
    p, index, (batch, L, n, hk, hv, dk, dv) = _delta(q, k, v, g, beta, h0, offsets)
    if out is None:
        out = torch.empty((batch, L, hv, dv), dtype=q.dtype, device=q.device)
    if state is None and want_state:
        state = torch.empty((n, hv, dk, dv), dtype=torch.float32, device=q.device)
    ws, wp, wn = _workspace(load_library().vm_gated_delta_workspace(batch, L, n, hv, dk, dv, _dtype_code(q),
                                                                    offsets is not None, 0), q.device)
    _launch("vm_gated_delta_fwd", index, p, _arg(out, "out", q.dtype, (batch, L, hv, dv), index),
            _arg(state, "state", torch.float32, (n, hv, dk, dv), index), dk ** -0.5 if scale is None else scale, batch, L,
            n, hk, hv, dk, dv, _dtype_code(q), int(bool(reverse)), wp, wn)
    return out, state


def vm_gated_delta_bwd(q, k, v, g, beta, dout, scale=None, h0=None, dstate=None, reverse=False, offsets=None):
    """Gradients of sum(dout * out) + sum(dstate * state) of vm_gated_delta_fwd.
    Returns a dict: q, k, v (dense, in their dtype), g, beta (fp32) and, when h0
    is given, h0 (fp32).  Rows behind the last packed sequence are not written: clear
    them before a sum over all rows."""
    p, index, (batch, L, n, hk, hv, dk, dv) = _delta(q, k, v, g, beta, h0, offsets)
    po = _arg(dout, "dout", q.dtype, (batch, L, hv, dv), index)
    ps = _arg(dstate, "dstate", torch.float32, (n, hv, dk, dv), index)
    make = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=q.device)
    d = dict(q=make(q.dtype, batch, L, hk, dk), k=make(q.dtype, batch, L, hk, dk), v=make(q.dtype, batch, L, hv, dv),
             g=make(torch.float32, batch, L, hv), beta=make(torch.float32, batch, L, hv))
    if h0 is not None:
        d["h0"] = make(torch.float32, n, hv, dk, dv)
    grads = VmDeltaGrad(*(d[x].data_ptr() if x in d else None for x in ("q", "k", "v", "g", "beta", "h0")))
    ws, wp, wn = _workspace(load_library().vm_gated_delta_workspace(batch, L, n, hv, dk, dv, _dtype_code(q),
                                                                    offsets is not None, 1), q.device)
    _launch("vm_gated_delta_bwd", index, p, po, ps, grads, dk ** -0.5 if scale is None else scale, batch, L, n, hk, hv,
            dk, dv, _dtype_code(q), int(bool(reverse)), wp, wn)
    return d


def vm_gated_delta_step(q, k, v, g, beta, state, scale=None, slots=None, out=None):
    """One token of the gated delta rule on kept states; returns out.
    q, k: [batch, hk, dk]; v: [batch, hv, dv]; g, beta: [batch, hv] fp32; state
    [n_slots, hv, dk, dv] fp32 is updated in place.  slots (int32 [batch]): each
    row's state (distinct); a row with a slot outside [0, n_slots) is idle: zero
    out, no state touched."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a [batch, heads, dim] tensor")
    batch, hk, dk = q.shape
    hv, dv = v.shape[1:]
    index, dtype = q.get_device(), q.dtype
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a [n_slots, hv, dk, dv] tensor")
    n = state.shape[0]
    if out is None:
        out = torch.empty_like(v)                # (v is dense, which the call checks)
    _launch("vm_gated_delta_step", index, _arg(q, "q", dtype, (batch, hk, dk), index),
            _arg(k, "k", dtype, (batch, hk, dk), index), _arg(v, "v", dtype, (batch, hv, dv), index),
            _arg(g, "g", torch.float32, (batch, hv), index), _arg(beta, "beta", torch.float32, (batch, hv), index),
            _arg(state, "state", torch.float32, (n, hv, dk, dv), index),
            _arg(slots, "slots", torch.int32, (batch,), index), _arg(out, "out", dtype, (batch, hv, dv), index),
            dk ** -0.5 if scale is None else scale, batch, n, hk, hv, dk, dv, _dtype_code(q))
    return out


def _head_norm(q, k, wq, wk, cos, sin, positions):
    for name, t in (("q", q), ("k", k)):
        if t is not None and (not isinstance(t, torch.Tensor) or t.dim() != 4):
            raise ValueError(f"{name} must be a [batch, seqlen, heads, dim] tensor")
    batch, L, hq, dim = q.shape
    hk = k.shape[2] if k is not None else 0
    index, dtype = q.get_device(), q.dtype
    pq, sq = _tokens(q, "q", dtype, (batch, L, hq, dim), index)
    pk, sk = _tokens(k, "k", dtype, (batch, L, hk, dim), index) if k is not None else (None, 0)
    table = rot = 0
    pc = ps = pp = None
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError("cos must be a [table, rot / 2] tensor")
        shape = cos.shape
        table, rot = shape[0], 2 * shape[1]
        pc, ps = _arg(cos, "cos", torch.float32, shape, index), _arg(sin, "sin", torch.float32, shape, index)
        pp = _arg(positions, "positions", torch.int32, (batch, L), index)
    s = VmHeadNorm(pq, pk, _arg(wq, "wq", torch.float32, (dim,), index), _arg(wk, "wk", torch.float32, (dim,), index),
                   pc, ps, pp, sq, sk, table, rot)
    return s, index, (batch, L, hq, hk, dim)


def _norm_options(l2, interleaved):
    return (VM_NORM_L2 if l2 else 0) | (VM_ROPE_INTERLEAVED if interleaved else 0)


def vm_head_norm_rope(q, k=None, wq=None, wk=None, cos=None, sin=None, positions=None, eps=1e-6, l2=False,
                      interleaved=False, q_out=None, k_out=None):
    """Queries and keys normalised per head, scaled by a gain and rotated by
    position, in one launch; returns (q_out, k_out), dense.
    q: [batch, L, hq, dim]; k: [batch, L, hk, dim] or None (fp32 or bf16; slices
    of a common projection row are read in place); wq, wk: [dim] fp32 or None;
    cos, sin: [table, rot / 2] fp32 or None (no rotation); positions: int32
    [batch, L], None = 0 .. L - 1, outside the table = padding (zero output).
    l2=True divides by sqrt(sum x^2 + eps) instead of sqrt(mean x^2 + eps);
    interleaved=True pairs (2i, 2i + 1) instead of (i, i + rot / 2)."""
    p, index, (batch, L, hq, hk, dim) = _head_norm(q, k, wq, wk, cos, sin, positions)
    if q_out is None:
        q_out = torch.empty((batch, L, hq, dim), dtype=q.dtype, device=q.device)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = torch.empty((batch, L, hk, dim), dtype=q.dtype, device=q.device)
    _launch("vm_head_norm_rope", index, p, _arg(q_out, "q_out", q.dtype, (batch, L, hq, dim), index),
            _arg(k_out, "k_out", q.dtype, (batch, L, hk, dim), index), batch, L, hq, hk, dim, eps,
            _norm_options(l2, interleaved), _dtype_code(q))
    return q_out, k_out


def vm_head_norm_rope_bwd(dq_out, dk_out, q, k=None, wq=None, wk=None, cos=None, sin=None, positions=None, eps=1e-6,
                          l2=False, interleaved=False):
    """Gradients of sum(dq_out * q_out) + sum(dk_out * k_out) of
    vm_head_norm_rope: (dq, dk, dwq, dwk); dq, dk dense in their dtype, dwq and
    dwk fp32 (None without the gain)."""
    p, index, (batch, L, hq, hk, dim) = _head_norm(q, k, wq, wk, cos, sin, positions)
    if (dk_out is None) != (k is None):
        raise ValueError("dk_out comes with k")
    pq = _arg(dq_out, "dq_out", q.dtype, (batch, L, hq, dim), index)
    pk = _arg(dk_out, "dk_out", q.dtype, (batch, L, hk, dim), index)
    make = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=q.device)
    dq = make(q.dtype, batch, L, hq, dim)
    dk = make(q.dtype, batch, L, hk, dim) if k is not None else None
    dwq = make(torch.float32, dim) if wq is not None else None
    dwk = make(torch.float32, dim) if wk is not None and k is not None else None
    ptr = lambda t: t.data_ptr() if t is not None else None
    ws, wp, wn = _workspace(load_library().vm_head_norm_rope_workspace(dim) if dwq is not None or dwk is not None else 0,
                            q.device)
    _launch("vm_head_norm_rope_bwd", index, p, pq, pk, ptr(dq), ptr(dk), ptr(dwq), ptr(dwk), batch, L, hq, hk, dim, eps,
            _norm_options(l2, interleaved), _dtype_code(q), wp, wn)
    return dq, dk, dwq, dwk


def vm_clip_grad_norm(grads, max_norm, out=None):
    """Scale the gradients to at most the Euclidean norm max_norm over all of
    them; returns the norm before (fp32 tensor of no dimensions, on the GPU).
    grads: a list of contiguous fp32 and bf16 tensors on one GPU, scaled in
    place, or into the tensors of the list `out` (of the same dtypes and as many
    elements)."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError("out must hold one tensor for each gradient")
    # a model has hundreds of gradients: every test is one pass of a C function
    # over the list, and only where one fails is the tensor looked for
    T = torch.Tensor
    try:
        index = T.get_device(grads[0])
        sizes, types = list(map(T.numel, grads)), [x.dtype for x in grads]
        codes = [_GRAD_CODES[types[0]]] * len(types) if types.count(types[0]) == len(types) else \
            [_GRAD_CODES[x] for x in types]
        good = index >= 0 and set(map(T.get_device, grads)) == {index} and all(map(T.is_contiguous, grads))
        ins = list(map(T.data_ptr, grads))
        if outs is grads:
            to = ins
        else:
            good = good and set(map(T.get_device, outs)) == {index} and all(map(T.is_contiguous, outs)) and \
                list(map(T.numel, outs)) == sizes and [x.dtype for x in outs] == types
            to = list(map(T.data_ptr, outs))
    except (TypeError, KeyError):
        good = False
    if not good:
        dev = getattr(grads[0], "device", None)
        for i, (x, y) in enumerate(zip(grads, outs)):
            _dev(x, f"grads[{i}]", None, None, dev)
            _dtype_code(x)
            _dev(y, f"out[{i}]", x.dtype, None, dev)
            if x.numel() != y.numel():
                raise ValueError(f"out[{i}] has {y.numel()} elements, expected {x.numel()}")
    table = array.array("q", bytes(32 * len(grads)))
    table[0::4] = first = array.array("q", ins)                # VmGradTensor: four fields of 8 bytes
    table[1::4] = first if to is ins else array.array("q", to)
    table[2::4], table[3::4] = array.array("q", sizes), array.array("q", codes)
    dev = grads[0].device
    norm = torch.empty((), dtype=torch.float32, device=dev)
    ws, wp, wn = _workspace(load_library().vm_clip_grad_workspace(len(grads)), dev)
    _launch("vm_clip_grad_norm", index, ctypes.cast(table.buffer_info()[0], ctypes.POINTER(VmGradTensor)), len(grads),
            max_norm, norm.data_ptr(), wp, wn)
    return norm


_GRAD_CODES = {torch.float32: VM_F32, torch.bfloat16: VM_BF16}


# ------------------------------------------- prompts, single tokens and norms
def _row_tensor(t, name, dtype, shape, index):
    """A tensor [..., dim] whose rows are contiguous and evenly spaced.  Returns
    the address and the C ABI's row stride (0 = dense)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} must be on a GPU device{', cuda:%d' % index if index >= 0 else ''} (got {t.device})")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    strides, shape = t.stride(), tuple(shape)
    if len(shape) == 2 and strides[1] == 1 and strides[0] >= shape[1]:
        return t.data_ptr(), strides[0]
    if len(shape) == 3 and strides[2] == 1 and strides[1] >= shape[2] and strides[0] == shape[1] * strides[1]:
        return t.data_ptr(), strides[1]
    step, rows = 0, 1                            # of one row, and rows so far, from the last axis to the first
    good = strides[-1] == 1 or shape[-1] == 1
    for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if rows == 1:
            step = stride
        elif stride != step * rows:
            good = False
        rows *= size
    if good and (rows == 1 or step >= shape[-1]):
        return t.data_ptr(), step if rows > 1 else 0
    raise ValueError(f"{name} must have contiguous rows, evenly spaced (shape {tuple(shape)}, strides {strides})")


def _out(t, name, like, dtype, shape, index):
    """An output of a call: the caller's tensor, or a new one beside `like` (which was
    checked).  Returns it and its address."""
    if t is None:
        t = like.new_empty(shape) if like.dtype is dtype else torch.empty(shape, dtype=dtype, device=like.device)
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, index)


def _float_arg(t, name, shape, index):
    return None if t is None else _arg(t, name, torch.float32, shape, index)


def _sequences(batch, offsets, slots, fresh, h0, state, index):
    """Returns (VmSequences or None, sequences, kept states)."""
    n, po = batch, None
    if offsets is not None:
        if batch != 1:
            raise ValueError("packed sequences (offsets) take batch 1")
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError("offsets must be an int32 tensor [sequences + 1]")
        n = offsets.shape[0] - 1
        po = _arg(offsets, "offsets", torch.int32, (n + 1,), index)
    kept = n
    if slots is not None:
        some = h0 if h0 is not None else state
        if some is None or some.dim() < 1:
            raise ValueError("slots come with h0 or state [n_slots, ...]")
        kept = some.shape[0]
    elif po is None and fresh is None:
        return None, n, kept
    return VmSequences(po, _arg(slots, "slots", torch.int32, (n,), index), _arg(fresh, "fresh", torch.int32, (n,), index), n,
                       kept), n, kept


def _clear(offsets, new=True):
    """Packed rows in new outputs: what lies behind the last sequence is set to 0."""
    return VM_CLEAR_REST if new and offsets is not None else 0


def _three(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [batch, seqlen, channels] tensor")
    return t


def _conv_weights(w, dim):
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] != dim:
        raise ValueError("w must be a [dim, width] tensor")
    return w.shape[1]


def vm_prompt_conv(x, w, bias=None, silu=True, h0=None, state=None, want_state=False, offsets=None, slots=None, fresh=None,
                   out=None):
    """Depthwise causal convolution over rows of tokens, with SiLU; returns
    (out, state).  x: [batch, L, dim] (fp32 or bf16; a slice of a projection's row
    is read in place); w: [dim, width] fp32, width 2 to 4; bias: [dim] fp32 or None.
    h0: the inputs before each sequence's first token, [n, width - 1, dim] of x's
    dtype, None = 0.  state (the last inputs, may be h0 itself) is None unless
    want_state or a buffer is given.  offsets (int32 [n + 1], batch 1): sequence i is
    tokens offsets[i] .. offsets[i + 1] - 1.  slots (int32 [n]): h0 and state are
    pools [n_slots, ...] and each sequence's lies there (outside: starts from 0, not
    kept; no two alike).  fresh (int32 [n]): nonzero = starts from 0.  Rows behind the
    last sequence are 0 in a new out and stay as they are in the caller's."""
    batch, L, dim = _three(x, "x").shape
    width = _conv_weights(w, dim)
    index, dtype = x.get_device(), x.dtype
    px, xs = _row_tensor(x, "x", dtype, (batch, L, dim), index)
    seq, n, kept = _sequences(batch, offsets, slots, fresh, h0, state, index)
    shape = (kept, width - 1, dim)
    clear = _clear(offsets, out is None)
    out, po = _out(out, "out", x, dtype, (batch, L, dim), index)
    if state is None and want_state:
        if slots is not None:
            raise ValueError("with slots, state is a pool of the caller's")
        state = torch.empty(shape, dtype=dtype, device=x.device)
    _launch("vm_prompt_conv", index, seq, px, xs, _float_arg(w, "w", (dim, width), index),
            _float_arg(bias, "bias", (dim,), index), _arg(h0, "h0", dtype, shape, index),
            _arg(state, "state", dtype, shape, index), po, batch, L, dim, width, int(bool(silu)) | clear,
            _dtype_code(x))
    return out, state


def vm_prompt_conv_bwd(x, w, dout, bias=None, silu=True, h0=None, dstate=None, offsets=None):
    """Gradients of sum(dout * out) + sum(dstate * state) of vm_prompt_conv.
    Returns a dict: x (dense, in its dtype; 0 behind the last sequence), w, bias (fp32,
    with bias) and, when h0 is given, h0."""
    batch, L, dim = _three(x, "x").shape
    width = _conv_weights(w, dim)
    index, dtype = x.get_device(), x.dtype
    px, xs = _row_tensor(x, "x", dtype, (batch, L, dim), index)
    seq, n, _ = _sequences(batch, offsets, None, None, h0, None, index)
    shape = (n, width - 1, dim)
    make = lambda kind, *size: torch.empty(size, dtype=kind, device=x.device)
    d = dict(x=make(dtype, batch, L, dim), w=make(torch.float32, dim, width))
    if bias is not None:
        d["bias"] = make(torch.float32, dim)
    if h0 is not None:
        d["h0"] = make(dtype, *shape)
    grads = VmConvGrad(*(d[k].data_ptr() if k in d else None for k in ("x", "w", "bias", "h0")))
    ws, wp, wn = _workspace(load_library().vm_prompt_conv_workspace(batch, L, n, dim, width, _dtype_code(x),
                                                                    offsets is not None), x.device)
    _launch("vm_prompt_conv_bwd", index, seq, px, xs, _float_arg(w, "w", (dim, width), index),
            _float_arg(bias, "bias", (dim,), index), _arg(h0, "h0", dtype, shape, index),
            _arg(dout, "dout", dtype, (batch, L, dim), index), _arg(dstate, "dstate", dtype, shape, index), grads, batch, L,
            dim, width, int(bool(silu)) | _clear(offsets), _dtype_code(x), wp, wn)
    return d


def vm_token_conv(x, w, state, bias=None, silu=True, slots=None, out=None):
    """One token of that convolution on kept windows; returns out [batch, dim].
    x: [batch, dim] (a slice of a projection's row is read in place); state
    [n_slots, width - 1, dim] of x's dtype is advanced in place.  slots (int32
    [batch]): each row's window (distinct); a row with a slot outside [0, n_slots)
    is idle: zero out, no window touched."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a [batch, dim] tensor")
    batch, dim = x.shape
    width = _conv_weights(w, dim)
    index, dtype = x.get_device(), x.dtype
    px, xs = _row_tensor(x, "x", dtype, (batch, dim), index)
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be a [n_slots, width - 1, dim] tensor")
    n = state.shape[0]
    out, po = _out(out, "out", x, dtype, (batch, dim), index)
    _launch("vm_token_conv", index, px, xs, _float_arg(w, "w", (dim, width), index), _float_arg(bias, "bias", (dim,), index),
            _arg(state, "state", dtype, (n, width - 1, dim), index), _arg(slots, "slots", torch.int32, (batch,), index), po,
            batch, n, dim, width, int(bool(silu)), _dtype_code(x))
    return out


def _scan_rows(u, delta, A, B, C, D, delta_bias, z):
    """Validate the inputs of a scan over rows [..., dim]; returns (VmScanRows, GPU, dim, N)."""
    if not isinstance(u, torch.Tensor):
        raise TypeError("u must be a torch.Tensor")
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [dim, N] tensor")
    lead, dim, N = tuple(u.shape[:-1]), u.shape[-1], A.shape[1]
    index, dtype = u.get_device(), u.dtype
    pu, su = _row_tensor(u, "u", dtype, (*lead, dim), index)
    pd, sd = _row_tensor(delta, "delta", dtype, (*lead, dim), index)
    pb, sb = _row_tensor(B, "B", dtype, (*lead, N), index)
    pc, sc = _row_tensor(C, "C", dtype, (*lead, N), index)
    pz, sz = _row_tensor(z, "z", dtype, (*lead, dim), index) if z is not None else (None, 0)
    return VmScanRows(pu, pd, _float_arg(A, "A", (dim, N), index), pb, pc, _float_arg(D, "D", (dim,), index),
                      _float_arg(delta_bias, "delta_bias", (dim,), index), pz, su, sd, sb, sc, sz), index, dim, N


def vm_prompt_scan(u, delta, A, B, C, D=None, delta_bias=None, z=None, delta_softplus=True, h0=None, state=None,
                   want_state=False, offsets=None, slots=None, fresh=None, out=None):
    """Selective scan over rows of tokens; returns (out, state).  u, delta, z:
    [batch, L, dim]; B, C: [batch, L, N] (fp32 or bf16; slices of a projection's row
    are read in place); A: [dim, N], D, delta_bias: [dim] fp32.  h0, state: [n, dim,
    N] fp32; state (the last states, may be h0 itself) is None unless want_state or a
    buffer is given.  offsets, slots, fresh and what lies behind the last sequence as in
    vm_prompt_conv.  out is dense."""
    batch, L, dim = _three(u, "u").shape
    p, index, dim, N = _scan_rows(u, delta, A, B, C, D, delta_bias, z)
    seq, n, kept = _sequences(batch, offsets, slots, fresh, h0, state, index)
    clear = _clear(offsets, out is None)
    out, po = _out(out, "out", u, u.dtype, (batch, L, dim), index)
    if state is None and want_state:
        if slots is not None:
            raise ValueError("with slots, state is a pool of the caller's")
        state = torch.empty((n, dim, N), dtype=torch.float32, device=u.device)
    ws, wp, wn = _workspace(load_library().vm_prompt_scan_workspace(batch, L, n, dim, N, offsets is not None, 0), u.device)
    _launch("vm_prompt_scan", index, p, seq, _float_arg(h0, "h0", (kept, dim, N), index),
            _float_arg(state, "state", (kept, dim, N), index), po, batch, L, dim, N, _dtype_code(u),
            _options(delta_softplus, False) | clear, wp, wn)
    return out, state


def vm_prompt_scan_bwd(u, delta, A, B, C, dout, D=None, delta_bias=None, z=None, delta_softplus=True, h0=None, dstate=None,
                       offsets=None):
    """Gradients of sum(dout * out) + sum(dstate * state) of vm_prompt_scan.
    Returns a dict: u, delta, B, C and (with z) z, dense in their dtype (0 behind the
    last sequence); A and, where given, D, delta_bias, h0 in fp32."""
    batch, L, dim = _three(u, "u").shape
    p, index, dim, N = _scan_rows(u, delta, A, B, C, D, delta_bias, z)
    seq, n, _ = _sequences(batch, offsets, None, None, h0, None, index)
    make = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=u.device)
    dt, f32 = u.dtype, torch.float32
    d = dict(u=make(dt, batch, L, dim), delta=make(dt, batch, L, dim), A=make(f32, dim, N), B=make(dt, batch, L, N),
             C=make(dt, batch, L, N))
    if D is not None:
        d["D"] = make(f32, dim)
    if delta_bias is not None:
        d["delta_bias"] = make(f32, dim)
    if z is not None:
        d["z"] = make(dt, batch, L, dim)
    if h0 is not None:
        d["h0"] = make(f32, n, dim, N)
    grads = VmRowsGrad(*(d[k].data_ptr() if k in d else None
                         for k in ("u", "delta", "A", "B", "C", "D", "delta_bias", "z", "h0")))
    ws, wp, wn = _workspace(load_library().vm_prompt_scan_workspace(batch, L, n, dim, N, offsets is not None, 1), u.device)
    _launch("vm_prompt_scan_bwd", index, p, seq, _float_arg(h0, "h0", (n, dim, N), index),
            _arg(dout, "dout", dt, (batch, L, dim), index), _float_arg(dstate, "dstate", (n, dim, N), index), grads, batch, L,
            dim, N, _dtype_code(u), _options(delta_softplus, False) | _clear(offsets), wp, wn)
    return d


def vm_token_scan(u, delta, A, B, C, state, D=None, delta_bias=None, z=None, delta_softplus=True, slots=None, out=None):
    """One token of the selective scan on kept states; returns out [batch, dim].
    u, delta, z: [batch, dim]; B, C: [batch, N]; state [n_slots, dim, N] fp32 is
    updated in place.  slots as in vm_token_conv."""
    if not isinstance(u, torch.Tensor) or u.dim() != 2:
        raise ValueError("u must be a [batch, dim] tensor")
    p, index, dim, N = _scan_rows(u, delta, A, B, C, D, delta_bias, z)
    batch = u.shape[0]
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be a [n_slots, dim, N] tensor")
    n = state.shape[0]
    out, po = _out(out, "out", u, u.dtype, (batch, dim), index)
    _launch("vm_token_scan", index, p, _float_arg(state, "state", (n, dim, N), index),
            _arg(slots, "slots", torch.int32, (batch,), index), po, batch, n, dim, N, _dtype_code(u),
            _options(delta_softplus, False))
    return out


def _lead(t, name):
    """Rows and channels of a tensor [..., dim]."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1:
        raise ValueError(f"{name} must be a [..., dim] tensor")
    dim = t.shape[-1]
    return t.numel() // dim if dim else 0, dim


def _residual_type(t, x_dtype):
    return x_dtype if t is None else t.dtype


def vm_norm_before(x, w=None, b=None, residual=None, scale=None, factor=1.0, center=False, eps=1e-5, want_residual=True,
                   y=None, r=None):
    """The norm before a block: r = residual + factor * scale * x, y = norm(r) * w +
    b; returns (y, r).  x: [..., dim] (fp32 or bf16; rows may be slices); residual:
    the same shape, of x's dtype or fp32, or None; w, b, scale: [dim] fp32 or None.
    The norm divides by the root mean square (center=True: after taking the mean
    off).  r (of residual's dtype; may be residual itself) is None unless
    want_residual or a buffer is given."""
    rows, dim = _lead(x, "x")
    index, dtype, shape = x.get_device(), x.dtype, x.shape
    px, xs = _row_tensor(x, "x", dtype, shape, index)
    rtype = _residual_type(residual, _residual_type(r, dtype))
    pres = _arg(residual, "residual", rtype, shape, index)
    y, py = _out(y, "y", x, dtype, shape, index)
    pr = None
    if want_residual or r is not None:
        r, pr = _out(r, "r", x if residual is None else residual, rtype, shape, index)
    p = VmBlockNorm(px, _float_arg(w, "w", (dim,), index), _float_arg(b, "b", (dim,), index),
                    _float_arg(scale, "scale", (dim,), index), None, xs, 0, 0, 0, eps, factor, VM_NORM_CENTER if center else 0)
    _launch("vm_norm_before", index, p, pres, py, pr, rows, dim, _dtype_code(x), _GRAD_CODES.get(rtype, -1))
    return y, r


def vm_norm_before_bwd(dy, r, w=None, b=None, dr=None, x=None, scale=None, factor=1.0, center=False, eps=1e-5):
    """Gradients of sum(dy * y) + sum(dr * r) of vm_norm_before at the residual r
    that it returned.  Returns a dict: residual (r's dtype), x (dy's dtype; the same
    tensor where the two are equal) and, where given, w, b, scale (fp32; scale needs
    x)."""
    rows, dim = _lead(dy, "dy")
    index, dtype, shape = dy.get_device(), dy.dtype, dy.shape
    if not isinstance(r, torch.Tensor):
        raise TypeError("r must be a torch.Tensor")
    if scale is not None and x is None:
        raise ValueError("the gradient of scale needs x")
    rtype = r.dtype
    px, xs = _row_tensor(x, "x", dtype, shape, index) if scale is not None else (None, 0)
    make = lambda kind, size: torch.empty(size, dtype=kind, device=dy.device)
    d = dict(residual=make(rtype, shape))
    same = scale is None and factor == 1.0 and rtype is dtype
    d["x"] = d["residual"] if same else make(dtype, shape)
    for name, t in (("w", w), ("b", b), ("scale", scale)):
        if t is not None:
            d[name] = make(torch.float32, (dim,))
    ptr = lambda name: d[name].data_ptr() if name in d else None
    grads = VmNormGrad(None if same else ptr("x"), ptr("residual"), None, ptr("w"), ptr("b"), ptr("scale"))
    vec = lambda t, name: _float_arg(t, name, (dim,), index)
    p = VmBlockNorm(px, vec(w, "w"), vec(b, "b"), vec(scale, "scale"), None, xs, 0, 0, 0, eps, factor,
                    VM_NORM_CENTER if center else 0)
    some = w is not None or b is not None or scale is not None
    ws, wp, wn = _workspace(load_library().vm_block_norm_workspace(rows, dim, 0) if some else 0, dy.device)
    _launch("vm_norm_before_bwd", index, p, _arg(r, "r", rtype, shape, index), _arg(dy, "dy", dtype, shape, index),
            _arg(dr, "dr", rtype, shape, index), grads, rows, dim, _dtype_code(dy), _GRAD_CODES.get(rtype, -1), wp, wn)
    return d


def _norm_after(x, w, z, group, scale, factor, gate_first, eps):
    rows, dim = _lead(x, "x")
    index, dtype = x.get_device(), x.dtype
    group = dim if group is None else int(group)
    if group < 1 or dim % group:
        raise ValueError(f"group {group} does not divide {dim} channels")
    px, xs = _row_tensor(x, "x", dtype, x.shape, index)
    pz, zs = _row_tensor(z, "z", dtype, x.shape, index) if z is not None else (None, 0)
    gains = dim
    if w is not None:
        if not isinstance(w, torch.Tensor) or w.dim() != 1 or w.shape[0] not in (dim, group):
            raise ValueError(f"w must hold {dim} or {group} gains")
        gains = w.shape[0]
    if gate_first and z is None:
        raise ValueError("gate_first needs z")
    p = VmBlockNorm(px, _float_arg(w, "w", (gains,), index), None, _float_arg(scale, "scale", (dim,), index), pz, xs, zs,
                    gains, group, eps, factor, VM_NORM_GATE_FIRST if gate_first else 0)
    return p, index, rows, dim, group, gains


def vm_norm_after(x, w=None, z=None, group=None, residual=None, scale=None, factor=1.0, gate_first=False, eps=1e-5, out=None):
    """The norm of a block's output, gated and added to the residual; returns
    residual + factor * scale * y, y = norm(x) * w * SiLU(z), or, gate_first, norm(x *
    SiLU(z)) * w.  x, z: [..., dim] (fp32 or bf16; rows may be slices); group:
    channels normed together (None = all); w: [dim] or [group] fp32; scale: [dim]
    fp32; residual: the shape of x, of its dtype or fp32, or None.  out has
    residual's dtype and may be residual itself."""
    p, index, rows, dim, _, _ = _norm_after(x, w, z, group, scale, factor, gate_first, eps)
    rtype = _residual_type(residual, _residual_type(out, x.dtype))
    pres = _arg(residual, "residual", rtype, x.shape, index)
    out, po = _out(out, "out", x if residual is None else residual, rtype, x.shape, index)
    _launch("vm_norm_after", index, p, pres, po, rows, dim, _dtype_code(x), _GRAD_CODES.get(rtype, -1))
    return out


def vm_norm_after_bwd(dout, x, w=None, z=None, group=None, scale=None, factor=1.0, gate_first=False, eps=1e-5):
    """Gradients of sum(dout * out) of vm_norm_after (the residual's is dout itself).
    Returns a dict: x, z (dense, x's dtype) and, where given, w, scale (fp32)."""
    p, index, rows, dim, group, gains = _norm_after(x, w, z, group, scale, factor, gate_first, eps)
    if not isinstance(dout, torch.Tensor):
        raise TypeError("dout must be a torch.Tensor")
    make = lambda kind, size: torch.empty(size, dtype=kind, device=x.device)
    d = dict(x=make(x.dtype, x.shape))
    if z is not None:
        d["z"] = make(x.dtype, x.shape)
    if w is not None:
        d["w"] = make(torch.float32, (gains,))
    if scale is not None:
        d["scale"] = make(torch.float32, (dim,))
    ptr = lambda name: d[name].data_ptr() if name in d else None
    grads = VmNormGrad(ptr("x"), None, ptr("z"), ptr("w"), None, ptr("scale"))
    some = w is not None or scale is not None
    ws, wp, wn = _workspace(load_library().vm_block_norm_workspace(rows, dim, group) if some else 0, x.device)
    _launch("vm_norm_after_bwd", index, p, _arg(dout, "dout", dout.dtype, x.shape, index), grads, rows, dim, _dtype_code(x),
            _GRAD_CODES.get(dout.dtype, -1), wp, wn)
    return d


__all__ = ["vm_selective_scan_fwd", "vm_bidir_scan_fwd", "vm_bidir_scan_fwd_noalloc", "vm_atrous_gather", "vm_atrous_scatter",
           "vm_pool_scan_repeat", "vm_ss2d_scan_fwd", "vm_causal_conv1d_silu",
           "vm_causal_conv1d_silu_bwd", "vm_pool_scan_repeat_bwd", "vm_ss2d_scan_bwd",
           "vm_selective_scan_bwd", "vm_bidir_scan_bwd", "VmScanGrad", "vm_atrous_group_len", "vm_status_string", "vm_version",
           "VmScanDir", "VmError",
           "vm_gated_delta_fwd", "vm_gated_delta_bwd", "vm_gated_delta_step", "vm_head_norm_rope",
           "vm_head_norm_rope_bwd", "vm_clip_grad_norm", "VmDelta", "VmDeltaGrad", "VmHeadNorm", "VmGradTensor",
           "vm_prompt_conv", "vm_prompt_conv_bwd", "vm_token_conv", "vm_prompt_scan", "vm_prompt_scan_bwd", "vm_token_scan",
           "vm_norm_before", "vm_norm_before_bwd", "vm_norm_after", "vm_norm_after_bwd", "VmSequences", "VmConvGrad",
           "VmScanRows", "VmRowsGrad", "VmBlockNorm", "VmNormGrad", "load_library", "LIB_PATH", "EXPORTED"]
