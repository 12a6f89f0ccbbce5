"""Token rows that are slices of one projection row with every slice 16-byte
aligned, which the kernels read in whole pieces (test_mixers_gpu.py's slices are
not aligned, its dense rows have a stride of their own length); and each of the
norm's options with each other.  Tolerances as there.
"""
import numpy as np
import pytest
import torch

import selective_scan_fwd_amd as vm
from oracle import mixers
from test_mixers_gpu import BF16, DEV, F32, _case, close, delta_inputs, host

pytestmark = pytest.mark.gpu


def aligned_rows(parts):
    """Slices of one projection row with 8 elements of NaN before, between and after them."""
    b, l = parts[0].shape[:2]
    slack = torch.full((b, l, 8), float("nan"), dtype=parts[0].dtype, device=DEV)
    row = torch.cat([slack] + [y for p in parts for y in (p.reshape(b, l, -1), slack)], dim=-1)
    out, at = [], 8
    for p in parts:
        n = p.shape[2] * p.shape[3]
        out.append(row[:, :, at:at + n].unflatten(-1, p.shape[2:]))
        assert not out[-1].is_contiguous() and out[-1].data_ptr() % 16 == 0 and row.shape[2] * row.element_size() % 16 == 0
        at += n + 8
    return out


# one, two and four pairs of waves to a workgroup; values in pieces of 16 and (36) of 4 bytes
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(2, 193, 1, 2, 64, 64), (1, 321, 2, 4, 128, 128), (9, 130, 2, 4, 128, 128),
                                  (2, 130, 1, 2, 96, 72), (10, 70, 2, 4, 64, 128), (40, 67, 2, 4, 64, 80)])
@pytest.mark.parametrize("reverse", [False, True])
def test_delta(size, dtype, reverse):
    _case(f"delta aligned slices {size} {dtype} reverse {reverse}")
    b, l, hk, hv, dk, dv = size
    x, g = delta_inputs(61, *size, dtype, decay=0.1)
    x["q"], x["k"], x["v"] = aligned_rows([x["q"], x["k"], x["v"]])
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    h0, dstate, dout = rn(b, hv, dk, dv), rn(b, hv, dk, dv), rn(b, l, hv, dv).to(dtype)
    ref_in = {m: host(t) for m, t in x.items()}
    out, state = vm.vm_gated_delta_fwd(**x, scale=0.3, h0=h0, want_state=True, reverse=reverse)
    ro, rs, _ = mixers.delta(**ref_in, scale=0.3, h0=host(h0), reverse=reverse)
    close(out, ro, "out")
    close(state, rs, "state")
    d = vm.vm_gated_delta_bwd(**x, dout=dout, scale=0.3, h0=h0, dstate=dstate, reverse=reverse)
    rd = mixers.delta_grad(**ref_in, scale=0.3, dout=host(dout), h0=host(h0), dstate=host(dstate), reverse=reverse)
    for m in ("q", "k", "v", "g", "beta", "h0"):
        close(d[m], rd[m], "d" + m)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 40)])
@pytest.mark.parametrize("reverse", [False, True])
def test_delta_packed(dk, dv, dtype, reverse):
    _case(f"delta packed aligned slices {dk} {dv} {dtype} reverse {reverse}")
    lens, hk, hv = [65, 0, 1, 200, 64, 131], 2, 4
    x, g = delta_inputs(62, 1, sum(lens), hk, hv, dk, dv, dtype, decay=0.1)
    x["q"], x["k"], x["v"] = aligned_rows([x["q"], x["k"], x["v"]])
    off = np.concatenate([[0], np.cumsum(lens)])
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    h0, dstate, dout = rn(len(lens), hv, dk, dv), rn(len(lens), hv, dk, dv), rn(*x["v"].shape).to(dtype)
    ref_in = {m: host(t) for m, t in x.items()}
    out, state = vm.vm_gated_delta_fwd(**x, scale=0.5, h0=h0, want_state=True, reverse=reverse, offsets=offsets)
    ro, rs, _ = mixers.delta(**ref_in, scale=0.5, h0=host(h0), reverse=reverse, offsets=off)
    close(out, ro, "out")
    close(state, rs, "state")
    d = vm.vm_gated_delta_bwd(**x, dout=dout, scale=0.5, h0=h0, dstate=dstate, reverse=reverse, offsets=offsets)
    rd = mixers.delta_grad(**ref_in, scale=0.5, dout=host(dout), h0=host(h0), dstate=host(dstate), reverse=reverse,
                           offsets=off)
    for m in ("q", "k", "v", "g", "beta", "h0"):
        close(d[m], rd[m], "d" + m)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,l,hq,hk,dim,rot", [(2, 7, 3, 1, 64, 64), (3, 5, 4, 2, 128, 32), (8, 1, 16, 4, 128, 128),
                                               (2, 197, 6, 6, 64, 32), (1, 300, 5, 3, 80, 40), (1, 9, 2, 2, 512, 512),
                                               (1, 6, 2, 1, 256, 0), (2, 5, 2, 1, 66, 34)])
@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("strided", [False, True])
def test_head_norm(b, l, hq, hk, dim, rot, dtype, l2, interleaved, strided):
    _case(f"head norm {b} {l} {hq} {hk} {dim} {rot} {dtype} l2 {l2} interleaved {interleaved} strided {strided}")
    g = torch.Generator(device=DEV)
    g.manual_seed(dim + l)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    parts = [(3 * rn(b, l, h, dim)).to(dtype) for h in (hq, hk)]
    if strided and dim % 8 == 0:
        parts = aligned_rows(parts)
    elif strided:
        row = torch.cat([p.reshape(b, l, -1) for p in parts], dim=-1)
        parts = [y.unflatten(-1, (h, dim)) for y, h in zip(row.split([hq * dim, hk * dim], dim=-1), (hq, hk))]
    more = dict(eps=1e-5, l2=l2, interleaved=interleaved)
    ref_more = dict(more)
    if rot:
        angle = 6 * torch.rand(l + 3, rot // 2, generator=g, device=DEV)
        pos = torch.randint(-1, l + 4, (b, l), generator=g, device=DEV).to(torch.int32)
        more.update(cos=angle.cos(), sin=angle.sin(), positions=pos)
        ref_more.update(cos=host(more["cos"]), sin=host(more["sin"]), positions=pos.cpu().numpy())
    w = [1 + 0.2 * rn(dim) for _ in parts]
    dy = [rn(b, l, h, dim).to(dtype) for h in (hq, hk)]
    outs = vm.vm_head_norm_rope(*parts, *w, **more)
    grads = vm.vm_head_norm_rope_bwd(*dy, *parts, *w, **more)
    for i in range(2):
        close(outs[i], mixers.head_norm(host(parts[i]), host(w[i]), **ref_more), "qk"[i])
        rx, rw = mixers.head_norm(host(parts[i]), host(w[i]), dy=host(dy[i]), **ref_more)
        close(grads[i], rx, "d" + "qk"[i])
        close(grads[2 + i], rw, "dw" + "qk"[i])
