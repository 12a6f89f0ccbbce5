"""Gradients of the prompt operators over some thousand tokens, in chunks and walked whole, against a recurrence in
64 bits; and over rows past 32-bit offsets.

Tolerances are those of the short rows.  What length adds: a sum of L terms of either sign in fp32 meets L roundings
of 2^-24 of a partial sum, which grows as sqrt(L): of the final sum's size that is 2^-24 sqrt(L / 2), 2.3e-6 for 3000
tokens and well inside SUMS.  Sums over chunks and rows are formed in fp64."""
import pytest
import torch

import selective_scan_fwd_amd as vm
from _prompts import BF16, DEV, SUMS, Scan, close, dev, gen, host, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if DEV is None:
        pytest.fail("GPU test run without a visible GPU")
    vm.load_library()
    print(f"[case] {request.node.name}", flush=True)


def gradients(s):
    """Of a single row, token by token in 64 bits on the GPU."""
    a = {k: None if v is None else v.double() for k, v in s.a.items()}
    u, delta, z, B, C, dout = (t[0] for t in (a["u"], a["delta"], a["z"], a["B"], a["C"], s.dout.double()))
    A, D, l = a["A"], a["D"], s.shape[1]
    pre = delta + a["delta_bias"]
    dt, slope, gate = torch.nn.functional.softplus(pre), torch.sigmoid(pre), torch.sigmoid(z)
    dy = dout * z * gate
    decay = torch.exp(dt[..., None] * A)
    h = [s.h0[0].double()]
    for t in range(l):
        h.append(decay[t] * h[t] + (dt[t] * u[t])[:, None] * B[t])
    p, g = s.dstate[0].double(), [None] * l
    for t in range(l - 1, -1, -1):
        g[t] = p + dy[t][:, None] * C[t]
        p = decay[t] * g[t]
    h, g = torch.stack(h), torch.stack(g)
    y = torch.bmm(h[1:].contiguous(), C[..., None].contiguous())[..., 0] + D * u
    along = torch.bmm(g, B[..., None].contiguous())[..., 0]
    through = decay * g * h[:-1]
    dd = (u * along + (through * A).sum(-1)) * slope
    return dict(u=dt * along + D * dy, delta=dd, A=(dt[..., None] * through).sum(0), B=((dt * u)[..., None] * g).sum(1),
                C=(dy[..., None] * h[1:]).sum(1), D=(dy * u).sum(0), delta_bias=dd.sum(0),
                z=dout * y * gate * (1 + z * (1 - gate)), h0=p)


def tol(t):
    return SUMS + (BF16 if t.dtype == torch.bfloat16 else 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqlen,dim", [(3001, 64), (4097, 24)])
def test_gradients_of_a_long_row_in_chunks(dtype, seqlen, dim):
    s = Scan(dim, 1, seqlen, dim, 16, dtype)
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate)
    want = gradients(s)
    for k, v in d.items():
        w = want[k] if k in ("A", "D", "delta_bias") else want[k][None]
        close(v, host(w), tol(v), k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_long_rows_walked_whole(dtype):
    """Enough rows of a kind that each is one chunk (the workspace then holds no chunks' ends)."""
    many, seqlen, dim, n = 768, 2001, 64, 16
    tokens, blocks = many * seqlen, dim // 16
    parts = [(tokens // 8 + many + 1) * blocks * 1024, many * dim * n * 4, many * 2 * dim * 4, tokens * 2 * n * 4]
    size = vm.load_library().vm_prompt_scan_workspace(many, seqlen, many, dim, n, 0, 1)
    assert size == sum((x + 255) // 256 * 256 for x in parts)
    s = Scan(31, 1, seqlen, dim, n, dtype)
    wide = lambda t: t.expand(many, -1, -1).contiguous()
    a = {k: v if k in ("A", "D", "delta_bias") else wide(v) for k, v in s.a.items()}
    d = vm.vm_prompt_scan_bwd(**a, dout=wide(s.dout), h0=wide(s.h0), dstate=wide(s.dstate))
    want = gradients(s)
    for k, v in d.items():
        if k in ("A", "D", "delta_bias"):
            close(v.double() / many, host(want[k]), tol(v), k)
        else:
            assert torch.equal(v[0], v[-1])
            close(v[:1], host(want[k][None]), tol(v), k)


def test_gradients_past_32_bit_offsets():
    """Rows of a projection of more than 2^31 values (4.3 GB), the last ones against calls on a copy of them."""
    tokens, dim, wide, tail = 70_000, 64, 32_768, 300
    g = gen(1)
    row = torch.zeros(1, tokens, wide, device=DEV, dtype=torch.bfloat16)
    x = dev(randn(g, 1, tail, 2 * dim + 32), torch.bfloat16)
    row[:, -tail:, -x.shape[2]:] = x
    cut = lambda t: (t[..., -x.shape[2]: -x.shape[2] + dim], t[..., -dim - 32: -32], t[..., -32: -16], t[..., -16:])
    u, z, B, C = cut(row)
    A, w, gain = dev(-torch.ones(dim, 16)), dev(randn(g, dim, 4)), dev(1 + 0.1 * randn(g, dim))
    delta, dout = (torch.zeros(1, tokens, dim, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    dout[:, -tail:] = dev(randn(g, 1, tail, dim), torch.bfloat16)
    offsets = torch.tensor([0, tokens - tail, tokens], device=DEV, dtype=torch.int32)
    got = dict(scan=vm.vm_prompt_scan_bwd(u, delta, A, B, C, dout, z=z, offsets=offsets),
               conv=vm.vm_prompt_conv_bwd(u, w, dout, offsets=offsets),
               after=vm.vm_norm_after_bwd(dout, u, gain, z, group=64),
               before=vm.vm_norm_before_bwd(dout, dout, gain, x=u, scale=gain))
    us, zs, Bs, Cs = (t.contiguous() for t in cut(row[:, -tail:]))
    ds, os = delta[:, -tail:].contiguous(), dout[:, -tail:].contiguous()
    want = dict(scan=vm.vm_prompt_scan_bwd(us, ds, A, Bs, Cs, os, z=zs), conv=vm.vm_prompt_conv_bwd(us, w, os),
                after=vm.vm_norm_after_bwd(os, us, gain, zs, group=64), before=vm.vm_norm_before_bwd(os, os, gain, x=us, scale=gain))
    for op, d in got.items():
        assert set(d) == set(want[op])
        for k, v in d.items():
            if v.dim() == 3:
                assert (v[:, :-tail] == 0).all(), (op, k)
                v = v[:, -tail:]
            close(v, host(want[op][k]), 2 * tol(v), f"{op} {k}")
