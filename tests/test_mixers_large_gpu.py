"""Matrix-state mixers past 2^31 elements, and packed rows of many sequences.

The large calls are compared with short ones on their last tokens, which have to
give the same bits: with log decays of -3 a step what lies 128 steps back or ahead
has faded to exactly 0 in fp32 (e^-384), and chunks start at the same tokens.
"""
import numpy as np
import pytest
import torch

import selective_scan_fwd_amd as vm
from oracle import mixers
from test_mixers_gpu import BF16, DEV, F32, _case, close, delta_inputs, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,hv", [(64, 3), (65, 3), (90, 4)])
def test_many_packed_sequences(n, hv):
    """Up to 64 sequences are taken in order of length, more in the order given;
    heads in numbers that leave the last round over the XCDs part empty."""
    _case(f"packed {n} sequences")
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 70, n)
    lens[n // 2] = 140
    x, g = delta_inputs(21, 1, int(lens.sum()), 1, hv, 20, 12, F32, decay=0.2)
    off = np.concatenate([[0], np.cumsum(lens)])
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    dout = torch.randn(x["v"].shape, generator=g, device=DEV)
    ref_in = {m: host(t) for m, t in x.items()}
    out, state = vm.vm_gated_delta_fwd(**x, scale=0.5, want_state=True, offsets=offsets)
    ro, rs, _ = mixers.delta(**ref_in, scale=0.5, offsets=off)
    close(out, ro, "out")
    close(state, rs, "state")
    d = vm.vm_gated_delta_bwd(**x, dout=dout, scale=0.5, offsets=offsets)
    rd = mixers.delta_grad(**ref_in, scale=0.5, dout=host(dout), offsets=off)
    for m in ("q", "k", "v", "g", "beta"):
        close(d[m], rd[m], "d" + m)


def test_delta_past_2_31_elements():
    _case("delta past 2^31 elements")
    hk, hv, dk, dv, last = 1, 16, 8, 128, 256
    l = 2 ** 31 // (hv * dv) + 64
    g = torch.Generator(device=DEV).manual_seed(31)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=BF16)
    x = dict(q=rn(1, l, hk, dk), k=rn(1, l, hk, dk) / 4, v=rn(1, l, hv, dv), beta=torch.rand(1, l, hv, generator=g, device=DEV),
             g=torch.full((1, l, hv), -3.0, device=DEV))
    dout = rn(1, l, hv, dv)
    assert x["v"].numel() > 2 ** 31
    out, state = vm.vm_gated_delta_fwd(**x, want_state=True)
    d = vm.vm_gated_delta_bwd(**x, dout=dout)
    y = {m: t[:, l - last:].contiguous() for m, t in x.items()}
    short, short_state = vm.vm_gated_delta_fwd(**y, want_state=True)
    e = vm.vm_gated_delta_bwd(**y, dout=dout[:, l - last:].contiguous())
    assert torch.equal(out[:, l - 64:], short[:, last - 64:]) and torch.equal(state, short_state)
    for m in d:
        assert torch.equal(d[m][:, l - 64:], e[m][:, last - 64:]), m


def test_head_norm_past_2_31_elements():
    _case("head norm past 2^31 elements")
    hq, dim, last = 16, 128, 33
    l = 2 ** 31 // (hq * dim) + 5
    g = torch.Generator(device=DEV).manual_seed(32)
    q, dq = (torch.randn(1, l, hq, dim, generator=g, device=DEV, dtype=BF16) for _ in range(2))
    table = torch.randn(7, 32, generator=g, device=DEV)
    pos = (torch.arange(l, device=DEV, dtype=torch.int32) % 7)[None]
    y, _ = vm.vm_head_norm_rope(q, cos=table, sin=table, positions=pos)
    back = vm.vm_head_norm_rope_bwd(dq, None, q, cos=table, sin=table, positions=pos)[0]
    tail = lambda t: t[:, l - last:].contiguous()
    assert torch.equal(tail(y), vm.vm_head_norm_rope(tail(q), cos=table, sin=table, positions=tail(pos))[0])
    assert torch.equal(tail(back), vm.vm_head_norm_rope_bwd(tail(dq), None, tail(q), cos=table, sin=table,
                                                            positions=tail(pos))[0])


def test_step_past_2_31_elements():
    _case("step past 2^31 elements")
    hv, dk, dv = 16, 128, 128
    n = 2 ** 31 // (hv * dk * dv) + 1
    states = torch.zeros(n, hv, dk, dv, device=DEV)
    x, g = delta_inputs(33, 2, 1, 4, hv, dk, dv, F32)
    x = {m: t[:, 0].contiguous() for m, t in x.items()}
    small = torch.randn(2, hv, dk, dv, generator=g, device=DEV)
    states[n - 1], states[3] = small[0], small[1]
    out = vm.vm_gated_delta_step(**x, state=states, slots=torch.tensor([n - 1, 3], device=DEV, dtype=torch.int32))
    want = vm.vm_gated_delta_step(**x, state=small)
    assert torch.equal(out, want) and torch.equal(states[n - 1], small[0]) and torch.equal(states[3], small[1])
    assert int(torch.count_nonzero(states[4:8])) == 0


def test_clip_past_2_31_elements():
    _case("clip past 2^31 elements")
    x = torch.zeros(2 ** 31 + 5, dtype=BF16, device=DEV)
    x[5], x[-1] = 4.0, -3.0
    small = torch.zeros(3, dtype=F32, device=DEV)
    norm = vm.vm_clip_grad_norm([x, small], 1.0)
    assert abs(float(norm) - 5.0) < 1e-6
    # 4 / 5 and 3 / 5 rounded to bf16 (the divisor's 1e-6 is below that)
    assert float(x[5]) == float(torch.tensor(0.8, dtype=BF16)) and float(x[-1]) == -float(torch.tensor(0.6, dtype=BF16))
    assert int(torch.count_nonzero(x[6:1 << 20])) == 0
