"""bf16 outputs of the gated delta rule are its fp32 results rounded once.

Two bounds, both from the definition in 64 bits:
  share of outputs that are not the correctly rounded ones: a result with a
        relative error of e (rms) falls on the other side of a rounding in some
        1000 e of normally spread values (their spacing is 2^-8 to 2^-7 of them,
        and small values among them take the error of the large ones); fp32
        results are 1e-7 to 5e-7 off, so 1e-3 is twice what they may give.  One
        operand of 16 bits alone is 3e-6 off.
  large first states: what the state and the chunk's own values give cancels where
        keys are read back at full strength.  Values of 2000 in fp32, some 30
        roundings of 2^-24 in sequence, are 3.6e-3 off, and 2^-8 the rounding of
        the output: together below the bf16 tolerance of 8e-3.
"""
import numpy as np
import pytest
import torch

import selective_scan_fwd_amd as vm
from oracle import mixers
from test_mixers_gpu import BF16, DEV, TOL, _case, close, delta_inputs, host

pytestmark = pytest.mark.gpu

# (batch, seqlen, key heads, value heads, key width, value width): one, two and four
# pairs of waves to a workgroup, wide and narrow keys, whole pieces and not
SIZES = [(1, 197, 1, 2, 128, 128), (9, 130, 2, 4, 128, 128), (2, 130, 1, 2, 64, 64), (10, 130, 2, 4, 64, 128),
         (40, 66, 2, 4, 64, 96), (2, 130, 1, 2, 50, 33), (3, 65, 1, 3, 100, 40)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("reverse", [False, True])
def test_outputs_are_rounded_once(size, reverse):
    _case(f"delta outputs rounded once {size} reverse {reverse}")
    x, g = delta_inputs(51, *size, BF16, decay=0.1)
    b, _, _, hv, dk, dv = size
    h0 = torch.randn(b, hv, dk, dv, generator=g, device=DEV)
    out, _ = vm.vm_gated_delta_fwd(**x, h0=h0, reverse=reverse)
    ref, _, _ = mixers.delta(**{m: host(t) for m, t in x.items()}, scale=dk ** -0.5, h0=host(h0), reverse=reverse)
    # (to fp32 first: a second rounding that matters in 2^-16 of the values)
    want = torch.from_numpy(ref).to(torch.float32).to(BF16)
    share = float((out.cpu() != want).double().mean())
    print(f"share {share:.2e}")
    assert share < 1e-3


@pytest.mark.parametrize("size", SIZES)
def test_large_first_states_that_cancel(size):
    _case(f"delta large first state {size}")
    b, _, _, hv, dk, dv = size
    x, g = delta_inputs(52, *size, BF16, alike=0.0)
    x["q"] = x["k"].clone()
    x["g"].zero_()
    x["beta"].fill_(1.0)
    h0 = 2000 * torch.randn(b, hv, dk, dv, generator=g, device=DEV)
    out, _ = vm.vm_gated_delta_fwd(**x, scale=1.0, h0=h0)
    ref, _, _ = mixers.delta(**{m: host(t) for m, t in x.items()}, scale=1.0, h0=host(h0))
    close(out, ref, "out", TOL[BF16])


def test_packed_outputs_are_rounded_once():
    _case("delta packed outputs rounded once")
    lens, hk, hv, dk, dv = [70, 1, 0, 200, 64, 133], 2, 4, 64, 100
    x, g = delta_inputs(53, 1, sum(lens), hk, hv, dk, dv, BF16, decay=0.1)
    off = np.concatenate([[0], np.cumsum(lens)])
    h0 = torch.randn(len(lens), hv, dk, dv, generator=g, device=DEV)
    out, _ = vm.vm_gated_delta_fwd(**x, h0=h0, offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
    ref, _, _ = mixers.delta(**{m: host(t) for m, t in x.items()}, scale=dk ** -0.5, h0=host(h0), offsets=off)
    want = torch.from_numpy(ref).to(torch.float32).to(BF16)
    share = float((out.cpu() != want).double().mean())
    print(f"share {share:.2e}")
    assert share < 1e-3
