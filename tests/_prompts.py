"""Inputs and comparisons of the prompt and token operators' tests.

Tolerances.  Outputs are compared by the Euclidean norm of their error over that of
the expected values.  fp32 outputs: every value is a sum of at most a few hundred
products with at most 2^-24 each from the inputs' widening, the product and the sum,
decays from v_exp_f32 (1 ulp) with an argument of two roundings: below 40 roundings
of 2^-24 = 2.4e-6 along the longest chain that counts (a state forgets), taken as
F32 = 4e-6.  Sums over tokens of both signs (gradients of parameters) lose up to the
ratio of the terms' size to the sum's, some ten here: SUMS = 4e-5.  bf16 outputs add
one rounding of at most 2^-8 relative to each value: BF16 = 2^-8 + F32.
"""
import numpy as np
import torch

import oracle.prompts as ref

F32, SUMS, BF16 = 4e-6, 4e-5, 2.0 ** -8 + 4e-6
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def dev(t, dtype=torch.float32):
    return None if t is None else t.to(DEV, dtype)


def slices(parts, dtype, strided):
    """The parts [..., dim] on the GPU, dense or cut from a common row with a value more."""
    if not strided:
        return [dev(p, dtype) for p in parts]
    row = torch.cat([*parts, torch.full((*parts[0].shape[:-1], 1), float("nan"))], dim=-1).to(DEV, dtype)
    return list(row.split([*(p.shape[-1] for p in parts), 1], dim=-1))[:-1]


def offsets_of(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)


def off(got, want):
    """Relative error by Euclidean norms."""
    want = np.asarray(want, dtype=np.float64)
    got = host(got) if isinstance(got, torch.Tensor) else np.asarray(got)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.isfinite(got).all(), "non-finite output"
    size = np.sqrt((want * want).sum())
    err = np.sqrt(((got - want) ** 2).sum())
    return err / size if size > 0 else err


def close(got, want, tol, what):
    e = off(got, want)
    print(f"{what}: {e:.2e} (<= {tol:.1e})", flush=True)
    assert e <= tol, f"{what}: {e:.2e} > {tol:.1e}"


def tol_of(t, sums=False):
    return BF16 if t.dtype == torch.bfloat16 else SUMS if sums else F32


class Scan:
    """Inputs of one selective scan over rows: on the GPU (`a`) and, of the same
    values, for the oracle."""

    def __init__(self, seed, batch, seqlen, dim, n, dtype, lens=None, gate=True, D=True, bias=True, strided=False, soft=True):
        g = gen(seed)
        self.dtype, self.soft = DTYPES[dtype], soft
        self.offsets = None if lens is None else offsets_of(lens).to(DEV)
        if lens is not None:
            batch, seqlen = 1, max(seqlen, sum(lens))
        self.n = batch if lens is None else len(lens)
        self.shape = (batch, seqlen, dim, n)
        lead = (batch, seqlen)
        u, z, extra = slices([randn(g, *lead, dim), randn(g, *lead, dim), randn(g, *lead, 3)], self.dtype, strided)
        delta = dev(randn(g, *lead, dim) if soft else 0.2 * randn(g, *lead, dim).abs(), self.dtype)
        _, B, C = slices([randn(g, *lead, 5), randn(g, *lead, n), randn(g, *lead, n)], self.dtype, strided)
        A = dev(-(1 + torch.arange(n)) * torch.exp(0.1 * randn(g, dim, n)))
        self.a = dict(u=u, delta=delta, A=A, B=B, C=C, D=dev(1 + 0.1 * randn(g, dim)) if D else None,
                      # (without softplus a step must be >= 0, or states grow past all bounds)
                      delta_bias=dev(-2 + randn(g, dim) if soft else 0.1 * randn(g, dim).abs()) if bias else None,
                      z=z if gate else None)
        self.h0, self.dstate = dev(randn(g, self.n, dim, n)), dev(randn(g, self.n, dim, n))
        self.dout = dev(randn(g, *lead, dim), self.dtype)

    def ref(self, first=None):
        h = {k: host(v) for k, v in self.a.items()}
        return ref.scan(h["u"], h["delta"], h["A"], h["B"], h["C"], h["D"], h["delta_bias"], h["z"], self.soft, first,
                        self.offsets)

    def ref_grad(self, first=None, dlast=None):
        h = {k: host(v) for k, v in self.a.items()}
        return ref.scan_grad(h["u"], h["delta"], h["A"], h["B"], h["C"], host(self.dout), h["D"], h["delta_bias"], h["z"],
                             self.soft, first, dlast, self.offsets)

    def inside(self, x):
        """Only the tokens of some sequence."""
        return x if self.offsets is None else x[:, : int(self.offsets[-1])]
