"""A gated delta rule mixer trained and then served token by token.

Queries and keys are normalised per head and turned by position
(vm_head_norm_rope), the gated delta rule mixes the tokens
(vm_gated_delta_fwd / _bwd), the gradients of all weights are clipped to one norm
(vm_clip_grad_norm), and a trained layer answers a prompt at once and then single
tokens on its stored states (vm_gated_delta_step).

    python examples/gated_delta_mixer.py [--steps 30]

The layer learns a few rows of random symbols by heart; the losses and the served
tokens' difference from the whole rows' outputs are printed.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_scan_fwd_amd as vm  # noqa: E402


class HeadNormRope(torch.autograd.Function):
    """vm_head_norm_rope and its backward: heads of length one, a gain for the
    queries, positions 0, 1, ... of each row."""

    @staticmethod
    def forward(ctx, q, k, wq, cos, sin):
        ctx.save_for_backward(q, k, wq, cos, sin)
        return vm.vm_head_norm_rope(q, k, wq, None, cos, sin, l2=True)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, wq, cos, sin = ctx.saved_tensors
        d = vm.vm_head_norm_rope_bwd(dq.contiguous(), dk.contiguous(), q, k, wq, None, cos, sin, l2=True)
        return (*d[:3], None, None)


class GatedDelta(torch.autograd.Function):
    """vm_gated_delta_fwd and its backward, from a zero state."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, reverse):
        ctx.save_for_backward(q, k, v, g, beta)
        ctx.reverse = reverse
        return vm.vm_gated_delta_fwd(q, k, v, g, beta, reverse=reverse)[0]

    @staticmethod
    def backward(ctx, dout):
        d = vm.vm_gated_delta_bwd(*ctx.saved_tensors, dout.contiguous(), reverse=ctx.reverse)
        return d["q"], d["k"], d["v"], d["g"], d["beta"], None


def angles(positions, rot, device):
    """Tables [positions, rot/2] of the rotation's cosines and sines."""
    turn = torch.arange(positions, device=device)[:, None] * 1e4 ** (-torch.arange(rot // 2, device=device) / (rot // 2))
    return turn.cos(), turn.sin()


class Mixer:
    """One layer: projections, normed and turned queries and keys, gated delta rule,
    projection back.  Weights are fp32, the mixing is computed in `dtype`."""

    def __init__(self, width, hk, hv, dk, dv, positions, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        make = lambda *s: (torch.randn(*s, device=device, generator=gen) / s[0] ** 0.5).requires_grad_()
        self.hk, self.hv, self.dk, self.dv, self.dtype = hk, hv, dk, dv, dtype
        self.w = dict(q=make(width, hk * dk), k=make(width, hk * dk), v=make(width, hv * dv), g=make(width, hv),
                      beta=make(width, hv), out=make(hv * dv, width),
                      gain=torch.full((dk,), dk ** 0.5, device=device, requires_grad=True))
        self.cos, self.sin = angles(positions, dk // 2, device)

    def inputs(self, x):
        """q, k, v [batch, seqlen, heads, dim], log decays and write strengths."""
        heads = lambda name, n, d: (x @ self.w[name]).to(self.dtype).view(*x.shape[:2], n, d)
        return (heads("q", self.hk, self.dk), heads("k", self.hk, self.dk), heads("v", self.hv, self.dv),
                F.logsigmoid(x @ self.w["g"] + 4), torch.sigmoid(x @ self.w["beta"]))

    def forward(self, x, reverse=False):
        q, k, v, g, beta = self.inputs(x)
        q, k = HeadNormRope.apply(q, k, self.w["gain"], self.cos, self.sin)
        y = GatedDelta.apply(q, k, v, g, beta, reverse)
        return y.reshape(*x.shape[:2], -1).float() @ self.w["out"]

    @torch.no_grad()
    def prompt(self, x):
        """The outputs of whole rows, and the state after them."""
        q, k, v, g, beta = self.inputs(x)
        q, k = vm.vm_head_norm_rope(q, k, self.w["gain"], None, self.cos, self.sin, l2=True)
        y, state = vm.vm_gated_delta_fwd(q, k, v, g, beta, want_state=True)
        return y.reshape(*x.shape[:2], -1).float() @ self.w["out"], state

    @torch.no_grad()
    def token(self, x, states, slots, positions):
        """One token [batch, width] of each row on its stored state, which it
        advances; slots [batch] says which states, positions [batch] where."""
        q, k, v, g, beta = self.inputs(x[:, None])
        q, k = vm.vm_head_norm_rope(q, k, self.w["gain"], None, self.cos, self.sin, positions=positions[:, None], l2=True)
        y = vm.vm_gated_delta_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], states, slots=slots)
        return y.reshape(x.shape[0], -1).float() @ self.w["out"]


def rows_of_symbols(batch, length, width, symbols, seed, device="cuda"):
    """Rows of random symbols: embedded [batch, length, width], and for each token
    the symbol that follows."""
    gen = torch.Generator(device=device).manual_seed(seed)
    s = torch.randint(symbols, (batch, length + 1), device=device, generator=gen)
    table = torch.randn(symbols, width, device=device, generator=torch.Generator(device=device).manual_seed(1))
    return table[s[:, :-1]], s[:, 1:]


def train(steps, batch=8, length=80, width=128, symbols=32, rate=1e-2, most=1.0, dtype=torch.bfloat16):
    """Trains a layer and a read-out with Adam on clipped gradients; returns the
    layer, the losses and the gradients' norms."""
    layer = Mixer(width, hk=2, hv=4, dk=64, dv=48, positions=length, dtype=dtype)
    read = torch.randn(width, symbols, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) / width ** 0.5
    weights = [*layer.w.values(), read.requires_grad_()]
    adam = torch.optim.Adam(weights, lr=rate)
    x, follow = rows_of_symbols(batch, length, width, symbols, 10)
    losses, norms = [], []
    for _ in range(steps):
        logits = layer.forward(x) @ read
        loss = F.cross_entropy(logits.reshape(-1, symbols), follow.reshape(-1))
        grads = [g.contiguous() for g in torch.autograd.grad(loss, weights)]
        norms.append(vm.vm_clip_grad_norm(grads, most))
        for w, g in zip(weights, grads):
            w.grad = g
        adam.step()
        losses.append(loss.detach())
    return layer, torch.stack(losses).tolist(), torch.stack(norms).tolist()


def serve(layer, rows=3, prompt=70, tokens=8, width=128):
    """Prompts at once, then single tokens on states kept in slots; returns the
    largest difference from the whole rows' outputs, relative to their largest."""
    x, _ = rows_of_symbols(rows, prompt + tokens, width, 32, 99)
    whole, _ = layer.prompt(x)
    first, state = layer.prompt(x[:, :prompt])
    states = torch.zeros(2 * rows, *state.shape[1:], device="cuda")
    slots = torch.arange(rows, device="cuda", dtype=torch.int32) * 2 + 1
    states[slots.long()] = state
    out = [first]
    for t in range(prompt, prompt + tokens):
        at = torch.full((rows,), t, device="cuda", dtype=torch.int32)
        out.append(layer.token(x[:, t], states, slots, at)[:, None])
    return float((torch.cat(out, 1) - whole).abs().max() / whole.abs().max())


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--steps", type=int, default=30)
    layer, losses, norms = train(a.parse_args().steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}, gradient norm {norms[0]:.3f} -> {norms[-1]:.3f}")
    print(f"served tokens: {serve(layer):.2e} off the whole rows'")
