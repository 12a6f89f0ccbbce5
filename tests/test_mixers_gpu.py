"""GPU parity of the matrix-state mixers (gated delta rule, per-head norm with
rotation, gradient clipping) with their 64-bit definitions.

Tolerances, as max |got - ref| over max(|ref|, rms(ref)):
  fp32  4e-5: sums of up to 128 products and a chunk's triangular solve in
        fp32 (2^-24 each, some 100 roundings in sequence at the worst) stay
        near 1e-5; fp32 results of bf16 inputs are computed alike
  bf16  8e-3: one rounding to 8 bits (2^-9 relative to the value, 2^-8 where
        it falls into the coarse half of a binade) on top of that
"""
import math
import sys

import numpy as np
import pytest
import torch

import selective_scan_fwd_amd as vm
from oracle import mixers

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 4e-5, BF16: 8e-3}


def _case(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(autouse=True)
def _need_gpu():
    if DEV is None:
        pytest.fail("GPU test run without a visible GPU")
    vm.load_library()


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def close(got, ref, what, tol=None):
    tol = TOL[got.dtype] if tol is None else tol
    got = host(got)
    assert got.shape == ref.shape, what
    if not ref.size:
        return
    assert np.isfinite(got).all(), what
    rms = math.sqrt((ref * ref).mean())
    err = np.abs(got - ref) / np.maximum(np.maximum(np.abs(ref), rms), 1e-30)
    print(f"{what}: {err.max():.3e}")
    assert err.max() <= tol, (what, float(err.max()))


def rows(parts, strided):
    """Token tensors as slices of one projection row (with some slack), or dense."""
    if not strided:
        return [p.contiguous() for p in parts]
    b, l = parts[0].shape[:2]
    slack = torch.full((b, l, 3), float("nan"), dtype=parts[0].dtype, device=DEV)
    row = torch.cat([slack] + [p.reshape(b, l, -1) for p in parts] + [slack], dim=-1)
    out, at = [], 3
    for p in parts:
        n = p.shape[2] * p.shape[3]
        out.append(row[:, :, at:at + n].unflatten(-1, p.shape[2:]))
        at += n
    return out


def delta_inputs(seed, b, l, hk, hv, dk, dv, dtype, strided=False, decay=1.0, alike=0.3):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    ru = lambda *s: torch.rand(s, generator=g, device=DEV)
    common = rn(b, 1, hk, dk)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    q, k = unit(rn(b, l, hk, dk)), unit(rn(b, l, hk, dk) + alike * common)
    q, k, v = rows([q.to(dtype), k.to(dtype), rn(b, l, hv, dv).to(dtype)], strided)
    return dict(q=q, k=k, v=v, g=-decay * ru(b, l, hv), beta=ru(b, l, hv)), g


# (batch, seqlen, key heads, value heads, key width, value width)
SIZES = [(1, 1, 1, 1, 1, 1), (2, 63, 1, 2, 16, 16), (1, 64, 2, 2, 64, 64), (2, 65, 1, 3, 33, 17),
         (1, 130, 1, 1, 128, 128), (3, 197, 2, 4, 50, 100), (1, 200, 1, 2, 128, 33), (2, 5, 3, 3, 96, 80)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("reverse,strided", [(False, True), (True, False)])
def test_delta_forward_and_gradients(size, dtype, reverse, strided):
    _case(f"delta {size} {dtype} reverse {reverse} strided {strided}")
    b, l, hk, hv, dk, dv = size
    x, g = delta_inputs(sum(size) + reverse, *size, dtype, strided, decay=0.3)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    h0, dstate = rn(b, hv, dk, dv), rn(b, hv, dk, dv)
    dout = rn(b, l, hv, dv).to(dtype)
    ref_in = {n: host(t) for n, t in x.items()}
    scale = 0.3
    out, state = vm.vm_gated_delta_fwd(**x, scale=scale, h0=h0, want_state=True, reverse=reverse)
    ro, rs, _ = mixers.delta(**ref_in, scale=scale, h0=host(h0), reverse=reverse)
    close(out, ro, "out")
    close(state, rs, "state")
    d = vm.vm_gated_delta_bwd(**x, dout=dout, scale=scale, h0=h0, dstate=dstate, reverse=reverse)
    rd = mixers.delta_grad(**ref_in, scale=scale, dout=host(dout), h0=host(h0), dstate=host(dstate), reverse=reverse)
    for n in ("q", "k", "v", "g", "beta", "h0"):
        close(d[n], rd[n], "d" + n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_delta_defaults_without_states(dtype):
    _case(f"delta defaults {dtype}")
    x, g = delta_inputs(9, 2, 70, 2, 2, 32, 48, dtype)
    dout = torch.randn(x["v"].shape, generator=g, device=DEV).to(dtype)
    ref_in = {n: host(t) for n, t in x.items()}
    out, state = vm.vm_gated_delta_fwd(**x)
    assert state is None
    close(out, mixers.delta(**ref_in, scale=32 ** -0.5)[0], "out")
    d = vm.vm_gated_delta_bwd(**x, dout=dout)
    assert "h0" not in d
    rd = mixers.delta_grad(**ref_in, scale=32 ** -0.5, dout=host(dout))
    for n in ("q", "k", "v", "g", "beta"):
        close(d[n], rd[n], "d" + n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("lens", [[0, 1, 64, 0, 65, 3, 128, 0], [200], [1, 1, 1, 1, 1], [63, 129, 2]])
def test_delta_packed_sequences(lens, reverse, dtype):
    _case(f"delta packed {lens} {dtype} reverse {reverse}")
    n, hk, hv, dk, dv = len(lens), 2, 4, 24, 40
    x, g = delta_inputs(11, 1, sum(lens), hk, hv, dk, dv, dtype, strided=True, decay=0.2)
    off = np.concatenate([[0], np.cumsum(lens)])
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    h0, dstate, dout = rn(n, hv, dk, dv), rn(n, hv, dk, dv), rn(*x["v"].shape).to(dtype)
    ref_in = {m: host(t) for m, t in x.items()}
    out, state = vm.vm_gated_delta_fwd(**x, scale=0.5, h0=h0, want_state=True, reverse=reverse, offsets=offsets)
    ro, rs, _ = mixers.delta(**ref_in, scale=0.5, h0=host(h0), reverse=reverse, offsets=off)
    close(out, ro, "out")
    close(state, rs, "state")
    for i, length in enumerate(lens):
        if length == 0:
            assert torch.equal(state[i], h0[i])
    d = vm.vm_gated_delta_bwd(**x, dout=dout, scale=0.5, h0=h0, dstate=dstate, reverse=reverse, offsets=offsets)
    rd = mixers.delta_grad(**ref_in, scale=0.5, dout=host(dout), h0=host(h0), dstate=host(dstate), reverse=reverse,
                           offsets=off)
    for m in ("q", "k", "v", "g", "beta", "h0"):
        close(d[m], rd[m], "d" + m)


# rows of up to 128 in bf16 are loaded by waves of their own, two chunks ahead: one to
# seven chunks, whole and ragged ends, values in pieces of 16 and of 4 bytes
@pytest.mark.parametrize("size", [(1, 449, 1, 2, 128, 128), (2, 321, 2, 2, 96, 36), (1, 128, 1, 1, 72, 8), (3, 192, 1, 1, 128, 62)])
@pytest.mark.parametrize("reverse", [False, True])
def test_delta_wide_keys_over_many_chunks(size, reverse):
    _case(f"delta wide keys {size} reverse {reverse}")
    b, l, hk, hv, dk, dv = size
    x, g = delta_inputs(41, *size, BF16, decay=0.05)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    h0, dstate, dout = rn(b, hv, dk, dv), rn(b, hv, dk, dv), rn(b, l, hv, dv).to(BF16)
    ref_in = {m: host(t) for m, t in x.items()}
    out, state = vm.vm_gated_delta_fwd(**x, scale=0.3, h0=h0, want_state=True, reverse=reverse)
    ro, rs, _ = mixers.delta(**ref_in, scale=0.3, h0=host(h0), reverse=reverse)
    close(out, ro, "out")
    close(state, rs, "state")
    d = vm.vm_gated_delta_bwd(**x, dout=dout, scale=0.3, h0=h0, dstate=dstate, reverse=reverse)
    rd = mixers.delta_grad(**ref_in, scale=0.3, dout=host(dout), h0=host(h0), dstate=host(dstate), reverse=reverse)
    for m in ("q", "k", "v", "g", "beta", "h0"):
        close(d[m], rd[m], "d" + m)


# the number of workgroups decides how many pairs of waves each has: with more heads
# than the card has compute units four (wide keys: two), with a quarter of them two
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(90, 70, 1, 3, 48, 40), (90, 66, 3, 3, 50, 17), (70, 67, 2, 4, 72, 20),
                                  (20, 130, 2, 4, 64, 72), (25, 65, 4, 4, 104, 36)])
def test_delta_many_heads(size, dtype):
    _case(f"delta many heads {size} {dtype}")
    x, g = delta_inputs(43, *size, dtype, decay=0.2)
    dout = torch.randn(x["v"].shape, generator=g, device=DEV).to(dtype)
    ref_in = {m: host(t) for m, t in x.items()}
    out, state = vm.vm_gated_delta_fwd(**x, scale=0.5, want_state=True)
    ro, rs, _ = mixers.delta(**ref_in, scale=0.5)
    close(out, ro, "out")
    close(state, rs, "state")
    d = vm.vm_gated_delta_bwd(**x, dout=dout, scale=0.5)
    rd = mixers.delta_grad(**ref_in, scale=0.5, dout=host(dout))
    for m in ("q", "k", "v", "g", "beta"):
        close(d[m], rd[m], "d" + m)


@pytest.mark.parametrize("reverse", [False, True])
def test_delta_wide_keys_packed(reverse):
    _case(f"delta wide keys packed reverse {reverse}")
    lens, hk, hv, dk, dv = [0, 1, 64, 0, 65, 3, 200, 130, 128, 0], 1, 3, 104, 40
    x, g = delta_inputs(42, 1, sum(lens), hk, hv, dk, dv, BF16, decay=0.1)
    off = np.concatenate([[0], np.cumsum(lens)])
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    h0, dstate, dout = rn(len(lens), hv, dk, dv), rn(len(lens), hv, dk, dv), rn(*x["v"].shape).to(BF16)
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
@pytest.mark.parametrize("reverse", [False, True])
def test_gate_gradient_of_a_first_token_is_zero(dtype, reverse):
    # nothing decays before the first token: its gate's gradient is 0, not a rounding of it
    _case(f"gate gradient of first tokens {dtype} reverse {reverse}")
    for l, zero_state in ((1, False), (1, True), (64, False), (130, True)):
        x, g = delta_inputs(44, 3, l, 2, 4, 64, 48, dtype)
        dout = torch.randn(x["v"].shape, generator=g, device=DEV).to(dtype)
        h0 = torch.zeros(3, 4, 64, 48, device=DEV) if zero_state else None
        d = vm.vm_gated_delta_bwd(**x, dout=dout, h0=h0, reverse=reverse)
        assert (d["g"][:, l - 1 if reverse else 0] == 0).all()
        rd = mixers.delta_grad(**{m: host(t) for m, t in x.items()}, scale=64 ** -0.5, dout=host(dout), reverse=reverse)
        close(d["g"], rd["g"], "dg")
    x, g = delta_inputs(45, 1, 9, 1, 2, 32, 16, dtype)
    offsets = torch.tensor([0, 1, 1, 4, 9], dtype=torch.int32, device=DEV)
    d = vm.vm_gated_delta_bwd(**x, dout=torch.ones_like(x["v"]), offsets=offsets, reverse=reverse)
    assert (d["g"][0, [0, 3, 8] if reverse else [0, 1, 4]] == 0).all()


def test_delta_offsets_outside_the_row_stay_inside():
    # offsets past the tokens are clamped: the first sequence still holds, the rest is empty
    _case("delta clamped offsets")
    x, _ = delta_inputs(12, 1, 70, 1, 1, 16, 16, F32)
    off = torch.tensor([0, 70, 500, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out, state = vm.vm_gated_delta_fwd(**x, scale=1.0, want_state=True, offsets=off)
    ro, rs, _ = mixers.delta(**{m: host(t) for m, t in x.items()}, scale=1.0)
    close(out, ro, "out")
    close(state[:1], rs, "state")
    assert (state[1:] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_delta_equal_keys_full_strength(dtype):
    # the worst-conditioned triangle: every key the same, beta = 1, no decay.
    # Then out_t = scale (q.k) v_t exactly, and no power of the triangle is small.
    _case(f"delta equal keys {dtype}")
    x, _ = delta_inputs(13, 1, 150, 1, 2, 64, 32, dtype)
    k = torch.zeros(64, device=DEV)
    k[5] = 1.0
    x["k"] = k.to(dtype).expand(1, 150, 1, 64).contiguous()
    x["g"].zero_()
    x["beta"].fill_(1.0)
    out, state = vm.vm_gated_delta_fwd(**x, scale=1.0, want_state=True)
    ro, rs, _ = mixers.delta(**{m: host(t) for m, t in x.items()}, scale=1.0)
    close(out, ro, "out")
    close(state, rs, "state")


@pytest.mark.parametrize("low", [-50.0, -1e4, -math.inf])
def test_delta_strong_decay_clears_the_state(low):
    # a token with a decay to (nearly) nothing in the middle of a chunk and on its edges
    _case(f"delta decay {low}")
    x, g = delta_inputs(14, 1, 140, 1, 2, 32, 32, F32, decay=0.1)
    for t in (3, 63, 64, 100):
        x["g"][:, t] = low
    h0 = torch.randn(1, 2, 32, 32, generator=g, device=DEV)
    dout = torch.randn(x["v"].shape, generator=g, device=DEV)
    ref_in = {m: host(t) for m, t in x.items()}
    out, state = vm.vm_gated_delta_fwd(**x, scale=1.0, h0=h0, want_state=True)
    ro, rs, _ = mixers.delta(**ref_in, scale=1.0, h0=host(h0))
    close(out, ro, "out")
    close(state, rs, "state")
    d = vm.vm_gated_delta_bwd(**x, dout=dout, scale=1.0, h0=h0)
    rd = mixers.delta_grad(**ref_in, scale=1.0, dout=host(dout), h0=host(h0))
    for m in ("q", "k", "v", "g", "beta", "h0"):
        close(d[m], rd[m], "d" + m)


def test_delta_state_in_place_and_split_sequence():
    # a sequence in two calls, the state handed on in its own buffer, equals one call
    _case("delta split sequence")
    x, _ = delta_inputs(15, 2, 150, 2, 2, 32, 32, F32, decay=0.1)
    whole, last = vm.vm_gated_delta_fwd(**x, scale=1.0, want_state=True)
    state = torch.zeros_like(last)
    parts = []
    for lo, hi in ((0, 77), (77, 150)):
        part = {m: t[:, lo:hi].contiguous() for m, t in x.items()}
        out, got = vm.vm_gated_delta_fwd(**part, scale=1.0, h0=state, state=state)
        assert got is state
        parts.append(out)
    close(torch.cat(parts, 1), host(whole), "out")
    close(state, host(last), "state")


def test_delta_is_deterministic_and_runs_on_the_current_stream():
    _case("delta side stream")
    x, g = delta_inputs(16, 2, 197, 2, 4, 64, 64, BF16)
    dout = torch.randn(x["v"].shape, generator=g, device=DEV).to(BF16)
    one = vm.vm_gated_delta_bwd(**x, dout=dout)
    out, state = vm.vm_gated_delta_fwd(**x, want_state=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        two = vm.vm_gated_delta_bwd(**x, dout=dout)
        out2, state2 = vm.vm_gated_delta_fwd(**x, want_state=True)
    side.synchronize()
    assert all(torch.equal(one[m], two[m]) for m in one)
    assert torch.equal(out, out2) and torch.equal(state, state2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1), (3, 2, 4, 128, 128), (9, 1, 3, 33, 17), (2, 4, 4, 64, 100), (17, 1, 1, 96, 36)])
def test_step_matches_and_advances(size, dtype):
    _case(f"step {size} {dtype}")
    b, hk, hv, dk, dv = size
    x, g = delta_inputs(17, b, 3, hk, hv, dk, dv, dtype)
    state = torch.randn(b + 2, hv, dk, dv, generator=g, device=DEV)
    kept = state.clone()
    slots = torch.randperm(b + 2, generator=g, device=DEV)[:b].to(torch.int32)
    idle = b // 2 if b > 2 else None
    if idle is not None:
        slots[idle] = -1 if b % 2 else 2 ** 31 - 1
    h0 = torch.stack([kept[s] if 0 <= s < b + 2 else torch.zeros_like(kept[0]) for s in slots.tolist()])
    outs = [vm.vm_gated_delta_step(*(x[m][:, t].contiguous() for m in ("q", "k", "v", "g", "beta")), state, scale=0.4,
                                   slots=slots) for t in range(3)]
    ro, rs, _ = mixers.delta(**{m: host(t) for m, t in x.items()}, scale=0.4, h0=host(h0))
    out = torch.stack(outs, 1)
    live = [i for i in range(b) if i != idle]
    close(out[live], ro[live], "out")
    close(state[slots[live].long()], rs[live], "state")
    if idle is not None:
        assert (out[idle] == 0).all()
    others = [s for s in range(b + 2) if s not in set(slots[live].tolist())]
    assert torch.equal(state[others], kept[others])


def test_step_replays_in_a_graph():
    _case("step in a graph")
    x, g = delta_inputs(18, 4, 1, 2, 4, 64, 64, BF16)
    args = [x[m][:, 0].contiguous() for m in ("q", "k", "v", "g", "beta")]
    start = torch.randn(4, 4, 64, 64, generator=g, device=DEV)
    state, out = start.clone(), torch.empty(4, 4, 64, dtype=BF16, device=DEV)
    vm.vm_gated_delta_step(*args, state, out=out)
    torch.cuda.synchronize()
    state.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vm.vm_gated_delta_step(*args, state, out=out)
    eager = start.clone()
    state.copy_(start)
    for _ in range(4):
        graph.replay()
        want = vm.vm_gated_delta_step(*args, eager)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, eager)


def test_delta_forward_replays_in_a_graph():
    # the binding's workspace comes from torch's allocator, so a capture allocates nothing of its own
    _case("delta forward in a graph")
    x, _ = delta_inputs(19, 2, 130, 2, 4, 64, 64, BF16)
    vm.vm_gated_delta_fwd(**x, want_state=True)
    torch.cuda.synchronize()
    out, state = torch.empty_like(x["v"]), torch.empty(2, 4, 64, 64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vm.vm_gated_delta_fwd(**x, out=out, state=state)
    for k in range(4):
        x["v"].mul_(0.5)
        want, last = vm.vm_gated_delta_fwd(**x, want_state=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, last)


def test_calls_without_a_workspace_use_the_pool():
    _case("delta from the pool")
    import ctypes
    x, g = delta_inputs(20, 1, 100, 1, 2, 32, 32, F32)
    want, _ = vm.vm_gated_delta_fwd(**x, scale=0.5)
    out = torch.empty_like(want)
    p = vm.VmDelta(*(x[m].data_ptr() for m in ("q", "k", "v", "g", "beta")), None, None, 0, 0, 0)
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        out.zero_()
        assert vm.load_library().vm_gated_delta_fwd(ctypes.byref(p), ctypes.c_void_p(out.data_ptr()), None, 0.5, 1, 100, 1,
                                                    1, 2, 32, 32, vm.VM_F32, 0, None, 0, s) == 0
        assert torch.equal(out, want)


# ---------------------------------------------------- norm with rotation
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,l,hq,hk,dim,rot", [(1, 1, 1, 1, 1, 0), (2, 7, 3, 1, 64, 64), (3, 5, 4, 2, 128, 32),
                                                (2, 3, 1, 0, 33, 10), (2, 197, 6, 6, 64, 32), (1, 9, 2, 2, 512, 512),
                                                (1, 300, 5, 3, 80, 40), (2, 4, 2, 2, 66, 66), (1, 5, 2, 1, 257, 256)])
@pytest.mark.parametrize("l2,interleaved,strided", [(False, False, True), (True, True, False)])
def test_head_norm(b, l, hq, hk, dim, rot, dtype, l2, interleaved, strided):
    _case(f"head norm {b} {l} {hq} {hk} {dim} {rot} {dtype} l2 {l2}")
    g = torch.Generator(device=DEV)
    g.manual_seed(dim + l)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    parts = [(3 * rn(b, l, h, dim)).to(dtype) for h in (hq, hk) if h]
    parts = rows(parts, strided)
    q, k = parts[0], parts[1] if hk else None
    more = dict(eps=1e-5, l2=l2, interleaved=interleaved)
    ref_more = dict(more)
    if rot:
        angle = 6 * torch.rand(l + 3, rot // 2, generator=g, device=DEV)
        more.update(cos=angle.cos(), sin=angle.sin())
        ref_more.update(cos=host(more["cos"]), sin=host(more["sin"]))
        if l > 1:
            pos = torch.randint(-1, l + 4, (b, l), generator=g, device=DEV).to(torch.int32)   # some outside
            more["positions"] = pos
            ref_more["positions"] = pos.cpu().numpy()
    wq, wk = 1 + 0.2 * rn(dim), (1 + 0.2 * rn(dim) if hk else None)
    oq, ok = vm.vm_head_norm_rope(q, k, wq, wk, **more)
    dq_out = rn(b, l, hq, dim).to(dtype)
    dk_out = rn(b, l, hk, dim).to(dtype) if hk else None
    dq, dk, dwq, dwk = vm.vm_head_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, **more)
    for x, w, o, do, dx, dw, name in ((q, wq, oq, dq_out, dq, dwq, "q"), (k, wk, ok, dk_out, dk, dwk, "k")):
        if x is None:
            assert o is None and dx is None and dw is None
            continue
        close(o, mixers.head_norm(host(x), host(w), **ref_more), name)
        rx, rw = mixers.head_norm(host(x), host(w), dy=host(do), **ref_more)
        close(dx, rx, "d" + name)
        close(dw, rw, "dw" + name)
    oq, ok = vm.vm_head_norm_rope(q, k, **more)                     # without gains
    close(oq, mixers.head_norm(host(q), None, **ref_more), "q without gain")
    _, _, dwq, dwk = vm.vm_head_norm_rope_bwd(dq_out, dk_out, q, k, **more)
    assert dwq is None and dwk is None


def test_head_norm_zero_rows():
    # a row of zeros has a finite norm through eps, forward and backward
    _case("head norm zero rows")
    q = torch.zeros(1, 2, 1, 64, device=DEV)
    q[0, 1] = 1.0
    o, _ = vm.vm_head_norm_rope(q, eps=1e-6)
    assert (o[0, 0] == 0).all() and torch.isfinite(o).all()
    dq, _, _, _ = vm.vm_head_norm_rope_bwd(torch.ones_like(q), None, q, eps=1e-6)
    rx, _ = mixers.head_norm(host(q), dy=np.ones(q.shape), eps=1e-6)
    close(dq, rx, "dq")


# ---------------------------------------------------------------- clipping
@pytest.mark.parametrize("count,most", [(1, 1.0), (5, 0.01), (131, 2.0), (300, 1e9)])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(count, most, in_place):
    _case(f"clip {count} {most} in place {in_place}")
    g = torch.Generator(device=DEV)
    g.manual_seed(count)
    sizes = [(1,), (16384,), (16385,), (7, 11), (0,), (40000,), (3, 5, 2)]
    store = torch.empty(400 * 60000, dtype=F32, device=DEV)
    grads, outs, at = [], [], 1                                     # outs at odd places of one buffer
    for i in range(count):
        x = torch.randn(sizes[i % len(sizes)], generator=g, device=DEV).to(BF16 if i % 3 == 1 else F32)
        grads.append(x)
        if x.dtype == F32:
            outs.append(store[at:at + x.numel()].view(x.shape))
            at += x.numel()
        else:
            outs.append(torch.empty_like(x))
    rn, rc = mixers.clip([host(x) for x in grads], most)
    before = [x.clone() for x in grads]
    norm = vm.vm_clip_grad_norm(grads, most, out=None if in_place else outs)
    assert norm.shape == () and norm.dtype == F32
    assert abs(float(norm) - rn) <= 1e-6 * rn                       # (the sums are fp64, the result fp32)
    for x, y, r in zip(before, grads if in_place else outs, rc):
        if x.numel():
            close(y, r, "clipped", tol=4e-3 if x.dtype == BF16 else 1e-6)
    if not in_place:
        assert all(torch.equal(x, y) for x, y in zip(before, grads))


def test_clip_large_and_non_finite_values():
    _case("clip large and non-finite")
    x = torch.full((1000,), 1e30, device=DEV)                       # squares past fp32
    norm = vm.vm_clip_grad_norm([x], 1.0)
    assert abs(float(norm) / (1e30 * math.sqrt(1000.0)) - 1) < 1e-6
    assert abs(float(x.double().norm()) - 1) < 1e-5
    x, y = torch.ones(5, device=DEV), torch.ones(7, device=DEV)
    y[3] = math.inf
    norm = vm.vm_clip_grad_norm([x, y], 1.0)
    assert float(norm) == math.inf
    assert (x == 0).all() and torch.isnan(y[3]) and (y[:3] == 0).all()
    z = torch.tensor([1.0, math.nan], device=DEV)
    norm = vm.vm_clip_grad_norm([z], 1.0)
    assert math.isnan(float(norm)) and torch.isnan(z).all()


def test_clip_norm_only_through_the_c_abi():
    _case("clip norm only")
    import ctypes
    x = torch.randn(5000, device=DEV)
    norm = torch.zeros((), device=DEV)
    arr = (vm.VmGradTensor * 1)(vm.VmGradTensor(x.data_ptr(), None, x.numel(), vm.VM_F32))
    lib = vm.load_library()
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.vm_clip_grad_norm(arr, 1, 1.0, ctypes.c_void_p(norm.data_ptr()), None, 0, s) == 0
    assert abs(float(norm) / float(x.double().norm()) - 1) < 1e-6
    assert lib.vm_clip_grad_norm(None, 0, 1.0, ctypes.c_void_p(norm.data_ptr()), None, 0, s) == 0
    assert float(norm) == 0.0
