"""The prompt and token operators at infinities, partial tiles and rows of no sequence, against their 64-bit
definitions: where those are infinite or no number, so are the outputs, and nowhere else.

Finite values are held to the tolerances of the other tests (their derivation stands beside them); the places of
infinities and of NaN have to be the same."""
import numpy as np
import pytest
import torch

import selective_scan_fwd_amd as vm
from _prompts import BF16, DEV, F32, SUMS, Scan, dev, host

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if DEV is None:
        pytest.fail("GPU test run without a visible GPU")
    vm.load_library()
    print(f"[case] {request.node.name}", flush=True)


def same(got, want, tol, what):
    """Infinities and NaN in the same places; the rest close by Euclidean norms."""
    want, got = np.asarray(want, dtype=np.float64), host(got)
    assert got.shape == want.shape, what
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), f"{what}: {got[odd][:8]} for {want[odd][:8]}"
    assert np.isfinite(got[~odd]).all(), f"{what}: {(~np.isfinite(got[~odd])).sum()} finite values are not"
    size = np.sqrt((want[~odd] ** 2).sum())
    err = np.sqrt(((got[~odd] - want[~odd]) ** 2).sum())
    assert err <= tol * size, f"{what}: {err / size:.2e} > {tol:.1e}"


def tol(t, sums=False):
    return (BF16 if t.dtype == torch.bfloat16 else 0) + (SUMS if sums else F32)


def mild(s, rate=0.25):
    """Positive B and C (infinite states do not cancel in the read-out) and decays that no step takes below 2^-126."""
    s.a = dict(s.a, A=s.a["A"] * rate, B=s.a["B"].abs(), C=s.a["C"].abs())
    return s


def put(s, name, where, value):
    t = s.a[name].clone()
    t[where] = value
    s.a[name] = t


def check_forward(s, **kw):
    out, state = vm.vm_prompt_scan(**s.a, h0=s.h0, want_state=True, offsets=s.offsets)
    with np.errstate(all="ignore"):
        want, last, _ = s.ref(list(host(s.h0)))
    same(out, want, tol(out), "out")
    same(state, last, F32, "state")


def check_backward(s):
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate, offsets=s.offsets)
    with np.errstate(all="ignore"):
        want = s.ref_grad(list(host(s.h0)), list(host(s.dstate)))
    for k, v in d.items():
        same(v, want[k], tol(v, True), "d" + k)


# ----------------------------------------------------- chunks of a long row
def test_an_infinite_state_stays_infinite_over_chunks():
    """A chunk's decays may round to 0 together where no single one does: an infinite state before it stays."""
    assert vm.load_library().vm_prompt_scan_workspace(1, 700, 1, 16, 16, 0, 0) > 0
    s = mild(Scan(21, 1, 700, 16, 16, "f32", bias=False))
    s.a["A"] = torch.full((16, 16), -8.0, device=DEV)
    put(s, "u", (0, 3, 5), INF)
    check_forward(s)
    check_backward(s)
    s = mild(Scan(22, 1, 700, 16, 16, "f32", bias=False))
    s.a["A"] = torch.full((16, 16), -8.0, device=DEV)
    s.dstate[0, 4] = INF
    check_backward(s)


# ------------------------------------------- fewer than 16 states or channels
SHAPES = [(1, 1, 1), (2, 37, 20), (1, 130, 33), (3, 18, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 8, 16])
@pytest.mark.parametrize("batch,seqlen,dim", SHAPES)
def test_infinite_tokens(batch, seqlen, dim, n, dtype):
    """A lane's places past the last state hold 0, whatever a token brings."""
    for name in ("u", "delta"):
        s = mild(Scan(seqlen + n, batch, seqlen, dim, n, dtype, gate=dim != 33))
        put(s, name, (batch - 1, seqlen // 2, dim // 2), INF)
        check_forward(s)
        put(s, "D", slice(None), s.a["D"].abs())
        put(s, "u", (0, 0, 0), -INF)
        check_forward(s)


@pytest.mark.parametrize("n", [1, 5, 8])
def test_infinite_tokens_of_packed_sequences(n):
    lens = [3, 0, 70, 1, 16, 129]
    s = mild(Scan(n, 1, sum(lens), 40, n, "f32", lens=lens))
    put(s, "u", (0, 20, 7), INF)
    put(s, "u", (0, sum(lens) - 129, 39), -INF)
    check_forward(s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 5, 8, 16])
def test_infinite_single_tokens(n, dtype):
    s = mild(Scan(n, 4, 1, 70, n, dtype))
    put(s, "u", (1, 0, 2), INF)
    put(s, "u", (2, 0, 69), -INF)
    put(s, "delta", (3, 0, 5), INF)
    state = s.h0.clone()
    a = {k: v if v is None or k in ("A", "D", "delta_bias") else v[:, 0].contiguous() for k, v in s.a.items()}
    out = vm.vm_token_scan(**a, state=state)
    with np.errstate(all="ignore"):
        want, last, _ = s.ref(list(host(s.h0)))
    same(out, want[:, 0], tol(out), "out")
    same(state, last, F32, "state")


def test_an_infinite_state_stays_infinite_over_chunks_with_one_state():
    s = mild(Scan(23, 1, 700, 16, 1, "f32", bias=False))
    s.a["A"] = torch.full((16, 1), -8.0, device=DEV)
    put(s, "u", (0, 3, 5), INF)
    check_forward(s)


# ------------------------------------------------------ rates and partial tiles
@pytest.mark.parametrize("seqlen", [1, 37, 700])
def test_gradients_at_a_rate_of_minus_infinity(seqlen):
    """Such a rate clears a state at every step; its gradients are those of a rate that does the same and is finite."""
    s = Scan(seqlen, 1, seqlen, 24, 16, "f32")
    put(s, "A", (3, slice(None)), -INF)
    put(s, "A", (20, 5), -INF)
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate)
    s.a["A"] = s.a["A"].clamp(min=-1e30)
    want = s.ref_grad(list(host(s.h0)), list(host(s.dstate)))
    for k, v in d.items():
        same(v, want[k], SUMS, "d" + k)


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("seqlen", [1, 2, 3, 5, 8, 13, 130])
def test_gradients_at_a_bad_last_token(seqlen, value):
    """What the last token brings to the state reaches no gradient that does not read that state, wherever in a tile
    the sequence ends."""
    s = mild(Scan(seqlen, 2, seqlen, 20, 16, "f32"))
    put(s, "u", (1, seqlen - 1, 2), value)
    check_backward(s)
    s = mild(Scan(seqlen, 2, seqlen, 20, 16, "f32"))
    s.dstate[0, 4] = value
    check_backward(s)


def test_gradients_at_bad_last_tokens_of_packed_sequences():
    lens = [6, 9, 4, 0, 2]
    s = mild(Scan(3, 1, sum(lens), 20, 16, "f32", lens=lens))
    for end, ch in ((6, 1), (15, 2), (19, 3)):
        put(s, "u", (0, end - 1, ch), NAN)
    check_backward(s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 5, 8, 16])
@pytest.mark.parametrize("batch,seqlen,dim", [*SHAPES, (1, 7, 1)])
def test_gradients_at_infinite_tokens(batch, seqlen, dim, n, dtype):
    """Places past the last state and lanes past the last channel take no part in any sum."""
    def case():
        return mild(Scan(seqlen + n, batch, seqlen, dim, n, dtype, gate=dim != 33))

    where = (batch - 1, seqlen // 2)
    for name in ("u", "delta"):
        s = case()
        put(s, name, (*where, dim // 2), INF)
        check_backward(s)
    s = case()
    s.dout[(*where, dim // 2)] = -INF
    check_backward(s)
    for name in ("B", "C"):
        s = case()
        put(s, name, (*where, n - 1), INF)
        check_backward(s)


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("n", [1, 5, 8])
@pytest.mark.parametrize("seqlen", [1, 5, 8, 130])
def test_gradients_at_a_bad_last_token_of_few_states(seqlen, n, value):
    s = mild(Scan(seqlen, 2, seqlen, 20, n, "f32"))
    put(s, "u", (1, seqlen - 1, 2), value)
    check_backward(s)
    s = mild(Scan(seqlen, 2, seqlen, 20, n, "f32"))
    s.dstate[0, 4] = value
    check_backward(s)


@pytest.mark.parametrize("n", [1, 16])
def test_gradients_at_infinite_tokens_over_chunks(n):
    s = mild(Scan(23, 1, 700, 20, n, "f32", bias=False))
    put(s, "u", (0, 3, 5), INF)
    put(s, "B", (0, 350, 0), INF)
    check_backward(s)


# ------------------------------------------------ rows behind the last sequence
class Filled:
    """New tensors hold NaN (torch fills uninitialised memory in its deterministic mode)."""

    def __enter__(self):
        torch.use_deterministic_algorithms(True)
        assert torch.isnan(torch.empty(8, device=DEV)).all()

    def __exit__(self, *_):
        torch.use_deterministic_algorithms(False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,lens,rest", [(24, [3, 0, 20], 1), (24, [5], 300), (33, [0, 0], 7), (520, [70, 1, 130], 900),
                                           (64, [1] * 70, 25), (64, [40, 41], 0)])
def test_new_outputs_are_zero_behind_the_last_sequence(dtype, dim, lens, rest):
    total, n = sum(lens), 8
    s = Scan(total, 1, total + rest, dim, n, dtype, lens=lens)
    x, w, bias = s.a["u"], dev(torch.ones(dim, 4)), dev(torch.ones(dim))
    with Filled():
        conv, _ = vm.vm_prompt_conv(x, w, bias, offsets=s.offsets)
        dc = vm.vm_prompt_conv_bwd(x, w, s.dout, bias, offsets=s.offsets)
        out, _ = vm.vm_prompt_scan(**s.a, offsets=s.offsets)
        d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, offsets=s.offsets)
    for name, t in dict(conv=conv, conv_dx=dc["x"], out=out, **{k: d[k] for k in ("u", "delta", "B", "C", "z")}).items():
        assert (t[:, total:] == 0).all(), name
        assert torch.isfinite(t).all(), name


def test_a_packed_row_with_room_left_through_a_block_backward():
    """Sums over all rows of a packed buffer: what lies behind the last sequence adds nothing."""
    import oracle.prompts as ref

    lens, room, dim = [7, 0, 30], 11, 40
    s = Scan(5, 1, sum(lens) + room, dim, 16, "f32", lens=lens)
    x, w = s.a["u"], dev(0.3 * torch.ones(dim, 4))
    gain, r = dev(1 + 0.1 * torch.arange(dim) / dim), s.a["z"].clone()
    with Filled():
        dc = vm.vm_prompt_conv_bwd(x, w, s.dout, offsets=s.offsets)
        d = vm.vm_norm_before_bwd(dc["x"], r, gain)
    want = ref.conv_grad(host(x), host(w), host(s.dout), offsets=s.offsets)["x"][0]
    same(d["w"], ref.norm_before_grad(want, host(r)[0], host(gain))["w"], SUMS, "dw")


def test_graph_of_packed_prompts_with_room_left():
    """Where the sequences end is read when a graph runs: the rest of its own outputs is cleared then."""
    dim, most = 64, 500
    s = Scan(17, 1, most, dim, 16, "bf16", lens=[1] * 4)
    x, w = s.a["u"], dev(torch.ones(dim, 4))
    off = s.offsets.clone()

    def run():
        u, _ = vm.vm_prompt_conv(x, w, offsets=off)
        d = vm.vm_prompt_scan_bwd(**dict(s.a, u=u), dout=s.dout, offsets=off)
        dc = vm.vm_prompt_conv_bwd(x, w, d["u"], offsets=off)
        return [u, vm.vm_prompt_scan(**dict(s.a, u=u), offsets=off)[0], d["u"], d["delta"], d["B"], d["C"], d["z"], dc["x"], dc["w"]]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for ends in ([500, 500, 500, 500], [1, 2, 3, 4], [100, 100, 350, 499], [0, 0, 0, 0]):
        off.copy_(torch.tensor([0] + ends))
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph.replay()
        junk = torch.randn(1 << 20, device=DEV).sum()      # (the program's own work between)
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b) and torch.isfinite(a).all(), (ends, i)
            assert i == 8 or (a[:, ends[-1]:] == 0).all(), (ends, i)


# ------------------------------------------------------------ far apart rows
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_single_tokens_far_apart(dtype):
    """The last token of every row of a long buffer, read in place (rows 2^23 values and more apart)."""
    batch, seqlen, dim, n = 3, 4096, 64, 16
    wide = 2 * dim + 2 * n + (1 << 23) // seqlen
    s = Scan(4, batch, 1, dim, n, dtype)
    row = torch.zeros(batch, seqlen, wide, device=DEV, dtype=s.dtype)
    names, at = ("u", "z", "B", "C"), 0
    a = {k: v if v is None or k in ("A", "D", "delta_bias") else v[:, 0] for k, v in s.a.items()}
    for k in names:
        size = a[k].shape[-1]
        row[:, -1, at: at + size] = a[k]
        a[k] = row[:, -1, at: at + size]
        at += size
    assert a["u"].stride(0) >= 1 << 23
    state = s.h0.clone()
    out = vm.vm_token_scan(**a, state=state)
    want, last, _ = s.ref(list(host(s.h0)))
    same(out, want[:, 0], tol(out), "out")
    same(state, last, F32, "state")


@pytest.mark.parametrize("n", [1, 16])
def test_an_infinite_gradient_stays_infinite_over_chunks(n):
    """As an infinite state does, walking back: a chunk gathers the gradient of the state before it with decays that may
    round to 0 together."""
    s = mild(Scan(24, 1, 700, 16, n, "f32", bias=False))
    s.a["A"] = torch.full((16, n), -8.0, device=DEV)
    for ch in range(8):                      # (at all kinds of places in a chunk)
        s.dout[0, 300 + 9 * ch, ch] = INF if ch % 2 else -INF
    check_backward(s)


def test_a_huge_gradient_decays_over_chunks():
    """Values whose sum overflows, though none is infinite, decay like others."""
    s = Scan(25, 1, 700, 16, 16, "f32", bias=False)
    s.a["A"] = torch.full((16, 16), -8.0, device=DEV)
    s.a.update({k: scale * s.a[k] for k, scale in (("u", 1e-2), ("B", 1e-3), ("C", 1e-3))})
    s.a["z"] = s.a["z"].clamp(-1, 1)
    for ch in range(8):
        at = slice(304 + 8 * ch, 312 + 8 * ch, 4)
        s.dout[0, at, ch] = 3e38
        put(s, "z", (0, at, ch), 1.0)
    check_backward(s)
