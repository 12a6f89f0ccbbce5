"""The prompt and token operators against their 64-bit definitions: the selective
scan and its convolution over dense, packed and single tokens with their gradients."""
import numpy as np
import pytest
import torch

import oracle.prompts as ref
import selective_scan_fwd_amd as vm
from _prompts import BF16, DEV, DTYPES, F32, SUMS, Scan, close, dev, gen, host, offsets_of, randn, slices, tol_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if DEV is None:
        pytest.fail("GPU test run without a visible GPU")
    vm.load_library()
    print(f"[case] {request.node.name}", flush=True)


# ----------------------------------------------------------------- scan
DENSE = [(1, 1, 1, 1), (2, 3, 5, 2), (1, 4, 16, 16), (3, 17, 33, 16), (2, 64, 64, 8), (1, 65, 130, 5), (2, 200, 48, 16),
         (1, 700, 40, 16), (5, 31, 17, 13), (1, 1500, 16, 3)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,seqlen,dim,n", DENSE)
def test_scan_dense(dtype, batch, seqlen, dim, n):
    s = Scan(seqlen + dim, batch, seqlen, dim, n, dtype, strided=dim % 2 == 0, gate=dim != 5, D=dim != 17, bias=dim != 33)
    out, state = vm.vm_prompt_scan(**s.a, h0=s.h0, want_state=True)
    want, last, _ = s.ref(list(host(s.h0)))
    close(out, want, tol_of(out), "out")
    close(state, last, F32, "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [0, 3, 0], [5, 0, 1, 64, 65, 16, 130, 2], [300, 1, 1, 600], [16] * 9])
def test_scan_packed_into_slots(dtype, lens):
    dim, n, pool = 40, 16, len(lens) + 3
    s = Scan(sum(lens), 1, sum(lens) + 7, dim, n, dtype, lens=lens, strided=True)
    g = gen(3)
    kept = randn(g, pool, dim, n)
    slots = torch.randperm(pool, generator=g)[: len(lens)].to(torch.int32)
    if len(lens) > 3:
        slots[2] = pool + 5                      # nowhere: from 0, not kept
    fresh = (torch.arange(len(lens)) % 3 == 1).to(torch.int32)
    state = dev(kept)
    out = torch.full((*s.shape[:2], dim), 7.0, device=DEV, dtype=s.dtype)
    vm.vm_prompt_scan(**s.a, h0=state, state=state, offsets=s.offsets, slots=slots.to(DEV), fresh=fresh.to(DEV), out=out)
    first = ref.first_states(len(lens), host(kept), slots, fresh, (dim, n))
    want, last, _ = s.ref(first)
    close(s.inside(out), s.inside(want), tol_of(out), "out")
    assert (out[:, sum(lens):] == 7.0).all()     # tokens behind the last sequence
    expect = host(kept)
    for i, j in enumerate(slots.tolist()):
        if j < pool:
            expect[j] = last[i]
    close(state, expect, F32, "pool")
    empty = [j for i, j in enumerate(slots.tolist()) if j < pool and lens[i] == 0 and not fresh[i]]
    assert all(torch.equal(state[j].cpu(), kept[j]) for j in empty)


@pytest.mark.parametrize("soft", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,seqlen,dim,n", [(1, 1, 1, 1), (2, 3, 5, 2), (3, 17, 33, 16), (2, 64, 64, 8), (1, 130, 130, 5),
                                                (1, 400, 24, 16), (2, 15, 70, 16)])
def test_scan_gradients(dtype, batch, seqlen, dim, n, soft):
    s = Scan(seqlen + dim, batch, seqlen, dim, n, dtype, strided=dim % 2 == 0, gate=dim != 5, D=dim != 24, bias=dim != 33,
             soft=soft)
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, delta_softplus=soft, h0=s.h0, dstate=s.dstate)
    want = s.ref_grad(list(host(s.h0)), list(host(s.dstate)))
    assert set(d) == {"u", "delta", "A", "B", "C", "h0"} | {k for k in ("D", "delta_bias", "z") if s.a[k] is not None}
    for k, v in d.items():
        close(v, want[k], tol_of(v, sums=k not in ("u", "z")) if v.dtype != torch.bfloat16 else BF16 + SUMS, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [0, 3, 0], [5, 0, 1, 64, 65, 16, 130, 2], [300, 1, 1, 200]])
def test_scan_gradients_packed(dtype, lens):
    dim, n = 40, 16
    s = Scan(sum(lens), 1, sum(lens) + 5, dim, n, dtype, lens=lens)
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate, offsets=s.offsets)
    want = s.ref_grad(list(host(s.h0)), list(host(s.dstate)))
    for k, v in d.items():
        if k in ("u", "delta", "B", "C", "z"):
            v, w = s.inside(v), s.inside(want[k])
        else:
            w = want[k]
        close(v, w, SUMS + (BF16 if v.dtype == torch.bfloat16 else 0), k)


def test_scan_gradients_leave_tokens_of_no_sequence():
    """dB and dC are summed by a launch of their own, which must not write past the last sequence either."""
    import ctypes

    lens = [3, 20]
    s = Scan(1, 1, 40, 20, 4, "f32", lens=lens)
    p, index, dim, n = vm._scan_rows(**s.a)
    seq = vm.VmSequences(s.offsets.data_ptr(), None, None, 2, 2)
    bufs = {k: torch.full(shape, 7.0, device=DEV) for k, shape in
            dict(u=(40, 20), delta=(40, 20), A=(20, 4), B=(40, 4), C=(40, 4), D=(20,), bias=(20,), z=(40, 20), h0=(2, 20, 4)).items()}
    grads = vm.VmRowsGrad(*(t.data_ptr() for t in bufs.values()))
    lib = vm.load_library()
    assert lib.vm_prompt_scan_bwd(p, ctypes.byref(seq), None, s.dout.data_ptr(), None, grads, 1, 40, dim, n, 0, 1, None, 0,
                                  torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for k in ("u", "delta", "B", "C", "z"):
        assert (bufs[k][23:] == 7.0).all(), k
        assert not (bufs[k][:23] == 7.0).any(), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,n", [(1, 1, 1), (3, 50, 16), (9, 64, 8), (20, 130, 5), (2, 70, 13)])
def test_token_scan(dtype, batch, dim, n):
    s = Scan(batch + dim, batch, 1, dim, n, dtype, strided=True, gate=dim != 50, D=dim != 70, bias=dim != 130)
    pool = batch + 2
    kept = randn(gen(2), pool, dim, n)
    slots = torch.randperm(pool, generator=gen(4))[:batch].to(torch.int32)
    if batch > 2:
        slots[1] = -1
    state = dev(kept)
    a = {k: v if v is None or k in ("A", "D", "delta_bias") else v[:, 0] for k, v in s.a.items()}
    out = vm.vm_token_scan(**a, state=state, slots=slots.to(DEV))
    want, last, _ = s.ref(ref.first_states(batch, host(kept), slots, None, (dim, n)))
    want = want[:, 0]
    expect = host(kept)
    for i, j in enumerate(slots.tolist()):
        if j < 0:
            want[i] = 0.0
            assert (out[i] == 0).all()
        else:
            expect[j] = last[i]
    close(out, want, tol_of(out), "out")
    close(state, expect, F32, "pool")


# ---------------------------------------------------------- convolution
def _conv_case(seed, batch, seqlen, dim, width, dtype, strided):
    g = gen(seed)
    x, _ = slices([randn(g, batch, seqlen, dim), randn(g, batch, seqlen, 3)], DTYPES[dtype], strided)
    return x, dev(0.5 * randn(g, dim, width)), dev(0.3 * randn(g, dim))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("batch,seqlen,dim", [(1, 1, 1), (2, 2, 8), (1, 33, 24), (3, 100, 13), (2, 70, 520)])
def test_conv_dense(dtype, width, batch, seqlen, dim):
    act = width != 3
    x, w, bias = _conv_case(seqlen, batch, seqlen, dim, width, dtype, strided=dim == 24)
    bias = None if dim == 13 else bias
    g = gen(9)
    h0, dlast = (dev(randn(g, batch, width - 1, dim), x.dtype) for _ in range(2))
    dout = dev(randn(g, batch, seqlen, dim), x.dtype)
    out, state = vm.vm_prompt_conv(x, w, bias, silu=act, h0=h0, want_state=True)
    want, last = ref.conv(host(x), host(w), host(bias), act, list(host(h0)))
    close(out, want, tol_of(out), "out")
    assert np.array_equal(host(state), last)
    d = vm.vm_prompt_conv_bwd(x, w, dout, bias, silu=act, h0=h0, dstate=dlast)
    want = ref.conv_grad(host(x), host(w), host(dout), host(bias), act, list(host(h0)), list(host(dlast)))
    assert set(d) == {"x", "w", "h0"} | ({"bias"} if bias is not None else set())
    for k, v in d.items():
        close(v, want[k], tol_of(v, sums=k in ("w", "bias")), k)
    # without a window: from zeros
    assert off_zero(vm.vm_prompt_conv(x, w, bias, silu=act)[0], ref.conv(host(x), host(w), host(bias), act)[0])


def off_zero(got, want):
    close(got, want, tol_of(got), "from zeros")
    return True


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [0, 2, 0], [5, 0, 1, 32, 33, 2, 96, 3]])
def test_conv_packed(dtype, lens):
    dim, width, tokens = 24, 4, sum(lens) + 5
    x, w, bias = _conv_case(len(lens), 1, tokens, dim, width, dtype, strided=True)
    offsets = offsets_of(lens)
    g = gen(7)
    pool = len(lens) + 2
    kept = dev(randn(g, pool, width - 1, dim), x.dtype)
    slots = torch.randperm(pool, generator=g)[: len(lens)].to(torch.int32)
    if len(lens) > 3:
        slots[3] = -2
    fresh = (torch.arange(len(lens)) % 2).to(torch.int32)
    state = kept.clone()
    out = torch.full((1, tokens, dim), 7.0, device=DEV, dtype=x.dtype)
    vm.vm_prompt_conv(x, w, bias, h0=state, state=state, offsets=offsets.to(DEV), slots=slots.to(DEV), fresh=fresh.to(DEV),
                      out=out)
    first = ref.first_states(len(lens), host(kept), slots, fresh, (width - 1, dim))
    want, last = ref.conv(host(x), host(w), host(bias), True, first, offsets)
    close(out[:, : sum(lens)], want[:, : sum(lens)], tol_of(out), "out")
    assert (out[:, sum(lens):] == 7.0).all()
    expect = host(kept)
    for i, j in enumerate(slots.tolist()):
        if j >= 0:
            expect[j] = last[i]
    assert np.array_equal(host(state), expect)
    h0, dlast = (dev(randn(g, len(lens), width - 1, dim), x.dtype) for _ in range(2))
    dout = dev(randn(g, 1, tokens, dim), x.dtype)
    d = vm.vm_prompt_conv_bwd(x, w, dout, bias, h0=h0, dstate=dlast, offsets=offsets.to(DEV))
    want = ref.conv_grad(host(x), host(w), host(dout), host(bias), True, list(host(h0)), list(host(dlast)), offsets)
    close(d["x"][:, : sum(lens)], want["x"][:, : sum(lens)], tol_of(d["x"]), "dx")
    for k in ("w", "bias", "h0"):
        close(d[k], want[k], tol_of(d[k], sums=k != "h0"), k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,width", [(1, 1, 2), (3, 40, 4), (9, 13, 3), (20, 264, 4)])
def test_token_conv(dtype, batch, dim, width):
    x, w, bias = _conv_case(batch, batch, 1, dim, width, dtype, strided=True)
    pool = batch + 2
    kept = dev(randn(gen(1), pool, width - 1, dim), x.dtype)
    slots = torch.randperm(pool, generator=gen(2))[:batch].to(torch.int32)
    if batch > 2:
        slots[2] = -1
    state = kept.clone()
    out = vm.vm_token_conv(x[:, 0], w, state, bias, slots=slots.to(DEV))
    first = ref.first_states(batch, host(kept), slots, None, (width - 1, dim))
    want, last = ref.conv(host(x), host(w), host(bias), True, first)
    want, expect = want[:, 0], host(kept)
    for i, j in enumerate(slots.tolist()):
        if j < 0:
            want[i] = 0.0
        else:
            expect[j] = last[i]
    close(out, want, tol_of(out), "out")
    assert np.array_equal(host(state), expect)


# ------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_prompt_then_tokens_are_the_whole_prompt(dtype):
    """Prompts of several lengths at once into slots, then single tokens, against whole sequences."""
    dim, n, width, more, lens = 64, 16, 4, 5, [1, 37, 90]
    dt = DTYPES[dtype]
    g = gen(11)
    total = [x + more for x in lens]
    x, z, delta = (dev(randn(g, 1, sum(total), dim), dt) for _ in range(3))
    B, C = (dev(randn(g, 1, sum(total), n), dt) for _ in range(2))
    w, bias = dev(0.5 * randn(g, dim, width)), dev(0.3 * randn(g, dim))
    par = dict(A=dev(-(1 + torch.arange(n)) * torch.ones(dim, 1)), D=dev(randn(g, dim)), delta_bias=dev(-2 + randn(g, dim)))
    u, _ = vm.vm_prompt_conv(x, w, bias, offsets=offsets_of(total).to(DEV))
    whole, _ = vm.vm_prompt_scan(u, delta, B=B, C=C, z=z, offsets=offsets_of(total).to(DEV), **par)
    starts = offsets_of(total).tolist()
    pick = torch.cat([torch.arange(s, s + n_) for s, n_ in zip(starts, lens)]).to(DEV)
    cut = lambda t: t[:, pick].contiguous()
    slots = torch.tensor([3, 0, 4], device=DEV, dtype=torch.int32)
    windows = torch.full((5, width - 1, dim), float("nan"), device=DEV, dtype=dt)
    states = torch.full((5, dim, n), float("nan"), device=DEV)
    fresh = torch.ones(3, device=DEV, dtype=torch.int32)
    how = dict(offsets=offsets_of(lens).to(DEV), slots=slots, fresh=fresh)
    up, _ = vm.vm_prompt_conv(cut(x), w, bias, h0=windows, state=windows, **how)
    out, _ = vm.vm_prompt_scan(up, cut(delta), B=cut(B), C=cut(C), z=cut(z), h0=states, state=states, **how, **par)
    tol = F32 if dtype == "f32" else 2 ** -7
    close(out, host(whole[:, pick]), tol, "prompts")
    for t in range(more):
        at = torch.tensor([s + n_ + t for s, n_ in zip(starts, lens)], device=DEV)
        one = lambda v: v[0, at].contiguous()
        ut = vm.vm_token_conv(one(x), w, windows, bias, slots=slots)
        yt = vm.vm_token_scan(ut, one(delta), B=one(B), C=one(C), z=one(z), state=states, slots=slots, **par)
        close(yt, host(whole[0, at]), tol, f"token {t}")
    assert torch.isnan(states[1]).all() and torch.isnan(windows[2].float()).all()     # nobody's slots
