"""Calls of the prompt and token operators beyond single ones: many sequences, chunks against whole walks, graphs,
streams, workspaces, repeated calls, bad values, and sizes past 32-bit offsets."""
import numpy as np
import pytest
import torch

import oracle.prompts as ref
import selective_scan_fwd_amd as vm
from _prompts import BF16, DEV, F32, SUMS, Scan, close, dev, gen, host, offsets_of, randn, tol_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if DEV is None:
        pytest.fail("GPU test run without a visible GPU")
    vm.load_library()
    print(f"[case] {request.node.name}", flush=True)


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("count", [64, 65, 300, 4500])
def test_many_sequences(count):
    """Up to 64 sequences are taken by length, more are looked for 64 at a time (4500: in three rounds)."""
    g = gen(count)
    lens = (torch.rand(count, generator=g) ** 3 * (40 if count < 4000 else 4)).int().tolist()
    lens[count // 3] = 0
    lens[7] = 333
    dim, n = (24, 16) if count < 4000 else (8, 2)
    s = Scan(count, 1, sum(lens), dim, n, "f32", lens=lens)
    out, state = vm.vm_prompt_scan(**s.a, h0=s.h0, want_state=True, offsets=s.offsets)
    want, last, _ = s.ref(list(host(s.h0)))
    close(out, want, F32, "out")
    close(state, last, F32, "state")
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate, offsets=s.offsets)
    want = s.ref_grad(list(host(s.h0)), list(host(s.dstate)))
    for k, v in d.items():
        close(v, want[k], SUMS, k)
    x, w = s.a["u"], dev(0.5 * randn(g, dim, 4))
    out, state = vm.vm_prompt_conv(x, w, want_state=True, offsets=s.offsets)
    want, last = ref.conv(host(x), host(w), offsets=s.offsets)
    close(out, want, F32, "conv")
    assert np.array_equal(host(state), last)
    d = vm.vm_prompt_conv_bwd(x, w, s.dout, offsets=s.offsets)
    want = ref.conv_grad(host(x), host(w), host(s.dout), offsets=s.offsets)
    for k, v in d.items():
        close(v, want[k], SUMS, "conv d" + k)


@pytest.mark.parametrize("count", [31, 32])
def test_one_long_sequence_among_many_short_ones(count):
    """Packed sequences of many channels: with 32 of 4096 only the longest is cut, with 31 chunks are shorter; the other
    launches' slots are those of the chunks that they have."""
    lens = [2] * 10 + [430] + [0, 7] + [1] * (count - 13)
    s = Scan(count, 1, sum(lens) + 3, 4096, 2, "f32", lens=lens)
    pool = s.h0.clone()
    out, _ = vm.vm_prompt_scan(**s.a, h0=pool, state=pool, offsets=s.offsets)
    want, last, _ = s.ref(list(host(s.h0)))
    close(s.inside(out), s.inside(want), F32, "out")
    close(pool, last, F32, "state")
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate, offsets=s.offsets)
    want = s.ref_grad(list(host(s.h0)), list(host(s.dstate)))
    for k, v in d.items():
        inside = s.inside if k in ("u", "delta", "B", "C", "z") else (lambda x: x)
        close(inside(v), inside(want[k]), SUMS, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chunks_are_the_whole_walk(dtype):
    """A row of few channels is cut in chunks; beside enough others of its kind it is walked whole."""
    many = 512
    s = Scan(3, 1, 600, 32, 16, dtype)
    lib = vm.load_library()
    assert lib.vm_prompt_scan_workspace(1, 600, 1, 32, 16, 0, 0) > 0
    assert lib.vm_prompt_scan_workspace(many, 600, many, 32, 16, 0, 0) == 0
    wide = {k: v if v is None or k in ("A", "D", "delta_bias") else v.expand(many, -1, -1).contiguous() for k, v in s.a.items()}
    one, h1 = vm.vm_prompt_scan(**s.a, h0=s.h0, want_state=True)
    all_, h2 = vm.vm_prompt_scan(**wide, h0=s.h0.expand(many, -1, -1).contiguous(), want_state=True)
    assert torch.equal(bits(all_[:1]), bits(all_[-1:]))
    # both are within their own rounding of the formula
    close(all_[:1], host(one), 2 * tol_of(one), "out")
    close(h2[:1], host(h1), 2 * F32, "state")


@pytest.mark.parametrize("dim,n", [(2000, 1), (1984, 16)])
def test_more_chunks_than_run_at_once(dim, n):
    """Chunks whose workgroups start when others have ended: every one joins the ends that the first launch left."""
    l = 4097
    s = Scan(dim, 1, l, dim, n, "f32", gate=False)
    a = {k: v.double() if v is not None else None for k, v in s.a.items()}
    h, want = s.h0[0].double(), []
    dt = torch.nn.functional.softplus(a["delta"] + a["delta_bias"])[0]
    for t in range(l):
        h = torch.exp(dt[t][:, None] * a["A"]) * h + (dt[t] * a["u"][0, t])[:, None] * a["B"][0, t]
        want.append((h * a["C"][0, t]).sum(-1) + a["D"] * a["u"][0, t])
    for _ in range(3):
        out, state = vm.vm_prompt_scan(**s.a, h0=s.h0, want_state=True)
        close(out[0], host(torch.stack(want)), F32, "out")
        close(state[0], host(h), F32, "state")


def test_results_repeat_bit_for_bit():
    s = Scan(5, 2, 700, 48, 16, "bf16", strided=True)
    run = lambda: vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate)
    first = run()
    for _ in range(3):
        again = run()
        assert all(torch.equal(bits(first[k]), bits(again[k])) for k in first)
    s = Scan(6, 1, 4000, 1000, 16, "f32")
    first = [t.clone() for t in vm.vm_prompt_scan(**s.a, want_state=True)]
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, vm.vm_prompt_scan(**s.a, want_state=True)))
    g = gen(2)
    x, w, dout = dev(randn(g, 2, 500, 40)), dev(randn(g, 40, 4)), dev(randn(g, 2, 500, 40))
    a, b = (vm.vm_prompt_conv_bwd(x, w, dout) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)
    rows = dev(randn(g, 5000, 96))
    a, b = (vm.vm_norm_before_bwd(rows, rows, w=dev(torch.ones(96))) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_graph_of_a_block():
    """A block (norm, convolution, scan, gated norm) with its gradients in one graph, replayed with new inputs between the
    program's own work, against the eager calls; and a second graph of single tokens on the same states."""
    b, l, dim, n = 2, 300, 64, 16
    g = gen(9)
    x, res = dev(randn(g, b, l, dim), torch.bfloat16), dev(randn(g, b, l, dim))
    w1, w2, cw = dev(1 + 0.1 * randn(g, dim)), dev(1 + 0.1 * randn(g, dim)), dev(0.5 * randn(g, dim, 4))
    s = Scan(9, b, l, dim, n, "bf16")
    rest = {k: v for k, v in s.a.items() if k != "u"}
    states, windows = torch.zeros(b, dim, n, device=DEV), torch.zeros(b, 3, dim, device=DEV, dtype=torch.bfloat16)
    dout = dev(randn(g, b, l, dim))

    def block():
        y, r = vm.vm_norm_before(x, w1, residual=res)
        u, _ = vm.vm_prompt_conv(y, cw, state=windows)
        o, _ = vm.vm_prompt_scan(u, **rest, state=states)
        out = vm.vm_norm_after(o, w2, s.a["z"], residual=r)
        d2 = vm.vm_norm_after_bwd(dout, o, w2, s.a["z"])
        d1 = vm.vm_prompt_scan_bwd(u, **rest, dout=d2["x"])
        dc = vm.vm_prompt_conv_bwd(y, cw, d1["u"])
        d0 = vm.vm_norm_before_bwd(dc["x"], r, w1, dr=dout)
        return [out, d0["x"], d0["w"], d0["residual"], dc["w"], d1["A"], d1["B"], d1["C"], d1["delta"], d2["w"], d2["z"]]

    one = {k: v if v is None or k in ("A", "D", "delta_bias") else v[:, 0].contiguous() for k, v in rest.items()}
    xt = dev(randn(g, b, dim), torch.bfloat16)

    def token():
        u = vm.vm_token_conv(xt, cw, windows)
        return vm.vm_token_scan(u, **one, state=states)

    block(), token()                                   # (warm-up outside)
    torch.cuda.synchronize()
    graph, tgraph = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block()
    with torch.cuda.graph(tgraph):
        tok = token()
    for i in range(4):
        x.copy_(randn(gen(20 + i), b, l, dim).to(torch.bfloat16))
        want = [t.clone() for t in block()]
        twant = token().clone()
        kept = states.clone(), windows.clone()
        states.zero_(), windows.zero_()
        torch.cuda.synchronize()
        graph.replay()
        junk = torch.randn(1 << 20, device=DEV).sum()  # (the program's own work between)
        tgraph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        assert all(torch.equal(bits(a), bits(c)) for a, c in zip(got, want)), i
        assert torch.equal(bits(tok), bits(twant)) and torch.equal(states, kept[0]) and torch.equal(bits(windows), bits(kept[1]))


def test_graph_of_packed_prompts():
    """One graph for every packed batch of a size: lengths, slots and fresh flags are read when it runs."""
    dim, n, pool, most = 64, 16, 9, 700
    g = gen(17)
    s = Scan(17, 1, most, dim, n, "bf16")
    x, cw = dev(randn(g, 1, most, dim), torch.bfloat16), dev(0.5 * randn(g, dim, 4))
    rest = {k: v for k, v in s.a.items() if k != "u"}
    states, windows = dev(randn(g, pool, dim, n)), dev(randn(g, pool, 3, dim), torch.bfloat16)
    first = states.clone(), windows.clone()
    offsets, slots, fresh = (torch.zeros(k, dtype=torch.int32, device=DEV) for k in (6, 5, 5))
    out = torch.empty(1, most, dim, device=DEV, dtype=torch.bfloat16)

    def prompts():
        u, _ = vm.vm_prompt_conv(x, cw, h0=windows, state=windows, offsets=offsets, slots=slots, fresh=fresh)
        vm.vm_prompt_scan(u, **rest, h0=states, state=states, offsets=offsets, slots=slots, fresh=fresh, out=out)
        return u

    def reset():
        states.copy_(first[0]), windows.copy_(first[1]), out.fill_(7.0)

    slots.copy_(torch.arange(5))
    prompts()                                          # (warm-up outside)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prompts()
    for i, lens in enumerate([[700, 0, 0, 0, 0], [1, 650, 3, 0, 46], [100] * 5, [0, 1, 2, 3, 4], [300, 1, 64, 65, 200]]):
        offsets.copy_(offsets_of(lens)), slots.copy_(torch.randperm(pool, generator=g)[:5]), fresh.copy_(torch.arange(5) % 2 == i % 2)
        reset()
        prompts()
        want = out.clone(), states.clone(), windows.clone()
        reset()
        torch.cuda.synchronize()
        graph.replay()
        junk = torch.randn(1 << 20, device=DEV).sum()  # (the program's own work between)
        torch.cuda.synchronize()
        assert torch.isfinite(junk) and (out[0, sum(lens):] == 7.0).all()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip((out, states, windows), want)), lens


def test_row_of_empty_sequences():
    s = Scan(1, 1, 5, 20, 4, "f32", lens=[0, 0])
    out = torch.full((1, 5, 20), 7.0, device=DEV)
    _, state = vm.vm_prompt_scan(**s.a, h0=s.h0, want_state=True, offsets=s.offsets, out=out)
    assert (out == 7.0).all() and torch.equal(state, s.h0)
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate, offsets=s.offsets)
    assert torch.equal(d["h0"], s.dstate) and not any(d[k].any() for k in ("A", "D", "delta_bias"))
    x, w, h0 = s.a["u"], dev(torch.ones(20, 4)), dev(randn(gen(1), 2, 3, 20))
    out.fill_(7.0)
    _, state = vm.vm_prompt_conv(x, w, h0=h0, want_state=True, offsets=s.offsets, out=out)
    assert (out == 7.0).all() and torch.equal(state, h0)
    d = vm.vm_prompt_conv_bwd(x, w, s.dout, h0=h0, dstate=h0, offsets=s.offsets)
    assert torch.equal(d["h0"], h0) and not d["w"].any()


def test_calls_from_threads_on_their_own_streams():
    import threading

    s = Scan(6, 1, 900, 200, 16, "f32")
    want = vm.vm_prompt_scan(**s.a, want_state=True)
    want_d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout)
    torch.cuda.synchronize()
    good = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got, d = vm.vm_prompt_scan(**s.a, want_state=True), vm.vm_prompt_scan_bwd(**s.a, dout=s.dout)
                stream.synchronize()
                good.append(all(torch.equal(x, y) for x, y in zip(got, want)) and all(torch.equal(d[k], want_d[k]) for k in d))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(good) == 60 and all(good)


def test_other_streams():
    s = Scan(4, 1, 2000, 64, 16, "f32")
    want = vm.vm_prompt_scan(**s.a)[0].clone()
    grads = {k: v.clone() for k, v in vm.vm_prompt_scan_bwd(**s.a, dout=s.dout).items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append((vm.vm_prompt_scan(**s.a)[0], vm.vm_prompt_scan_bwd(**s.a, dout=s.dout)))
    torch.cuda.synchronize()
    for o, d in outs:
        assert torch.equal(o, want) and all(torch.equal(d[k], grads[k]) for k in d)


def test_workspace_of_the_stated_size_is_enough():
    """The calls write nothing past their workspace, nor past their outputs."""
    s = Scan(6, 1, 1000, 40, 16, "f32")
    lib = vm.load_library()
    p, index, dim, n = vm._scan_rows(**s.a)
    stream = torch.cuda.current_stream().cuda_stream
    for back in (0, 1):
        size = lib.vm_prompt_scan_workspace(1, 1000, 1, dim, n, 0, back)
        ws = torch.full((size + 4096,), 77, device=DEV, dtype=torch.uint8)
        outs = {k: torch.full((v + 64,), 7.0, device=DEV) for k, v in
                dict(du=40000, ddelta=40000, dA=640, dB=16000, dC=16000, dD=40, ddelta_bias=40, dz=40000, dh0=640).items()}
        if back:
            st = lib.vm_prompt_scan_bwd(p, None, s.h0.data_ptr(), s.dout.data_ptr(), None,
                                        vm.VmRowsGrad(*(outs[k].data_ptr() for k, _ in vm.VmRowsGrad._fields_)), 1, 1000, dim, n,
                                        0, 1, ws.data_ptr(), size, stream)
        else:
            st = lib.vm_prompt_scan(p, None, s.h0.data_ptr(), outs["dh0"].data_ptr(), outs["du"].data_ptr(), 1, 1000, dim, n, 0, 1,
                                    ws.data_ptr(), size, stream)
        torch.cuda.synchronize()
        assert st == 0 and (ws[size:] == 77).all()
        assert all((v[-64:] == 7.0).all() for v in outs.values())


def test_bad_values_stay_where_they_are():
    """NaN and infinities of one sequence's channel reach that channel from there on, and nothing else."""
    lens = [40, 300, 90]
    s = Scan(8, 1, sum(lens), 48, 16, "f32", lens=lens)
    clean, h = vm.vm_prompt_scan(**s.a, want_state=True, offsets=s.offsets)
    bad = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in s.a.items()}
    bad["u"][0, 40 + 100, 5] = float("nan")
    bad["z"][0, 3, 7] = float("inf")
    out, hb = vm.vm_prompt_scan(**bad, want_state=True, offsets=s.offsets)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[0, 140:340, 5] = True
    hit[0, 3, 7] = True
    assert torch.equal(out[~hit], clean[~hit]) and torch.isnan(out[0, 140:340, 5]).all()
    assert torch.isnan(hb[1, 5]).all() and torch.equal(hb[[0, 2]], h[[0, 2]])
    assert torch.equal(hb[1, [i for i in range(48) if i != 5]], h[1, [i for i in range(48) if i != 5]])
    # a decay rate of -inf clears a state at every step, also at the end of a ragged group
    a = dict(s.a, A=s.a["A"].clone())
    a["A"][3] = float("-inf")
    out, hb = vm.vm_prompt_scan(**a, want_state=True, offsets=s.offsets)
    assert torch.isfinite(out).all() and torch.isfinite(hb).all()
    dt = torch.nn.functional.softplus(a["delta"][0, lens[0] - 1, 3].double() + a["delta_bias"][3].double())
    last = dt * a["u"][0, lens[0] - 1, 3].double() * a["B"][0, lens[0] - 1].double()
    close(hb[0, 3], host(last), F32, "cleared")


def test_rounded_once():
    """bf16 outputs are the fp32 result rounded: few lie further than half a step from the 64-bit result."""
    s = Scan(12, 2, 500, 64, 16, "bf16")
    out, _ = vm.vm_prompt_scan(**s.a)
    want = s.ref()[0]
    half = 2.0 ** -8
    far = np.abs(host(out) - want) > np.abs(want) * half * (1 + 1e-3) + 1e-6
    assert far.mean() < 1e-3


def test_a_step_is_a_prompt_of_one_token():
    b, dim, n = 5, 80, 16
    s = Scan(13, b, 1, dim, n, "bf16", strided=True)
    state = s.h0.clone()
    a = {k: v if v is None or k in ("A", "D", "delta_bias") else v[:, 0] for k, v in s.a.items()}
    step = vm.vm_token_scan(**a, state=state)
    out, last = vm.vm_prompt_scan(**s.a, h0=s.h0, want_state=True)
    close(step, host(out[:, 0]), 2 * BF16, "out")
    close(state, host(last), 2 * F32, "state")


def test_past_32_bit_offsets():
    """Rows of a projection of more than 2^31 values (4.3 GB), the last ones against a call on a copy of them."""
    tokens, dim, wide = 70_000, 64, 32_768
    row = torch.zeros(1, tokens, wide, device=DEV, dtype=torch.bfloat16)
    tail = 300
    g = gen(1)
    x = dev(randn(g, 1, tail, 2 * dim + 32), torch.bfloat16)
    row[:, -tail:, -x.shape[2]:] = x
    cut = lambda t: (t[..., -x.shape[2]: -x.shape[2] + dim], t[..., -dim - 32: -32], t[..., -32: -16], t[..., -16:])
    u, z, B, C = cut(row)
    A, w = dev(-torch.ones(dim, 16)), dev(randn(g, dim, 4))
    delta = torch.zeros(1, tokens, dim, device=DEV, dtype=torch.bfloat16)
    offsets = torch.tensor([0, tokens - tail, tokens], device=DEV, dtype=torch.int32)
    out, h = vm.vm_prompt_scan(u, delta, A, B, C, z=z, offsets=offsets, want_state=True)
    conv, _ = vm.vm_prompt_conv(u, w, offsets=offsets)
    n1, _ = vm.vm_norm_before(u)
    n2 = vm.vm_norm_after(u, z=z, group=32)
    us, zs, Bs, Cs = (t.contiguous() for t in cut(row[:, -tail:]))
    sout, sh = vm.vm_prompt_scan(us, delta[:, -tail:].contiguous(), A, Bs, Cs, z=zs, want_state=True)
    close(out[:, -tail:], host(sout), 2 * BF16, "scan")
    close(h[1:], host(sh), 2 * F32, "state")
    assert (out[:, :-tail] == 0).all()
    assert torch.equal(conv[:, -tail:], vm.vm_prompt_conv(us, w)[0])
    assert torch.equal(n1[:, -tail:], vm.vm_norm_before(us)[0])
    assert torch.equal(n2[:, -tail:], vm.vm_norm_after(us, z=zs, group=32))
    # a pool of more than 2^32 bytes, the last slot
    del row, u, z, B, C, out, conv, n1, n2
    slots = 1_100_000
    pool = torch.zeros(slots, dim, 16, device=DEV)
    pool[-1] = 1.0
    one = lambda t: t[:, 0].contiguous()
    where = torch.tensor([slots - 1], device=DEV, dtype=torch.int32)
    y = vm.vm_token_scan(one(us), one(delta[:, -tail:]), A, one(Bs), one(Cs), pool, slots=where)
    _, want = vm.vm_prompt_scan(us[:, :1].contiguous(), delta[:, :1].contiguous(), A, Bs[:, :1].contiguous(),
                                Cs[:, :1].contiguous(), h0=torch.ones(1, dim, 16, device=DEV), want_state=True)
    close(pool[-1:], host(want), 2 * F32, "last slot")
    assert torch.isfinite(y).all() and (pool[:-1] == 0).all()


def test_binding_refuses():
    g = gen(3)
    x, w = dev(randn(g, 2, 6, 8)), dev(randn(g, 8, 4))
    s = Scan(1, 2, 6, 8, 4, "f32")
    state = torch.zeros(2, 8, 4, device=DEV)
    i32 = lambda *v: torch.tensor(v, device=DEV, dtype=torch.int32)
    with pytest.raises(ValueError):
        vm.vm_prompt_conv(x.transpose(1, 2), w)                       # no rows
    with pytest.raises(ValueError):
        vm.vm_prompt_conv(x, w, offsets=i32(0, 6))                    # packed rows in a batch of two
    with pytest.raises(ValueError):
        vm.vm_prompt_conv(x, w, slots=i32(0, 1))                      # slots of nothing
    with pytest.raises(ValueError):
        vm.vm_prompt_conv(x, w, h0=torch.zeros(2, 2, 8, device=DEV))  # a window of 3 is due
    with pytest.raises(TypeError):
        vm.vm_prompt_conv(x, w, bias=torch.zeros(8, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(vm.VmError):
        vm.vm_prompt_conv(x, dev(randn(g, 8, 5)))
    with pytest.raises(TypeError):
        vm.vm_prompt_scan(**dict(s.a, delta=s.a["delta"].bfloat16()))
    with pytest.raises(ValueError):
        vm.vm_prompt_scan(**dict(s.a, B=s.a["B"].transpose(1, 2).contiguous().transpose(1, 2)))
    with pytest.raises(ValueError):
        vm.vm_prompt_scan(**s.a, h0=state[:1])
    with pytest.raises(ValueError):
        vm.vm_prompt_scan(**s.a, slots=i32(0, 1), h0=state, want_state=True)
    with pytest.raises(TypeError):
        vm.vm_prompt_scan(**s.a, slots=i32(0, 1).long(), h0=state, state=state)
    with pytest.raises(vm.VmError):
        vm.vm_prompt_scan(**s.a, out=s.a["u"])
    with pytest.raises(ValueError):
        vm.vm_prompt_scan(**{k: v.cpu() if v is not None else None for k, v in s.a.items()})
    with pytest.raises(ValueError):
        vm.vm_token_scan(**s.a, state=state)                          # rows of more than a token
    with pytest.raises(ValueError):
        vm.vm_norm_after(x, group=3)
    with pytest.raises(ValueError):
        vm.vm_norm_after(x, gate_first=True)
    with pytest.raises(ValueError):
        vm.vm_norm_after(x, w=torch.ones(5, device=DEV))
    with pytest.raises(ValueError):
        vm.vm_norm_before_bwd(x, x, scale=torch.ones(8, device=DEV))
    with pytest.raises(vm.VmError):
        vm.vm_norm_before(x, residual=x.half())
    with pytest.raises(vm.VmError):
        vm.vm_norm_before(x, residual=x.bfloat16())                   # a residual narrower than the rows
    with pytest.raises(ValueError):
        vm.vm_norm_before(x, w=torch.ones(7, device=DEV))
    with pytest.raises(vm.VmError):
        vm.vm_norm_before(torch.zeros(0, 8, device=DEV))              # no rows
