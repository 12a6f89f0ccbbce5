"""Cases and plain forms of the gated-delta operators, for timing and comparison.

Three operators that a user of the scans needs when the mixer's state is a
matrix per head instead of a vector per channel:

  norm_rope   per-head normalisation of queries and keys (root mean square or
              Euclidean), optional gains, rotation by position; with gradients
  delta       the gated delta rule  S_t = a_t S_{t-1} + b_t k_t (v_t - a_t
              S_{t-1}^T k_t)^T, o_t = scale S_t^T q_t, a_t = exp(g_t): over whole
              sequences, one token at a time on stored states, and its gradients
  clip        the Euclidean norm over a list of gradients, and the gradients
              scaled to a largest norm

`run` computes them with elementary torch operations in fp32 (own = False) or
through the package's entry points (own = True).  `exact` evaluates the
definitions in 64 bits, token by token where there is a recurrence.
"""
import math

import torch

own = False

CHUNK = 64
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of eight sequences on its way into a step: latency only
        dict(name="norm_rope one token", op="norm_rope", back=False, dtype="bf16", batch=8, seqlen=1, hq=16, hk=4,
             dim=128, rot=128, l2=False, gain=True, interleaved=False, strided=True),
        # a high-resolution image's 4097 tokens, queries and keys cut from one projection
        dict(name="norm_rope 4097 tokens", op="norm_rope", back=False, dtype="bf16", batch=4, seqlen=4097, hq=16, hk=8,
             dim=128, rot=128, l2=False, gain=True, interleaved=False, strided=True),
        # training at 197 tokens: six heads of 64, the first half of each rotated in neighbouring pairs
        dict(name="norm_rope back 197 tokens", op="norm_rope", back=True, dtype="f32", batch=128, seqlen=197, hq=6, hk=6,
             dim=64, rot=32, l2=False, gain=True, interleaved=True, strided=False),
        # the forward pass of the same training step, reversed direction, no states kept
        dict(name="delta 197 tokens reversed", op="delta", dtype="f32", batch=128, seqlen=197, hk=6, hv=6, dk=64, dv=64,
             ragged=0, reverse=True, state=False, strided=False),
        # prefill of long sequences that continue from earlier states and hand theirs on
        dict(name="delta 4097 tokens", op="delta", dtype="bf16", batch=4, seqlen=4097, hk=8, hv=16, dk=128, dv=128,
             ragged=0, reverse=False, state=True, strided=True),
        # forty packed sequences of 1 to some 1500 tokens, narrow keys and odd value width
        dict(name="delta packed", op="delta", dtype="bf16", batch=40, seqlen=1500, hk=4, hv=8, dk=64, dv=100,
             ragged=1, reverse=False, state=True, strided=False),
        # one token of one sequence
        dict(name="step one sequence", op="step", dtype="bf16", batch=1, slots=3, hk=8, hv=16, dk=128, dv=128),
        # one token of a full serving batch on a pool of states, some rows idle
        dict(name="step 128 sequences", op="step", dtype="bf16", batch=128, slots=144, hk=16, hv=32, dk=128, dv=128),
        # gradients at 197 tokens
        dict(name="delta back 197 tokens", op="delta_back", dtype="f32", batch=64, seqlen=197, hk=6, hv=6, dk=64, dv=64,
             reverse=False, strided=False),
        # gradients over a long sequence, two value heads to a key head
        dict(name="delta back 4097 tokens", op="delta_back", dtype="bf16", batch=2, seqlen=4097, hk=8, hv=16, dk=128,
             dv=128, reverse=False, strided=True),
        # every parameter gradient of a 24-block backbone of width 192: many small tensors, odd sizes
        dict(name="clip 24 blocks", op="clip", dtype="f32", blocks=24, width=192, inner=384, mixed=False, most=1.0),
        # few large matrices in bfloat16
        dict(name="clip large", op="clip", dtype="bf16", blocks=6, width=2048, inner=4096, mixed=False, most=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "delta", "delta", "step", "delta_back", "delta_back", "clip"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "clip":
        width = _log(rng, 48, 1500)
        return dict(op=op, dtype=dtype, blocks=_log(rng, 2, 24 if width < 700 else 6), width=width,
                    inner=2 * width + rng.choice([0, 1, 64]), mixed=rng.random() < 0.5, most=rng.choice([0.1, 1.0, 1e6]))
    hk = rng.choice([1, 2, 3, 4, 5, 7])
    group = rng.choice([1, 1, 2, 3])
    if op == "norm_rope":
        dim = rng.choice([32, 64, 80, 96, 128, 128, 66])
        seqlen = _log(rng, 1, 4097)
        batch = max(1, min(_log(rng, 1, 128), 16000 // seqlen))
        return dict(op=op, back=rng.random() < 0.5, dtype=dtype, batch=batch, seqlen=seqlen, hq=hk * group, hk=hk,
                    dim=dim, rot=rng.choice([0, dim // 4 * 2, dim]), l2=rng.random() < 0.5, gain=rng.random() < 0.7,
                    interleaved=rng.random() < 0.5, strided=rng.random() < 0.5)
    dk, dv = rng.choice([32, 64, 128, 128, 96, 50]), rng.choice([32, 64, 128, 128, 80, 33])
    hv = hk * group
    if op == "step":
        batch = max(1, min(_log(rng, 1, 256), 4096 // hv))
        return dict(op=op, dtype=dtype, batch=batch, slots=batch + 1 + rng.randrange(16), hk=hk, hv=hv, dk=dk, dv=dv)
    most = 4 * 4097 * 16 if op == "delta" else 2 * 4097 * 16      # tokens times value heads
    if dtype == "f32":
        most //= 8
    seqlen = _log(rng, 1, 4097)
    batch = max(1, min(_log(rng, 1, 128), most // (seqlen * hv)))
    case = dict(op=op, dtype=dtype, batch=batch, seqlen=seqlen, hk=hk, hv=hv, dk=dk, dv=dv, reverse=rng.random() < 0.3,
                strided=rng.random() < 0.5)
    if op == "delta":
        ragged = int(batch > 1 and rng.random() < 0.3)
        case.update(ragged=ragged, state=rng.random() < 0.5, reverse=case["reverse"] and not ragged)
    return case


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _tokens(parts, strided, dtype):
    """The parts [batch, seqlen, heads, dim] as they come from one projection: slices of a common row, or dense."""
    parts = [p.to(dtype) for p in parts]
    if not strided:
        return [p.contiguous() for p in parts]
    b, l = parts[0].shape[:2]
    sizes = [p.shape[2] * p.shape[3] for p in parts]
    row = torch.cat([p.reshape(b, l, -1) for p in parts], dim=-1)
    return [x.unflatten(-1, (p.shape[2], p.shape[3])) for x, p in zip(row.split(sizes, dim=-1), parts)]


def _all_lengths(case):
    """Ragged lengths: spread over 1 to seqlen by their logarithm, one of them empty."""
    n = case["batch"]
    lens = [round(case["seqlen"] ** ((i + 0.5) / n)) for i in range(n)]
    if n > 2:
        lens[n // 2] = 0
    return lens


def _lengths(case, seed):
    g = torch.Generator()
    g.manual_seed(int(seed))
    lens = _all_lengths(case)
    return [lens[i] for i in torch.randperm(len(lens), generator=g).tolist()]


def _delta_inputs(case, seed):
    g = _gen(seed)
    dtype = DT[case["dtype"]]
    lens = _lengths(case, seed) if case.get("ragged") else None
    b, l = (1, sum(lens)) if lens else (case["batch"], case["seqlen"])
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    common = _randn(g, b, 1, hk, dk)                   # tokens of one image resemble each other
    q = unit(_randn(g, b, l, hk, dk) + 0.3 * common)
    k = unit(_randn(g, b, l, hk, dk) + 0.3 * common)
    v = _randn(g, b, l, hv, dv)
    q, k, v = _tokens([q, k, v], case["strided"], dtype)
    # decay exp(-A dt) with A in [1, 16] and dt about 1e-3 to 1e-1, write strength in (0, 1)
    rate = 1 + 15 * _rand(g, hv)
    bias = torch.log(torch.expm1(torch.exp(math.log(1e-3) + math.log(100.0) * _rand(g, hv))))
    decay = -rate * torch.nn.functional.softplus(_randn(g, b, l, hv) + bias)
    beta = torch.sigmoid(_randn(g, b, l, hv))
    s = dict(q=q, k=k, v=v, g=decay, beta=beta, h0=None, offsets=None, longest=l)
    n = b
    if lens:
        n = len(lens)
        s["offsets"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["longest"] = max(lens)
    if case.get("state"):
        s["h0"] = 0.5 * _randn(g, n, hv, dk, dv)
    if case["op"] == "delta_back":
        s["dout"] = _randn(g, b, l, hv, dv).to(dtype)
    return s


def _step_inputs(case, seed):
    g = _gen(seed)
    dtype = DT[case["dtype"]]
    b, hk, hv, dk, dv = case["batch"], case["hk"], case["hv"], case["dk"], case["dv"]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = unit(_randn(g, b, hk, dk)).to(dtype), unit(_randn(g, b, hk, dk)).to(dtype)
    v = _randn(g, b, hv, dv).to(dtype)
    decay = -0.3 * _rand(g, b, hv)
    beta = torch.sigmoid(_randn(g, b, hv))
    # each sequence's slot in the pool; the last slot is nobody's, every ninth row is idle (-1)
    slots = torch.randperm(case["slots"] - 1, generator=g, device="cuda")[:b].to(torch.int32)
    if b > 8:
        slots[8::9] = -1
    return dict(q=q, k=k, v=v, g=decay, beta=beta, slots=slots, state=_randn(g, case["slots"], hv, dk, dv))


def _norm_inputs(case, seed):
    g = _gen(seed)
    b, l, d, r = case["batch"], case["seqlen"], case["dim"], case["rot"]
    q, k = _tokens([2 * _randn(g, b, l, case["hq"], d), 2 * _randn(g, b, l, case["hk"], d)], case["strided"],
                   DT[case["dtype"]])
    s = dict(q=q, k=k, wq=None, wk=None, cos=None, sin=None, positions=None)
    if case["gain"]:
        s["wq"], s["wk"] = 1 + 0.1 * _randn(g, d), 1 + 0.1 * _randn(g, d)
    if r:
        table = 2 * max(l, 64)
        freq = 10000.0 ** (-torch.arange(r // 2, device="cuda", dtype=torch.float64) * 2 / r)
        angle = torch.arange(table, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        first = torch.randint(0, table - l + 1, (b, 1), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(l, device="cuda")).to(torch.int32)
    if case["back"]:
        s["dq"] = _randn(g, b, l, case["hq"], d).to(q.dtype)
        s["dk"] = _randn(g, b, l, case["hk"], d).to(q.dtype)
    return s


def _clip_shapes(case):
    w, i = case["width"], case["inner"]
    block = [(i, w), (i, w), (w, i), (i, 16), (i,), (i,), (i, 4), (44, i), (i, 12), (w,)]
    return block * case["blocks"] + [(1000, w), (1000,), (1,)]


def _clip_inputs(case, seed):
    g = _gen(seed)
    shapes = _clip_shapes(case)
    grads, flat = [], {}
    types = [DT[case["dtype"]]] * len(shapes)
    if case["mixed"]:                                  # vectors stay in fp32 beside matrices in the case's type
        types = [DT["f32"] if len(s) == 1 else t for s, t in zip(shapes, types)]
    # the clipped gradients go to one flat buffer of each type, which the optimiser reads
    for t in sorted(set(types), key=str):
        n = sum(math.prod(s) for s, u in zip(shapes, types) if u == t)
        flat[str(t)[6:]] = torch.zeros(n, device="cuda", dtype=t)
    at = {k: 0 for k in flat}
    outs = []
    for s, t in zip(shapes, types):
        n, key = math.prod(s), str(t)[6:]
        grads.append((_randn(g, *s) * (0.01 if len(s) == 2 else 0.1)).to(t))
        outs.append(flat[key][at[key]: at[key] + n].view(s))
        at[key] += n
    return dict(grads=grads, outs=outs, flat=flat)


def prepare(case, seed):
    make = dict(norm_rope=_norm_inputs, delta=_delta_inputs, delta_back=_delta_inputs, step=_step_inputs, clip=_clip_inputs)
    state = make[case["op"]](case, seed)
    state["case"] = dict(case)
    return state


# ------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, r, interleaved, back=False):
    """The first r values of each head turned by the position's angles (the other way round for the gradient)."""
    if not r:
        return x
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
    if back:
        sin = -sin
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([y, z], dim=-1).flatten(-2) if interleaved else torch.cat([y, z], dim=-1)
    return torch.cat([y, x[..., r:]], dim=-1)


def _plain_norm(s):
    c = s["case"]
    r = c["rot"]
    cos = s["cos"][s["positions"].long()][:, :, None] if r else None
    sin = s["sin"][s["positions"].long()][:, :, None] if r else None
    over = 1.0 if c["l2"] else 1.0 / c["dim"]

    def forward(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) * over + EPS)
        return _rotate(y if w is None else y * w, cos, sin, r, c["interleaved"]).to(x.dtype)

    def backward(x, w, dy):
        x32 = x.float()
        inv = torch.rsqrt((x32 * x32).sum(-1, keepdim=True) * over + EPS)
        d = _rotate(dy.float(), cos, sin, r, c["interleaved"], back=True)
        n = x32 * inv
        dw = None if w is None else (d * n).sum((0, 1, 2))
        d = d if w is None else d * w
        dx = inv * (d - n * ((d * n).sum(-1, keepdim=True) * over))
        return dx.to(x.dtype), dw

    if not c["back"]:
        return dict(q=forward(s["q"], s["wq"]), k=forward(s["k"], s["wk"]))
    (dq, dwq), (dk, dwk) = backward(s["q"], s["wq"], s["dq"]), backward(s["k"], s["wk"], s["dk"])
    return dict(dq=dq, dk=dk) if s["wq"] is None else dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _unit_lower_inverse(a):
    """(I + a)^-1 of strictly lower triangular a [..., CHUNK, CHUNK], in doubling diagonal blocks."""
    n = a.shape[-1]
    t = torch.ones(a.shape[:-2] + (n, 1, 1), device=a.device, dtype=a.dtype)
    size = 1
    while size < n:
        blocks = a.unflatten(-1, (n // (2 * size), 2 * size)).unflatten(-3, (n // (2 * size), 2 * size))
        low = blocks.diagonal(dim1=-4, dim2=-2).movedim(-1, -3)[..., size:, :size]
        t1, t2 = t[..., 0::2, :, :], t[..., 1::2, :, :]
        top = torch.cat([t1, torch.zeros_like(t1)], dim=-1)
        t = torch.cat([top, torch.cat([-(t2 @ (low @ t1)), t2], dim=-1)], dim=-2)
        size *= 2
    return t[..., 0, :, :]


def _plain_delta(q, k, v, g, beta, h0, scale):
    """Chunked gated delta rule, fp32.  q, k [b, l, hk, dk], v [b, l, hv, dv], g, beta [b, l, hv]; returns out, state."""
    b, l, hv, dv = v.shape
    dk, group = q.shape[-1], hv // q.shape[2]
    pad = -l % CHUNK
    n = (l + pad) // CHUNK
    zero = lambda x: torch.cat([x, x.new_zeros((b, pad) + x.shape[2:])], dim=1) if pad else x  # noqa: E731
    cut = lambda x: zero(x).transpose(1, 2).reshape((b, hv, n, CHUNK) + x.shape[3:])  # noqa: E731
    q, k = cut(q.repeat_interleave(group, dim=2)) * scale, cut(k.repeat_interleave(group, dim=2))
    v, g, beta = cut(v), cut(g), cut(beta)
    total = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=q.device, dtype=torch.bool).tril()
    decay = (total[..., :, None] - total[..., None, :]).masked_fill(~low, -math.inf).exp()
    kt = k.transpose(-1, -2)
    a = (k * beta[..., None]) @ kt * decay
    t = _unit_lower_inverse(a.tril(-1))
    u = t @ (v * beta[..., None])
    w = t @ (k * (beta * total.exp())[..., None])
    p = q @ kt * decay
    q = q * total.exp()[..., None]
    last = total[..., -1:]
    k = (k * (last - total).exp()[..., None]).transpose(-1, -2)
    state = q.new_zeros(b, hv, dk, dv) if h0 is None else h0
    outs = []
    for i in range(n):                                 # the recurrence over chunks has no other order
        new = u[:, :, i] - w[:, :, i] @ state
        outs.append(q[:, :, i] @ state + p[:, :, i] @ new)
        state = state * last[:, :, i, :, None].exp() + k[:, :, i] @ new
    out = torch.stack(outs, dim=2).reshape(b, hv, n * CHUNK, dv)[:, :, :l]
    return out.transpose(1, 2), state


def _flip(x, yes):
    return x.flip(1) if yes else x


def _plain_forward(s):
    c = s["case"]
    scale = c["dk"] ** -0.5
    x = [s[n].float() for n in ("q", "k", "v", "g", "beta")]
    if s["offsets"] is None:
        out, state = _plain_delta(*[_flip(y, c["reverse"]) for y in x], s["h0"], scale)
        out = _flip(out, c["reverse"])
    else:
        # packed sequences laid out side by side: token t of sequence i at [i, t], nothing past its end
        off = s["offsets"].long()
        t = torch.arange(s["longest"], device="cuda")
        at = off[:-1, None] + t
        inside = at < off[1:, None]
        at = torch.where(inside, at, 0)
        side = [torch.where(inside.reshape(inside.shape + (1,) * (y.dim() - 2)), y[0][at], 0.0) for y in x]
        out, state = _plain_delta(*side, s["h0"], scale)
        token = torch.arange(x[0].shape[1], device="cuda")
        row = (token[:, None] >= off[1:]).sum(1)
        out = out[row, token - off[row]][None]
    out = out.to(s["v"].dtype).contiguous()
    return dict(out=out, state=state) if c["state"] else dict(out=out)


def _plain_backward(s):
    c = s["case"]
    x = [s[n].detach().float().requires_grad_(True) for n in ("q", "k", "v", "g", "beta")]
    out, _ = _plain_delta(*[_flip(y, c["reverse"]) for y in x], None, c["dk"] ** -0.5)
    got = torch.autograd.grad(_flip(out, c["reverse"]), x, s["dout"].float())
    return {n: d.to(s[n].dtype).contiguous() for n, d in zip(("q", "k", "v", "g", "beta"), got)}


def _plain_step(s):
    c = s["case"]
    group = c["hv"] // c["hk"]
    idle = (s["slots"] < 0)[:, None, None]
    at = torch.where(s["slots"] < 0, c["slots"] - 1, s["slots"]).long()      # idle rows put nobody's slot back as it was
    old = s["state"][at]
    q, k = (x.float().repeat_interleave(group, dim=1) for x in (s["q"], s["k"]))
    new = old * s["g"].exp()[..., None, None]
    err = (s["v"].float() - (k[..., None] * new).sum(-2)) * s["beta"][..., None]
    new = new + k[..., None] * err[..., None, :]
    out = (q[..., None] * new).sum(-2) * c["dk"] ** -0.5
    s["state"][at] = torch.where(idle[..., None], old, new)
    return dict(out=torch.where(idle, 0.0, out).to(s["v"].dtype), state=s["state"])


def _plain_clip(s):
    norm = torch.stack([(x.float() * x.float()).sum() for x in s["grads"]]).sum().sqrt()
    factor = (s["case"]["most"] / (norm + EPS)).clamp(max=1.0)
    for x, y in zip(s["grads"], s["outs"]):
        y.copy_(x.float() * factor)
    return dict(norm=norm, **s["flat"])


def _own(s):
    import selective_scan_fwd_amd as vm

    c = s["case"]
    if c["op"] == "norm_rope":
        more = dict(wq=s["wq"], wk=s["wk"], cos=s["cos"], sin=s["sin"], positions=s["positions"], eps=EPS, l2=c["l2"],
                    interleaved=c["interleaved"])
        if not c["back"]:
            q, k = vm.vm_head_norm_rope(s["q"], s["k"], **more)
            return dict(q=q, k=k)
        dq, dk, dwq, dwk = vm.vm_head_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], **more)
        return dict(dq=dq, dk=dk) if dwq is None else dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    if c["op"] == "delta":
        out, state = vm.vm_gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], h0=s["h0"], offsets=s["offsets"],
                                           reverse=c["reverse"], want_state=c["state"])
        return dict(out=out, state=state) if c["state"] else dict(out=out)
    if c["op"] == "delta_back":
        d = vm.vm_gated_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], reverse=c["reverse"])
        return {n: d[n] for n in ("q", "k", "v", "g", "beta")}
    if c["op"] == "step":
        out = vm.vm_gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return dict(out=out, state=s["state"])
    return dict(norm=vm.vm_clip_grad_norm(s["grads"], c["most"], out=s["outs"]), **s["flat"])


def run(state):
    if own:
        return _own(state)
    plain = dict(norm_rope=_plain_norm, delta=_plain_forward, delta_back=_plain_backward, step=_plain_step, clip=_plain_clip)
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------- the work of a pass
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "clip":
        n = sum(math.prod(s) for s in _clip_shapes(case))
        return dict(bytes=2 * n * es, flops=3 * n)
    b = case["batch"]
    if case["op"] == "norm_rope":
        t = b * case["seqlen"]
        n = t * (case["hq"] + case["hk"]) * case["dim"]
        table = 8 * min(t, 2 * max(case["seqlen"], 64)) * (case["rot"] // 2) + (4 * t if case["rot"] else 0)
        return dict(bytes=n * es * (3 if case["back"] else 2) + table, flops=n * (16 if case["back"] else 8))
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    if case["op"] == "step":
        active = b - (len(range(8, b, 9)) if b > 8 else 0)
        return dict(bytes=8 * active * hv * dk * dv + b * (2 * hk * dk + 2 * hv * dv) * es, flops=7 * active * hv * dk * dv)
    t = b * case["seqlen"]
    if case.get("ragged"):
        t = sum(_all_lengths(case))
    tokens = t * ((2 * hk * dk + 2 * hv * dv) * es + 8 * hv)
    state = (8 if case.get("state") else 0) * b * hv * dk * dv
    # products of a chunk: keys with keys and queries, the state read twice and written once, the triangle's solution and use
    flops = 2 * t * hv * (3 * dk * dv + CHUNK * (dk + dv))
    if case["op"] == "delta":
        return dict(bytes=tokens + state, flops=flops)
    return dict(bytes=2 * tokens + t * hv * dv * es, flops=3 * flops)


# -------------------------------------------- the definitions in 64 bits
def _exact_norm(case, s):
    r = case["rot"]

    def turned(x, sign):
        if not r:
            return x
        y = x.clone()
        i = torch.arange(r // 2, device=x.device)
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
        z = torch.complex(x[..., first], x[..., second])
        where = s["positions"].long()
        z = z * torch.complex(s["cos"].double()[where], sign * s["sin"].double()[where]).unsqueeze(2)
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def length(x):
        total = x.pow(2).sum(-1, keepdim=True)
        return (total + EPS).sqrt() if case["l2"] else (total / case["dim"] + EPS).sqrt()

    got = {}
    for n in ("q", "k"):
        x = s[n].double()
        w = s["w" + n].double() if s["w" + n] is not None else torch.ones(case["dim"], device="cuda", dtype=torch.float64)
        size = length(x)
        if not case["back"]:
            got[n] = turned(x / size * w, 1.0)
            continue
        d = turned(s["d" + n].double(), -1.0)
        if s["w" + n] is not None:
            got["dw" + n] = (d * x / size).sum((0, 1, 2))
        d = d * w
        share = 1.0 if case["l2"] else 1.0 / case["dim"]
        got["d" + n] = d / size - x * (d * x).sum(-1, keepdim=True) * share / size.pow(3)
    return got


def _exact_delta(case, s):
    hv, group, scale = case["hv"], case["hv"] // case["hk"], 1 / math.sqrt(case["dk"])
    q, k, v, g, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    heads = torch.arange(hv, device="cuda") // group
    q, k = q[:, :, heads], k[:, :, heads]
    out = torch.zeros_like(v)
    off = s["offsets"].tolist() if s["offsets"] is not None else None
    n = case["batch"]
    state = s["h0"].double().clone() if s["h0"] is not None else v.new_zeros(n, hv, case["dk"], case["dv"])
    for t in range(s["longest"]):
        if off is None:
            at = slice(None), case["seqlen"] - 1 - t if case["reverse"] else t
            live = slice(None)
        else:
            live = torch.tensor([i for i in range(n) if off[i] + t < off[i + 1]], device="cuda")
            at = 0, torch.tensor([off[i] + t for i in range(n) if off[i] + t < off[i + 1]], device="cuda")
        old = state[live] * g[at].exp()[..., None, None]
        miss = v[at] - torch.einsum("bhkv,bhk->bhv", old, k[at])
        new = old + torch.einsum("bh,bhk,bhv->bhkv", beta[at], k[at], miss)
        state[live] = new
        out[at] = scale * torch.einsum("bhkv,bhk->bhv", new, q[at])
    return dict(out=out, state=state) if case["state"] else dict(out=out)


def _exact_delta_back(case, s):
    b, l, hk, hv, dk, dv = (case[n] for n in ("batch", "seqlen", "hk", "hv", "dk", "dv"))
    if b * hv * dk * dv * 8 * (l + 8) > 60e9:
        return None
    group, scale = hv // hk, 1 / math.sqrt(dk)
    q, k, v, g, beta, dout = (s[n].double() for n in ("q", "k", "v", "g", "beta", "dout"))
    heads = torch.arange(hv, device="cuda") // group
    q, k = q[:, :, heads], k[:, :, heads]
    order = list(range(l))[::-1] if case["reverse"] else list(range(l))
    states = torch.zeros(l + 1, b, hv, dk, dv, device="cuda", dtype=torch.float64)
    for n, t in enumerate(order):
        old = states[n] * g[:, t].exp()[..., None, None]
        miss = v[:, t] - torch.einsum("bhkv,bhk->bhv", old, k[:, t])
        states[n + 1] = old + torch.einsum("bh,bhk,bhv->bhkv", beta[:, t], k[:, t], miss)
    d = {n: torch.zeros_like(x) for n, x in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta))}
    ds = torch.zeros_like(states[0])
    for n, t in list(enumerate(order))[::-1]:
        a = g[:, t].exp()[..., None, None]
        old = states[n] * a
        miss = v[:, t] - torch.einsum("bhkv,bhk->bhv", old, k[:, t])
        d["q"][:, t] = scale * torch.einsum("bhkv,bhv->bhk", states[n + 1], dout[:, t])
        ds = ds + scale * torch.einsum("bhk,bhv->bhkv", q[:, t], dout[:, t])
        along = torch.einsum("bhkv,bhk->bhv", ds, k[:, t])
        d["beta"][:, t] = (along * miss).sum(-1)
        dmiss = beta[:, t][..., None] * along
        d["v"][:, t] = dmiss
        d["k"][:, t] = beta[:, t][..., None] * torch.einsum("bhkv,bhv->bhk", ds, miss) - torch.einsum("bhkv,bhv->bhk", old, dmiss)
        ds = ds - torch.einsum("bhk,bhv->bhkv", k[:, t], dmiss)
        d["g"][:, t] = (ds * old).sum((-1, -2))
        ds = ds * a
    for n in ("q", "k"):
        d[n] = d[n].reshape(b, l, hk, group, dk).sum(3)
    return d


def _exact_step(case, s):
    group, scale = case["hv"] // case["hk"], 1 / math.sqrt(case["dk"])
    state, out = s["state"].double().clone(), torch.zeros(s["v"].shape, device="cuda", dtype=torch.float64)
    rows = [(i, j) for i, j in enumerate(s["slots"].tolist()) if j >= 0]
    i, j = (torch.tensor(x, device="cuda", dtype=torch.long) for x in zip(*rows))
    heads = torch.arange(case["hv"], device="cuda") // group
    q, k = s["q"].double()[i][:, heads], s["k"].double()[i][:, heads]
    old = state[j] * s["g"].double()[i].exp()[..., None, None]
    miss = s["v"].double()[i] - torch.einsum("bhkv,bhk->bhv", old, k)
    state[j] = old + torch.einsum("bh,bhk,bhv->bhkv", s["beta"].double()[i], k, miss)
    out[i] = scale * torch.einsum("bhkv,bhk->bhv", state[j], q)
    return dict(out=out, state=state)


def _exact_clip(case, s):
    norm = math.sqrt(math.fsum(float(x.double().pow(2).sum()) for x in s["grads"]))
    factor = min(1.0, case["most"] / (norm + EPS))
    got = dict(norm=torch.tensor(norm, device="cuda", dtype=torch.float64))
    for key in s["flat"]:
        got[key] = torch.cat([x.double().reshape(-1) * factor for x in s["grads"] if str(x.dtype)[6:] == key])
    return got


def exact(case, seed):
    s = prepare(case, seed)
    how = dict(norm_rope=_exact_norm, delta=_exact_delta, delta_back=_exact_delta_back, step=_exact_step, clip=_exact_clip)
    return how[case["op"]](case, s)
