"""Cases and plain forms of the prompt and token operators, for timing and comparison.

A block of a language model around the selective scan, whose tokens come as rows
of a projection, in packed prompts or one at a time:

  conv    the short causal convolution with SiLU over prompts (dense or packed,
          from kept windows), over single tokens, and its gradients
  scan    the selective scan  h_t = exp(dt A) h_{t-1} + dt B u,  y = C h + D u,
          out = y SiLU(z)  over prompts, over single tokens, and its gradients
  before  residual sum with a scale, then the norm a block reads; with gradients
  after   the norm of a block's output by groups, gated, added to the residual
          with a scale; with gradients

`run` computes them with elementary torch operations in fp32 (own = False) or
through the package's entry points (own = True).  `exact` evaluates the
definitions in 64 bits, token by token where there is a recurrence.
"""
import math

import torch

own = False

CHUNK = 64
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of eight sequences, cut from the projection's row: latency only
        dict(name="conv one token", op="conv_step", dtype="bf16", batch=8, slots=11, dim=4096, width=4, strided=True),
        # a serving batch of forty prompts of 1 to some 1500 tokens, part of them continued, windows kept in slots
        dict(name="conv packed prompts", op="conv", dtype="bf16", batch=40, seqlen=1500, dim=4096, width=4, packed=True,
             pool=True, strided=True),
        # gradients of a training step at 197 tokens
        dict(name="conv back 197 tokens", op="conv_back", dtype="f32", batch=128, seqlen=197, dim=384, width=4, packed=False,
             strided=False),
        # one token of a full serving batch on a pool of states, some rows idle
        dict(name="scan one token", op="scan_step", dtype="bf16", batch=128, slots=144, dim=4096, n=16, gate=True,
             strided=True),
        # one long prompt: few rows, the sequence is all there is to share out
        dict(name="scan one prompt", op="scan", dtype="bf16", batch=1, seqlen=4097, dim=4096, n=16, gate=True, packed=False,
             pool=False, strided=True),
        # a serving batch of forty prompts, part of them continued, states kept in slots
        dict(name="scan packed prompts", op="scan", dtype="bf16", batch=40, seqlen=1500, dim=4096, n=16, gate=True,
             packed=True, pool=True, strided=True),
        # gradients of a training step at 197 tokens
        dict(name="scan back 197 tokens", op="scan_back", dtype="f32", batch=128, seqlen=197, dim=384, n=16, gate=True,
             packed=False, state=False, strided=False),
        # gradients over two long rows that start from earlier states and hand theirs on
        dict(name="scan back 4097 tokens", op="scan_back", dtype="bf16", batch=2, seqlen=4097, dim=2048, n=16, gate=True,
             packed=False, state=True, strided=True),
        # the norm before a block for one token of eight sequences: latency only
        dict(name="norm before one token", op="before", back=False, dtype="bf16", rdtype="f32", rows=8, dim=2048,
             center=False, scaled=False),
        # its gradients over four long rows, residual kept in fp32, a learned scale for each channel
        dict(name="norm before back 4097 tokens", op="before", back=True, dtype="bf16", rdtype="f32", rows=4 * 4097,
             dim=2048, center=False, scaled=True),
        # the gated norm of 16 heads of 128 over four long rows, the gate cut from a projection's row
        dict(name="norm after heads", op="after", back=False, dtype="bf16", rdtype="", rows=4 * 4097, dim=2048, group=128,
             shared=True, gate_first=False, scaled=False, strided=True),
        # gradients at 197 tokens, whole rows gated before the norm, added to the residual with a scale
        dict(name="norm after back 197 tokens", op="after", back=True, dtype="f32", rdtype="f32", rows=128 * 197, dim=384,
             group=384, shared=False, gate_first=True, scaled=True, strided=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_back", "conv_step", "scan", "scan", "scan_step", "scan_back", "scan_back", "before", "after"])
    dtype = rng.choice(["f32", "bf16"])
    strided = rng.random() < 0.5
    if op in ("before", "after"):
        dim = _log(rng, 48, 8192)
        rows = _log(rng, 1, min(16000, 30_000_000 // dim))
        case = dict(op=op, back=rng.random() < 0.5, dtype=dtype, rows=rows, dim=dim, scaled=rng.random() < 0.5,
                    rdtype=rng.choice(["", "f32", dtype]))
        if op == "before":
            return dict(case, center=rng.random() < 0.4)
        group = rng.choice([dim, dim, 32, 64, 80, 128])
        dim = max(1, dim // group) * group
        return dict(case, dim=dim, group=group, shared=rng.random() < 0.5, gate_first=rng.random() < 0.5, strided=strided)
    dim = _log(rng, 24, 4096)
    width = rng.choice([2, 3, 4, 4, 4])
    n = rng.choice([16, 16, 16, 8, 5, 1])
    if op in ("conv_step", "scan_step"):
        batch = _log(rng, 1, 256)
        batch = max(1, min(batch, 128 * 4096 // dim))
        more = dict(width=width) if op == "conv_step" else dict(n=n, gate=rng.random() < 0.7)
        return dict(op=op, dtype=dtype, batch=batch, slots=batch + 1 + rng.randrange(16), dim=dim, strided=strided, **more)
    most = 16_000_000 if op != "scan_back" else 8_000_000         # tokens times channels
    seqlen = _log(rng, 1, min(4097, most // dim))
    batch = max(1, min(_log(rng, 1, 128), most // (seqlen * dim)))
    case = dict(op=op, dtype=dtype, batch=batch, seqlen=seqlen, dim=dim, packed=rng.random() < 0.4, strided=strided)
    if op in ("conv", "conv_back"):
        case["width"] = width
    else:
        case.update(n=n, gate=rng.random() < 0.7)
    if op in ("conv", "scan"):
        case["pool"] = rng.random() < 0.5
    if op == "scan_back":
        case["state"] = rng.random() < 0.5
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


def _slices(parts, strided, dtype):
    """The parts [..., dim] as slices of a common row of a projection, or dense."""
    parts = [p.to(dtype) for p in parts]
    if not strided:
        return parts
    return list(torch.cat(parts, dim=-1).split([p.shape[-1] for p in parts], dim=-1))


def _all_lengths(case):
    """Lengths of packed sequences: spread over 1 to seqlen by their logarithm, one of them empty."""
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


def _rows(case, seed, s):
    """Batch, length and offsets of a case's rows of tokens."""
    s["offsets"] = None
    if not case["packed"]:
        return case["batch"], case["seqlen"]
    lens = _lengths(case, seed)
    s["offsets"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    return 1, sum(lens)


def _pool(case, g, s, shape, dtype):
    """Kept states in slots: each sequence's slot (one of many has none), and which sequences start anew."""
    n = case["batch"]
    s["slots"] = torch.randperm(n + 3, generator=g, device="cuda")[:n].to(torch.int32)
    if n > 8:
        s["slots"][3] = -1
    s["fresh"] = (_rand(g, n) < 0.5).to(torch.int32)
    s["pool"] = (0.5 * _randn(g, n + 3, *shape)).to(dtype)


def _conv_inputs(case, seed):
    g = _gen(seed)
    dtype, d, w = DT[case["dtype"]], case["dim"], case["width"]
    s = dict(w=0.5 * (2 * _rand(g, d, w) - 1), bias=0.5 * (2 * _rand(g, d) - 1))
    if case["op"] == "conv_step":
        s["x"], _ = _slices([_randn(g, case["batch"], d), _randn(g, case["batch"], d)], case["strided"], dtype)
        s["pool"] = _randn(g, case["slots"], w - 1, d).to(dtype)
        s["slots"] = _step_slots(case, g)
        return s
    b, l = _rows(case, seed, s)
    s["x"], _ = _slices([_randn(g, b, l, d), _randn(g, b, l, d)], case["strided"], dtype)
    if case.get("pool"):
        _pool(case, g, s, (w - 1, d), dtype)
    if case["op"] == "conv_back":
        s["dout"] = _randn(g, b, l, d).to(dtype)
    return s


def _step_slots(case, g):
    """Each row's slot of the pool; the last slot is nobody's, every ninth row is idle (-1)."""
    b = case["batch"]
    slots = torch.randperm(case["slots"] - 1, generator=g, device="cuda")[:b].to(torch.int32)
    if b > 8:
        slots[8::9] = -1
    return slots


def _scan_inputs(case, seed):
    g = _gen(seed)
    dtype, d, n = DT[case["dtype"]], case["dim"], case["n"]
    s = {}
    lead = (case["batch"],) if case["op"] == "scan_step" else _rows(case, seed, s)
    # decays A about -1 to -n, steps softplus(delta + bias) about 1e-3 to 1e-1, as after training
    s["A"] = -(1 + torch.arange(n, device="cuda")) * torch.exp(0.1 * _randn(g, d, n))
    s["D"] = 1 + 0.1 * _randn(g, d)
    s["bias"] = torch.log(torch.expm1(torch.exp(math.log(1e-3) + math.log(100.0) * _rand(g, d))))
    s["u"] = torch.nn.functional.silu(1.5 * _randn(g, *lead, d)).to(dtype)
    s["delta"] = _randn(g, *lead, d).to(dtype)
    _, s["B"], s["C"] = _slices([_randn(g, *lead, max(1, d // 16)), _randn(g, *lead, n), _randn(g, *lead, n)],
                                case["strided"], dtype)
    s["z"] = None
    if case["gate"]:
        _, s["z"] = _slices([_randn(g, *lead, d), _randn(g, *lead, d)], case["strided"], dtype)
    if case["op"] == "scan_step":
        s["pool"] = _randn(g, case["slots"], d, n)
        s["slots"] = _step_slots(case, g)
    if case.get("pool"):
        _pool(case, g, s, (d, n), torch.float32)
    if case["op"] == "scan_back":
        s["dout"] = _randn(g, *lead, d).to(dtype)
        s["h0"] = 0.5 * _randn(g, case["batch"], d, n) if case["state"] else None
        s["dstate"] = 0.5 * _randn(g, case["batch"], d, n) if case["state"] else None
    return s


def _norm_inputs(case, seed):
    g = _gen(seed)
    r, d, dtype = case["rows"], case["dim"], DT[case["dtype"]]
    rd = DT[case["rdtype"]] if case["rdtype"] else None
    s = dict(scale=0.5 + 0.1 * _randn(g, d) if case["scaled"] else None, w=None, b=None, residual=None, dr=None)
    if case["op"] == "before":
        s["w"] = 1 + 0.1 * _randn(g, d)
        s["b"] = 0.1 * _randn(g, d) if case["center"] else None
        s["x"] = _randn(g, r, d).to(dtype)
        if rd is not None:
            s["residual"] = (3 * _randn(g, r, d)).to(rd)
        if case["back"]:
            s["dy"] = _randn(g, r, d).to(dtype)
            s["r"] = s.pop("residual") if rd is not None else (3 * _randn(g, r, d)).to(dtype)
            s["dr"] = _randn(g, r, d).to(rd) if rd is not None else None
        return s
    s["w"] = 1 + 0.1 * _randn(g, case["group"] if case["shared"] else d)
    s["x"] = _randn(g, r, d).to(dtype)
    _, s["z"] = _slices([_randn(g, r, d), _randn(g, r, d)], case["strided"], dtype)
    if case["back"]:
        s["dout"] = _randn(g, r, d).to(rd or dtype)
    elif rd is not None:
        s["residual"] = (3 * _randn(g, r, d)).to(rd)
    return s


def prepare(case, seed):
    kind = case["op"].split("_")[0]
    state = dict(conv=_conv_inputs, scan=_scan_inputs, before=_norm_inputs, after=_norm_inputs)[kind](case, seed)
    state["case"] = dict(case)
    return state


# ------------------------------------------------------------ plain forms
def _places(s, like):
    """Of every token of the flattened rows: its sequence and its place in it; and each sequence's first token and length."""
    b, l = like.shape[:2]
    t = torch.arange(b * l, device="cuda")
    if s["offsets"] is None:
        first = torch.arange(b, device="cuda") * l
        return t // l, t % l, first, torch.full_like(first, l)
    off = s["offsets"].long()
    seq = (t[:, None] >= off[1:]).sum(1)
    return seq, t - off[seq], off[:-1], off[1:] - off[:-1]


def _first_states(s, n):
    """Each sequence's first state out of the pool: 0 where it starts anew or has no slot."""
    if "pool" not in s:
        return None
    keep = (s["slots"] >= 0) & (s["fresh"] == 0)
    old = s["pool"][s["slots"].clamp(min=0).long()].float()
    return torch.where(keep.reshape((n,) + (1,) * (old.dim() - 1)), old, 0.0)


def _keep(s, last):
    """The pool with every sequence's last state in its slot (those without one put a slot back as it was)."""
    free = s["pool"].shape[0]
    pool = torch.cat([s["pool"], s["pool"][:1]])
    pool[torch.where(s["slots"] >= 0, s["slots"], free).long()] = last.to(pool.dtype)
    s["pool"].copy_(pool[:free])
    return s["pool"]


def _silu(x):
    return x * torch.sigmoid(x)


def _dsilu(x):
    y = torch.sigmoid(x)
    return y * (1 + x * (1 - y))


def _taps(s, x, width):
    """The inputs under each tap, tap by tap, and what the places are."""
    seq, pos, first, lens = _places(s, x)
    flat = x.float().flatten(0, 1)
    hist = _first_states(s, lens.shape[0])
    taps = []
    for k in range(width):
        back = width - 1 - k
        inside = (pos >= back)[:, None]
        before = 0.0 if hist is None else hist[seq, (width - 1 + pos - back).clamp(max=width - 2)]
        taps.append(torch.where(inside, flat[(torch.arange(flat.shape[0], device="cuda") - back).clamp(min=0)], before))
    return taps, flat, hist, (seq, pos, first, lens)


def _plain_conv(s):
    x, w, width = s["x"], s["w"], s["case"]["width"]
    taps, flat, hist, (_, _, first, lens) = _taps(s, x, width)
    v = s["bias"] + sum(t * w[:, k] for k, t in enumerate(taps))
    out = _silu(v).view(x.shape).to(x.dtype)
    if hist is None:
        return dict(out=out)
    last = []
    for j in range(width - 1):
        at = lens - (width - 1) + j
        rows = flat[(first + at).clamp(min=0, max=max(0, flat.shape[0] - 1))]
        old = hist[torch.arange(lens.shape[0], device="cuda"), (width - 1 + at).clamp(max=width - 2)]
        last.append(torch.where((at >= 0)[:, None], rows, old))
    return dict(out=out, state=_keep(s, torch.stack(last, dim=1)))


def _plain_conv_back(s):
    x, w, width = s["x"], s["w"], s["case"]["width"]
    taps, _, _, (_, pos, first, lens) = _taps(s, x, width)
    v = s["bias"] + sum(t * w[:, k] for k, t in enumerate(taps))
    dv = s["dout"].float().flatten(0, 1) * _dsilu(v)
    # 24-bit sums over a hundred thousand tokens lose what a gradient is compared by
    dw = torch.stack([(dv.double() * t).sum(0) for t in taps], dim=1).float()
    seq = _places(s, x)[0]
    dx = torch.zeros_like(dv)
    t = torch.arange(dv.shape[0], device="cuda")
    for k in range(width):
        ahead = width - 1 - k
        inside = (pos + ahead < lens[seq])[:, None]
        dx = dx + torch.where(inside, dv[(t + ahead).clamp(max=dv.shape[0] - 1)] * w[:, k], 0.0)
    return dict(x=dx.view(x.shape).to(x.dtype), w=dw, bias=dv.double().sum(0).float())


def _plain_conv_step(s):
    x, w, width = s["x"].float(), s["w"], s["case"]["width"]
    idle = s["slots"] < 0
    at = torch.where(idle, s["pool"].shape[0] - 1, s["slots"]).long()
    old = s["pool"][at]
    window = torch.cat([old.float(), x[:, None]], dim=1)
    out = _silu(s["bias"] + (window * w.t()).sum(1))
    s["pool"][at] = torch.where(idle[:, None, None], old, window[:, 1:].to(old.dtype))
    return dict(out=torch.where(idle[:, None], 0.0, out).to(s["x"].dtype), state=s["pool"])


def _steps(delta, bias):
    """softplus(delta + bias)"""
    x = delta.float() + bias
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _linear(logs, x):
    """h_t = exp(logs_t) h_{t-1} + x_t over the tokens of [t, d, n], from h = 0: chunks side by side, then joined."""
    t = x.shape[0]
    pad = -t % CHUNK
    if pad:
        logs, x = (torch.cat([y, y.new_zeros((pad,) + y.shape[1:])]) for y in (logs, x))
    c = (t + pad) // CHUNK
    logs, h = logs.view((c, CHUNK) + x.shape[1:]), x.view((c, CHUNK) + x.shape[1:]).clone()
    decay = logs.exp()
    for i in range(1, CHUNK):
        h[:, i].addcmul_(decay[:, i], h[:, i - 1])
    total = logs.cumsum(1).exp_()
    carry = torch.zeros_like(h[0, 0])
    before = torch.empty((c,) + carry.shape, device=x.device)
    for i in range(c):
        before[i] = carry
        carry = torch.addcmul(h[i, -1], total[i, -1], carry)
    h += total * before[:, None]
    return h.flatten(0, 1)[:t]


def _states(s, h0):
    """dt, dt u, decays' logarithms (-inf where a sequence starts) and states of every token, [t, d] and [t, d, n]."""
    u, B = (s[k].float().flatten(0, 1) for k in ("u", "B"))
    dt = _steps(s["delta"].flatten(0, 1), s["bias"])
    logs = dt[..., None] * s["A"]
    x = (dt * u)[..., None] * B[:, None, :]
    seq, pos, first, lens = _places(s, s["u"])
    if h0 is not None:                                   # a sequence's first state enters with its first token
        live = lens > 0
        at = first[live]
        x[at] += logs[at].exp() * h0[live]
    cut = torch.where((pos == 0)[:, None, None], -math.inf, logs)
    return u, B, dt, logs, cut, _linear(cut, x), (first, lens)


def _last(h, h0, first, lens):
    """Each sequence's last state; that of an empty one is its first."""
    rows = h[(first + lens - 1).clamp(min=0)]
    old = torch.zeros_like(rows) if h0 is None else h0
    return torch.where((lens > 0)[:, None, None], rows, old)


def _plain_scan(s):
    c = s["case"]
    n = c["batch"]
    h0 = _first_states(s, n)
    u, _, _, _, _, h, (first, lens) = _states(s, h0)
    y = (h * s["C"].float().flatten(0, 1)[:, None, :]).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float().flatten(0, 1))
    out = y.view(s["u"].shape).to(s["u"].dtype)
    last = _last(h, h0, first, lens)
    return dict(out=out, state=last if h0 is None else _keep(s, last))


def _plain_scan_back(s):
    u, B, dt, logs, cut, h, (first, lens) = _states(s, s["h0"])
    C = s["C"].float().flatten(0, 1)
    dout = s["dout"].float().flatten(0, 1)
    got = {}
    dy = dout
    if s["z"] is not None:
        z = s["z"].float().flatten(0, 1)
        dy = dout * _silu(z)
        y = (h * C[:, None, :]).sum(-1) + s["D"] * u
        got["z"] = dout * y * _dsilu(z)
    # the adjoint runs from a sequence's last token to its first
    x = dy[..., None] * C[:, None, :]
    live = lens > 0
    if s["dstate"] is not None:
        x[(first + lens - 1)[live]] += s["dstate"][live]
    after = torch.cat([cut[1:], torch.full_like(cut[:1], -math.inf)])
    grad = _linear(after.flip(0), x.flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    pos = _places(s, s["u"])[1]
    start = (pos == 0)[:, None, None]
    before = torch.where(start, 0.0, before)
    if s["h0"] is not None:
        before[first[live]] = s["h0"][live]
    passed = grad * logs.exp()
    through = passed * before
    dw = (grad * B[:, None, :]).sum(-1)
    ddt = dw * u + (through * s["A"]).sum(-1)
    x = s["delta"].float().flatten(0, 1) + s["bias"]
    ddelta = ddt * torch.sigmoid(x)
    got["u"] = dw * dt + s["D"] * dy
    got["delta"] = ddelta
    got["B"] = (grad * (dt * u)[..., None]).sum(1)
    got["C"] = (h * dy[..., None]).sum(1)
    got = {k: v.view(s[k].shape).to(s[k].dtype) for k, v in got.items()}
    got["A"] = (through * dt[..., None]).sum(0, dtype=torch.float64).float()
    got["D"] = (dy.double() * u).sum(0).float()
    got["bias"] = ddelta.sum(0, dtype=torch.float64).float()
    if s["h0"] is not None:
        got["h0"] = torch.where(live[:, None, None], passed[first.clamp(max=passed.shape[0] - 1)], s["dstate"])
    return got


def _plain_scan_step(s):
    idle = (s["slots"] < 0)[:, None]
    at = torch.where(s["slots"] < 0, s["pool"].shape[0] - 1, s["slots"]).long()
    old = s["pool"][at]
    u, dt = s["u"].float(), _steps(s["delta"], s["bias"])
    new = (dt[..., None] * s["A"]).exp() * old + (dt * u)[..., None] * s["B"].float()[:, None, :]
    y = (new * s["C"].float()[:, None, :]).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["pool"][at] = torch.where(idle[..., None], old, new)
    return dict(out=torch.where(idle, 0.0, y).to(s["u"].dtype), state=s["pool"])


def _normal(x, center):
    if center:
        x = x - x.mean(-1, keepdim=True)
    size = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * size, size


def _normal_back(d, n, size, center):
    d = d - n * (d * n).mean(-1, keepdim=True)
    if center:
        d = d - d.mean(-1, keepdim=True)
    return d * size


def _plain_before(s):
    c = s["case"]
    x = s["x"].float()
    if not c["back"]:
        r = x if s["scale"] is None else x * s["scale"]
        r = r if s["residual"] is None else s["residual"].float() + r
        y = _normal(r, c["center"])[0] * s["w"]
        y = y if s["b"] is None else y + s["b"]
        rd = s["x"].dtype if s["residual"] is None else s["residual"].dtype
        return dict(y=y.to(s["x"].dtype), r=r.to(rd))
    n, size = _normal(s["r"].float(), c["center"])
    dy = s["dy"].float()
    dr = _normal_back(dy * s["w"], n, size, c["center"])
    dr = dr if s["dr"] is None else dr + s["dr"].float()
    got = dict(residual=dr.to(s["r"].dtype), w=(dy.double() * n).sum(0).float())
    got["x"] = (dr if s["scale"] is None else dr * s["scale"]).to(s["x"].dtype)
    if s["b"] is not None:
        got["b"] = dy.double().sum(0).float()
    if s["scale"] is not None:
        got["scale"] = (dr.double() * x).sum(0).float()
    return got


def _plain_after(s):
    c = s["case"]
    rows, d, group = c["rows"], c["dim"], c["group"]
    cut = lambda y: y.view(rows, d // group, group)  # noqa: E731
    x, z = s["x"].float(), s["z"].float()
    w = s["w"] if c["shared"] else s["w"].view(d // group, group)
    gate = _silu(z)
    if not c["back"]:
        n = _normal(cut(x * gate if c["gate_first"] else x), False)[0] * w
        y = n.reshape(rows, d) * (1.0 if c["gate_first"] else gate)
        y = y if s["scale"] is None else y * s["scale"]
        if s["residual"] is None:
            return dict(out=y.to(s["x"].dtype))
        return dict(out=(s["residual"].float() + y).to(s["residual"].dtype))
    n, size = _normal(cut(x * gate if c["gate_first"] else x), False)
    dout = s["dout"].float()
    plain = (n * w).reshape(rows, d) * (1.0 if c["gate_first"] else gate)
    got = {}
    if s["scale"] is not None:
        got["scale"] = (dout.double() * plain).sum(0).float()
        dout = dout * s["scale"]
    dn = dout if c["gate_first"] else dout * gate
    dw = (cut(dn).double() * n).sum((0, 1) if c["shared"] else 0)
    got["w"] = dw.reshape(-1).float()
    dx = _normal_back(cut(dn) * w, n, size, False).reshape(rows, d)
    if c["gate_first"]:
        dz, dx = dx * x * _dsilu(z), dx * gate
    else:
        dz = dout * (n * w).reshape(rows, d) * _dsilu(z)
    return dict(got, x=dx.to(s["x"].dtype), z=dz.to(s["x"].dtype))


def _own(s):
    import selective_scan_fwd_amd as vm

    c = s["case"]
    if c["op"] == "conv_step":
        out = vm.vm_token_conv(s["x"], s["w"], s["pool"], bias=s["bias"], slots=s["slots"])
        return dict(out=out, state=s["pool"])
    if c["op"] == "conv":
        if "pool" not in s:
            return dict(out=vm.vm_prompt_conv(s["x"], s["w"], s["bias"], offsets=s["offsets"])[0])
        out, pool = vm.vm_prompt_conv(s["x"], s["w"], s["bias"], h0=s["pool"], state=s["pool"], offsets=s["offsets"],
                                      slots=s["slots"], fresh=s["fresh"])
        return dict(out=out, state=pool)
    if c["op"] == "conv_back":
        d = vm.vm_prompt_conv_bwd(s["x"], s["w"], s["dout"], s["bias"], offsets=s["offsets"])
        return {n: d[n] for n in ("x", "w", "bias")}
    if c["op"] == "scan_step":
        out = vm.vm_token_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["pool"], D=s["D"], delta_bias=s["bias"],
                               z=s["z"], slots=s["slots"])
        return dict(out=out, state=s["pool"])
    if c["op"] == "scan":
        more = dict(want_state=True)
        if "pool" in s:
            more = dict(h0=s["pool"], state=s["pool"], slots=s["slots"], fresh=s["fresh"])
        out, state = vm.vm_prompt_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], delta_bias=s["bias"],
                                       z=s["z"], offsets=s["offsets"], **more)
        return dict(out=out, state=state)
    if c["op"] == "scan_back":
        d = vm.vm_prompt_scan_bwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["dout"], D=s["D"], delta_bias=s["bias"],
                                  z=s["z"], h0=s["h0"], dstate=s["dstate"], offsets=s["offsets"])
        names = ["u", "delta", "B", "C", "A", "D"] + ["z"] * (s["z"] is not None) + ["h0"] * (s["h0"] is not None)
        return dict({n: d[n] for n in names}, bias=d["delta_bias"])
    if c["op"] == "before":
        if not c["back"]:
            y, r = vm.vm_norm_before(s["x"], s["w"], s["b"], residual=s["residual"], scale=s["scale"], center=c["center"],
                                     eps=EPS, want_residual=True)
            return dict(y=y, r=r)
        d = vm.vm_norm_before_bwd(s["dy"], s["r"], s["w"], s["b"], dr=s["dr"], x=s["x"], scale=s["scale"],
                                  center=c["center"], eps=EPS)
        names = ["residual", "w", "x"] + ["b"] * (s["b"] is not None) + ["scale"] * (s["scale"] is not None)
        return {n: d[n] for n in names}
    more = dict(group=c["group"], gate_first=c["gate_first"], scale=s["scale"], eps=EPS)
    if not c["back"]:
        return dict(out=vm.vm_norm_after(s["x"], s["w"], s["z"], residual=s["residual"], **more))
    d = vm.vm_norm_after_bwd(s["dout"], s["x"], s["w"], s["z"], **more)
    return {n: d[n] for n in ["x", "z", "w"] + ["scale"] * (s["scale"] is not None)}


def run(state):
    if own:
        return _own(state)
    plain = dict(conv=_plain_conv, conv_back=_plain_conv_back, conv_step=_plain_conv_step, scan=_plain_scan,
                 scan_back=_plain_scan_back, scan_step=_plain_scan_step, before=_plain_before, after=_plain_after)
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------- the work of a pass
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    op, d = case["op"], case["dim"]
    if op in ("before", "after"):
        rs = {"": es, "f32": 4, "bf16": 2}[case["rdtype"]]
        n = case["rows"] * d
        if op == "before":
            forward = 2 * es + (2 if case["rdtype"] else 1) * rs
            back = es + rs * (3 if case["rdtype"] else 2) + es * (2 if case["scaled"] else 1)
        else:
            forward = 2 * es + (2 if case["rdtype"] else 1) * rs
            back = 4 * es + rs
        return dict(bytes=n * (back if case["back"] else forward), flops=n * (20 if case["back"] else 10))
    if op in ("conv_step", "scan_step"):
        b = case["batch"]
        active = b - (len(range(8, b, 9)) if b > 8 else 0)
        if op == "conv_step":
            w = case["width"]
            return dict(bytes=active * d * (2 * es + 2 * (w - 1) * es) + 4 * d * (w + 1), flops=active * d * (2 * w + 4))
        n = case["n"]
        tokens = active * (d * es * (4 if case["gate"] else 3) + 2 * n * es)
        return dict(bytes=tokens + 8 * active * d * n + 4 * d * (n + 2), flops=7 * active * d * n)
    t = sum(_all_lengths(case)) if case["packed"] else case["batch"] * case["seqlen"]
    if op in ("conv", "conv_back"):
        w = case["width"]
        kept = 2 * case["batch"] * (w - 1) * d * es if case.get("pool") else 0
        return dict(bytes=t * d * es * (3 if op == "conv_back" else 2) + kept,
                    flops=t * d * (2 * w + 4) * (3 if op == "conv_back" else 1))
    n = case["n"]
    states = 4 * case["batch"] * d * n * ((2 if case.get("pool") else 1) if op == "scan" else (3 if case["state"] else 0))
    gate = 1 if case["gate"] else 0
    if op == "scan":
        return dict(bytes=t * (d * (3 + gate) + 2 * n) * es + states, flops=7 * t * d * n)
    return dict(bytes=t * (d * (5 + 2 * gate) + 4 * n) * es + states, flops=22 * t * d * n)


# -------------------------------------------- the definitions in 64 bits
def _spans(case, s):
    """(row, first token, end) of each sequence."""
    if s["offsets"] is None:
        return [(b, 0, case["seqlen"]) for b in range(case["batch"])]
    off = s["offsets"].tolist()
    return [(0, off[i], off[i + 1]) for i in range(len(off) - 1)]


def _begin(s, i, shape):
    if "pool" in s and int(s["slots"][i]) >= 0 and not int(s["fresh"][i]):
        return s["pool"][int(s["slots"][i])].double()
    return torch.zeros(shape, device="cuda", dtype=torch.float64)


def _exact_conv(case, s):
    w, width, d = s["w"].double(), case["width"], case["dim"]
    x = s["x"].double()
    out = torch.zeros_like(x)
    pool = s["pool"].double().clone() if "pool" in s else None
    got = dict(x=torch.zeros_like(x), w=torch.zeros_like(w), bias=torch.zeros(d, device="cuda", dtype=torch.float64))
    for i, (row, lo, hi) in enumerate(_spans(case, s)):
        full = torch.cat([_begin(s, i, (width - 1, d)), x[row, lo:hi]])
        if pool is not None and int(s["slots"][i]) >= 0:
            pool[int(s["slots"][i])] = full[hi - lo:]
        if hi == lo:
            continue
        window = full.unfold(0, width, 1)                # [tokens, d, width]
        v = torch.einsum("tdk,dk->td", window, w) + s["bias"].double()
        p = 1 / (1 + torch.exp(-v))
        if case["op"] == "conv":
            out[row, lo:hi] = v * p
            continue
        dv = s["dout"][row, lo:hi].double() * (p + v * p * (1 - p))
        got["w"] += torch.einsum("tdk,td->dk", window, dv)
        got["bias"] += dv.sum(0)
        dfull = torch.zeros_like(full)
        for k in range(width):
            dfull[k: k + hi - lo] += dv * w[:, k]
        got["x"][row, lo:hi] = dfull[width - 1:]
    if case["op"] == "conv_back":
        return got
    return dict(out=out) if pool is None else dict(out=out, state=pool)


def _exact_conv_step(case, s):
    pool, out = s["pool"].double().clone(), torch.zeros(s["x"].shape, device="cuda", dtype=torch.float64)
    for i, j in enumerate(s["slots"].tolist()):
        if j < 0:
            continue
        window = torch.cat([pool[j], s["x"][i].double()[None]])
        v = s["bias"].double() + torch.einsum("kd,dk->d", window, s["w"].double())
        out[i] = v / (1 + torch.exp(-v))
        pool[j] = window[1:]
    return dict(out=out, state=pool)


def _exact_dt(s, at):
    x = s["delta"][at].double() + s["bias"].double()
    return torch.logaddexp(x, torch.zeros_like(x)), torch.sigmoid(x)


def _walk(case, s):
    """For each place t: the sequences that have a token there, and where those tokens are."""
    spans = _spans(case, s)
    for t in range(max((hi - lo for _, lo, hi in spans), default=0)):
        live = [i for i, (_, lo, hi) in enumerate(spans) if lo + t < hi]
        rows, places = [spans[i][0] for i in live], [spans[i][1] + t for i in live]
        yield tuple(torch.tensor(v, device="cuda") for v in (live, rows, places))


def _exact_scan(case, s):
    n, d = case["batch"], case["dim"]
    A, D = s["A"].double(), s["D"].double()
    h = torch.stack([_begin(s, i, (d, case["n"])) for i in range(n)])
    out = torch.zeros(s["u"].shape, device="cuda", dtype=torch.float64)
    for live, row, place in _walk(case, s):
        at = row, place
        u, (dt, _) = s["u"][at].double(), _exact_dt(s, at)
        new = torch.exp(dt[..., None] * A) * h[live] + torch.einsum("bd,bn->bdn", dt * u, s["B"][at].double())
        h[live] = new
        y = torch.einsum("bdn,bn->bd", new, s["C"][at].double()) + D * u
        if s["z"] is not None:
            z = s["z"][at].double()
            y = y * z / (1 + torch.exp(-z))
        out[at] = y
    if "pool" not in s:
        return dict(out=out, state=h)
    pool = s["pool"].double().clone()
    for i, j in enumerate(s["slots"].tolist()):
        if j >= 0:
            pool[j] = h[i]
    return dict(out=out, state=pool)


def _exact_scan_back(case, s):
    n, d, N = case["batch"], case["dim"], case["n"]
    if 8 * d * N * s["u"].shape[0] * s["u"].shape[1] > 40e9:
        return None
    A, D = s["A"].double(), s["D"].double()
    zero = lambda *shape: torch.zeros(shape, device="cuda", dtype=torch.float64)  # noqa: E731
    h = s["h0"].double().clone() if s["h0"] is not None else zero(n, d, N)
    walk = list(_walk(case, s))
    kept = []
    for live, row, place in walk:                        # the states before each token
        at = row, place
        kept.append(h[live])
        dt, _ = _exact_dt(s, at)
        h[live] = torch.exp(dt[..., None] * A) * kept[-1] + \
            torch.einsum("bd,bn->bdn", dt * s["u"][at].double(), s["B"][at].double())
    got = {k: torch.zeros(s[k].shape, device="cuda", dtype=torch.float64) for k in ("u", "delta", "B", "C", "z") if s[k] is not None}
    got.update(A=zero(d, N), D=zero(d), bias=zero(d))
    g = s["dstate"].double().clone() if s["dstate"] is not None else zero(n, d, N)
    for (live, row, place), old in zip(walk[::-1], kept[::-1]):
        at = row, place
        u, B, C, dy = (s[k][at].double() for k in ("u", "B", "C", "dout"))
        dt, slope = _exact_dt(s, at)
        a = torch.exp(dt[..., None] * A)
        new = a * old + torch.einsum("bd,bn->bdn", dt * u, B)
        if s["z"] is not None:
            z = s["z"][at].double()
            p = torch.sigmoid(z)
            got["z"][at] = dy * (torch.einsum("bdn,bn->bd", new, C) + D * u) * (p + z * p * (1 - p))
            dy = dy * z * p
        dh = g[live] + torch.einsum("bd,bn->bdn", dy, C)
        got["C"][at] = torch.einsum("bdn,bd->bn", new, dy)
        got["B"][at] = torch.einsum("bdn,bd->bn", dh, dt * u)
        along = torch.einsum("bdn,bn->bd", dh, B)
        da = dh * old * a
        got["u"][at] = along * dt + D * dy
        got["D"] += (dy * u).sum(0)
        got["A"] += torch.einsum("bdn,bd->dn", da, dt)
        dd = (along * u + torch.einsum("bdn,dn->bd", da, A)) * slope
        got["delta"][at] = dd
        got["bias"] += dd.sum(0)
        g[live] = dh * a
    if s["h0"] is not None:
        got["h0"] = g
    return got


def _exact_scan_step(case, s):
    pool, out = s["pool"].double().clone(), torch.zeros(s["u"].shape, device="cuda", dtype=torch.float64)
    i, j = (torch.tensor(v, device="cuda", dtype=torch.long) for v in
            zip(*[(i, j) for i, j in enumerate(s["slots"].tolist()) if j >= 0]))
    u, (dt, _) = s["u"][i].double(), _exact_dt(s, i)
    new = torch.exp(dt[..., None] * s["A"].double()) * pool[j] + torch.einsum("bd,bn->bdn", dt * u, s["B"][i].double())
    y = torch.einsum("bdn,bn->bd", new, s["C"][i].double()) + s["D"].double() * u
    if s["z"] is not None:
        z = s["z"][i].double()
        y = y * z * torch.sigmoid(z)
    pool[j], out[i] = new, y
    return dict(out=out, state=pool)


def _exact_norm(x, w, b, center):
    """Norm over the last axis as a function that autograd differentiates."""
    if center:
        x = x - x.sum(-1, keepdim=True) / x.shape[-1]
    y = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    return y if b is None else y + b


def _leaves(s, *names):
    return {n: s[n].double().requires_grad_(True) for n in names if s[n] is not None}


def _exact_before(case, s):
    if not case["back"]:
        r = s["x"].double() * (1.0 if s["scale"] is None else s["scale"].double())
        r = r if s["residual"] is None else r + s["residual"].double()
        return dict(y=_exact_norm(r, s["w"].double(), None if s["b"] is None else s["b"].double(), case["center"]), r=r)
    v = _leaves(s, "r", "w", "b")
    y = _exact_norm(v["r"], v["w"], v.get("b"), case["center"])
    got = dict(zip(v, torch.autograd.grad(y, list(v.values()), s["dy"].double())))
    dr = got.pop("r")
    dr = dr if s["dr"] is None else dr + s["dr"].double()
    got.update(residual=dr, x=dr if s["scale"] is None else dr * s["scale"].double())
    if s["scale"] is not None:
        got["scale"] = torch.einsum("rd,rd->d", dr, s["x"].double())
    return got


def _exact_after(case, s):
    v = _leaves(s, "x", "z", "w", "scale")
    w = v["w"] if case["shared"] else v["w"].view(-1, case["group"])
    gate = v["z"] * torch.sigmoid(v["z"])
    x = v["x"] * gate if case["gate_first"] else v["x"]
    y = _exact_norm(x.unflatten(-1, (-1, case["group"])), w, None, False).flatten(-2)
    y = y if case["gate_first"] else y * gate
    y = y * v["scale"] if "scale" in v else y
    if case["back"]:
        return dict(zip(v, torch.autograd.grad(y, list(v.values()), s["dout"].double())))
    y = y.detach()
    return dict(out=y if s["residual"] is None else y + s["residual"].double())


def exact(case, seed):
    s = prepare(case, seed)
    how = dict(conv=_exact_conv, conv_back=_exact_conv, conv_step=_exact_conv_step, scan=_exact_scan,
               scan_back=_exact_scan_back, scan_step=_exact_scan_step, before=_exact_before, after=_exact_after)
    return how[case["op"]](case, s)
