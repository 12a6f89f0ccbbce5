"""64-bit definitions of the prompt and token operators, for the tests: the short
causal convolution and the selective scan over rows of tokens, token by token, with
their adjoints, and the norms around a block with their gradients.  Plain numpy;
shares no code with the GPU path."""
import numpy as np


def spans(batch, seqlen, offsets):
    """(row, first token, end) of each sequence."""
    if offsets is None:
        return [(b, 0, seqlen) for b in range(batch)]
    return [(0, int(offsets[i]), int(offsets[i + 1])) for i in range(len(offsets) - 1)]


def _sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def silu(x):
    return x * _sigmoid(x)


def dsilu(x):
    s = _sigmoid(x)
    return s + x * s * _sigmoid(-x)


def softplus(x):
    return np.logaddexp(x, 0.0)


def first_states(n, h0, slots=None, fresh=None, shape=None):
    """Each sequence's first state: h0 by slot, 0 without one."""
    out = []
    for i in range(n):
        s = i if slots is None else int(slots[i])
        keep = h0 is not None and 0 <= s < len(h0) and not (fresh is not None and fresh[i])
        out.append(np.array(h0[s], dtype=np.float64) if keep else np.zeros(shape))
    return out


# ------------------------------------------------------------- convolution
def conv(x, w, bias=None, act=True, first=None, offsets=None):
    """x [b, l, d], w [d, W]; first: each sequence's window [W - 1, d]; returns
    (out, last windows).  Tokens of no sequence stay 0."""
    b, l, d = x.shape
    W = w.shape[1]
    out, last = np.zeros(x.shape), []
    for i, (row, lo, hi) in enumerate(spans(b, l, offsets)):
        full = np.concatenate([np.zeros((W - 1, d)) if first is None else first[i], x[row, lo:hi]])
        for t in range(hi - lo):
            v = (full[t: t + W] * w.T).sum(0) + (0 if bias is None else bias)
            out[row, lo + t] = silu(v) if act else v
        last.append(full[hi - lo:])
    return out, np.stack(last)


def conv_grad(x, w, dout, bias=None, act=True, first=None, dlast=None, offsets=None):
    b, l, d = x.shape
    W = w.shape[1]
    got = dict(x=np.zeros(x.shape), w=np.zeros(w.shape), bias=np.zeros(d), h0=[])
    for i, (row, lo, hi) in enumerate(spans(b, l, offsets)):
        full = np.concatenate([np.zeros((W - 1, d)) if first is None else first[i], x[row, lo:hi]])
        dfull = np.zeros(full.shape)
        if dlast is not None:
            dfull[hi - lo:] += dlast[i]
        for t in range(hi - lo):
            win = full[t: t + W]
            v = (win * w.T).sum(0) + (0 if bias is None else bias)
            dv = dout[row, lo + t] * (dsilu(v) if act else 1.0)
            dfull[t: t + W] += dv * w.T
            got["w"] += (dv * win).T
            got["bias"] += dv
        got["x"][row, lo:hi] = dfull[W - 1:]
        got["h0"].append(dfull[: W - 1])
    got["h0"] = np.stack(got["h0"])
    return got


# -------------------------------------------------------------------- scan
def scan(u, delta, A, B, C, D=None, bias=None, z=None, soft=True, first=None, offsets=None):
    """u, delta, z [b, l, d], A [d, n], B, C [b, l, n]; first: each sequence's state
    [d, n]; returns (out, last states, trace of states before each token)."""
    b, l, d = u.shape
    out, last, trace = np.zeros(u.shape), [], []
    for i, (row, lo, hi) in enumerate(spans(b, l, offsets)):
        h = np.zeros(A.shape) if first is None else first[i]
        steps = []
        for t in range(lo, hi):
            x = delta[row, t] + (0 if bias is None else bias)
            dt = softplus(x) if soft else x
            steps.append(h)
            h = np.exp(dt[:, None] * A) * h + (dt * u[row, t])[:, None] * B[row, t]
            y = h @ C[row, t] + (0 if D is None else D * u[row, t])
            out[row, t] = y if z is None else y * silu(z[row, t])
        last.append(h)
        trace.append(steps)
    return out, np.stack(last), trace


def scan_grad(u, delta, A, B, C, dout, D=None, bias=None, z=None, soft=True, first=None, dlast=None, offsets=None):
    b, l, d = u.shape
    got = {k: np.zeros(v.shape) for k, v in (("u", u), ("delta", delta), ("A", A), ("B", B), ("C", C), ("z", u))}
    got.update(D=np.zeros(d), delta_bias=np.zeros(d), h0=[])
    _, _, trace = scan(u, delta, A, B, C, D, bias, z, soft, first, offsets)
    for i, (row, lo, hi) in enumerate(spans(b, l, offsets)):
        g = np.zeros(A.shape) if dlast is None else dlast[i]
        for t in range(hi - 1, lo - 1, -1):
            x = delta[row, t] + (0 if bias is None else bias)
            dt, slope = (softplus(x), _sigmoid(x)) if soft else (x, np.ones(d))
            ut, old = u[row, t], trace[i][t - lo]
            a = np.exp(dt[:, None] * A)
            h = a * old + (dt * ut)[:, None] * B[row, t]
            dy = dout[row, t]
            if z is not None:
                y = h @ C[row, t] + (0 if D is None else D * ut)
                got["z"][row, t] = dy * y * dsilu(z[row, t])
                dy = dy * silu(z[row, t])
            g = g + dy[:, None] * C[row, t]
            got["C"][row, t] = dy @ h
            got["B"][row, t] = (dt * ut) @ g
            w = g @ B[row, t]
            through = g * a * old
            got["u"][row, t] = dt * w + (0 if D is None else D * dy)
            got["D"] += dy * ut
            got["A"] += dt[:, None] * through
            dd = (ut * w + (through * A).sum(1)) * slope
            got["delta"][row, t] = dd
            got["delta_bias"] += dd
            g = g * a
        got["h0"].append(g)
    got["h0"] = np.stack(got["h0"])
    return got


# ------------------------------------------------------------------- norms
def _norm(v, eps, center=False):
    if center:
        v = v - v.mean(-1, keepdims=True)
    size = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v * size, size


def _norm_grad(d, n, size, center=False):
    d = d - n * (d * n).mean(-1, keepdims=True)
    if center:
        d = d - d.mean(-1, keepdims=True)
    return d * size


def norm_before(x, w=None, b=None, residual=None, scale=None, factor=1.0, center=False, eps=1e-5):
    r = factor * x * (1.0 if scale is None else scale) + (0 if residual is None else residual)
    y = _norm(r, eps, center)[0] * (1.0 if w is None else w) + (0 if b is None else b)
    return y, r


def norm_before_grad(dy, r, w=None, dr=None, x=None, scale=None, factor=1.0, center=False, eps=1e-5):
    n, size = _norm(r, eps, center)
    d = _norm_grad(dy * (1.0 if w is None else w), n, size, center) + (0 if dr is None else dr)
    got = dict(residual=d, x=d * factor * (1.0 if scale is None else scale), w=(dy * n).sum(0), b=dy.sum(0))
    if scale is not None:
        got["scale"] = factor * (d * x).sum(0)
    return got


def norm_after(x, w=None, z=None, group=None, residual=None, scale=None, factor=1.0, gate_first=False, eps=1e-5):
    rows, dim = x.shape
    group = dim if group is None else group
    gate = 1.0 if z is None else silu(z)
    v = (x * gate if gate_first else x).reshape(rows, -1, group)
    gain = 1.0 if w is None else np.broadcast_to(w.reshape(-1, group), (dim // group, group))
    y = (_norm(v, eps)[0] * gain).reshape(rows, dim) * (1.0 if gate_first else gate)
    return factor * y * (1.0 if scale is None else scale) + (0 if residual is None else residual)


def norm_after_grad(dout, x, w=None, z=None, group=None, scale=None, factor=1.0, gate_first=False, eps=1e-5):
    rows, dim = x.shape
    group = dim if group is None else group
    cut = lambda a: a.reshape(rows, -1, group)
    gate = np.ones(x.shape) if z is None else silu(z)
    n, size = _norm(cut(x * gate if gate_first else x), eps)
    gain = np.ones((1, group)) if w is None else np.broadcast_to(w.reshape(-1, group), (dim // group, group))
    after = np.ones(x.shape) if gate_first else gate
    got = dict(scale=factor * (dout * (n * gain).reshape(rows, dim) * after).sum(0))
    d = dout * factor * (1.0 if scale is None else scale)
    dw = (cut(d * after) * n).sum(0)
    if w is not None:
        got["w"] = dw.reshape(-1) if w.size == dim else dw.sum(0)
    dv = _norm_grad(cut(d * after) * gain, n, size).reshape(rows, dim)
    got["x"] = dv * gate if gate_first else dv
    if z is not None:
        got["z"] = (dv * x if gate_first else d * (n * gain).reshape(rows, dim)) * dsilu(z)
    return got
