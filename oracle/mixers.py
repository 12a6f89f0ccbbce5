"""64-bit definitions of the matrix-state mixers, for the tests: the gated
delta rule token by token with its adjoint, the per-head norm with rotation
and its gradients, and gradient clipping.  Plain numpy; shares no code with the
GPU path."""
import numpy as np


# --------------------------------------------------------- gated delta rule
def _spans(n, seqlen, offsets):
    if offsets is None:
        return [(b, 0, seqlen) for b in range(n)]
    return [(0, int(offsets[i]), int(offsets[i + 1])) for i in range(len(offsets) - 1)]


def delta(q, k, v, g, beta, scale, h0=None, reverse=False, offsets=None):
    """q, k [b, l, hk, dk], v [b, l, hv, dv], g, beta [b, l, hv]; returns
    (out, state [n, hv, dk, dv], trace) with trace[i]: a list of (token, state
    before, state after) of sequence i."""
    b, l, hv, dv = v.shape
    group, dk = hv // q.shape[2], q.shape[3]
    out = np.zeros((b, l, hv, dv))
    spans = _spans(b, l, offsets)
    state = np.zeros((len(spans), hv, dk, dv))
    trace = []
    for i, (row, lo, hi) in enumerate(spans):
        s = np.array(h0[i], dtype=np.float64) if h0 is not None else np.zeros((hv, dk, dv))
        steps = []
        for t in (range(hi - 1, lo - 1, -1) if reverse else range(lo, hi)):
            kt, qt = (np.repeat(x[row, t], group, axis=0) for x in (k, q))
            decayed = s * np.exp(g[row, t])[:, None, None]
            err = v[row, t] - (decayed * kt[:, :, None]).sum(1)
            new = decayed + beta[row, t][:, None, None] * kt[:, :, None] * err[:, None, :]
            out[row, t] = scale * (new * qt[:, :, None]).sum(1)
            steps.append((t, s, new))
            s = new
        state[i] = s
        trace.append(steps)
    return out, state, trace


def delta_grad(q, k, v, g, beta, scale, dout, h0=None, dstate=None, reverse=False, offsets=None):
    """Gradients of sum(dout * out) + sum(dstate * state), by the adjoint of
    each step in reverse order."""
    b, l, hv, dv = v.shape
    hk, dk = q.shape[2:]
    group = hv // hk
    d = dict(q=np.zeros(q.shape), k=np.zeros(k.shape), v=np.zeros(v.shape), g=np.zeros(g.shape),
             beta=np.zeros(beta.shape))
    spans = _spans(b, l, offsets)
    d["h0"] = np.zeros((len(spans), hv, dk, dv))
    _, _, trace = delta(q, k, v, g, beta, scale, h0, reverse, offsets)
    for i, (row, lo, hi) in enumerate(spans):
        ds = np.array(dstate[i], dtype=np.float64) if dstate is not None else np.zeros((hv, dk, dv))
        for t, before, after in trace[i][::-1]:
            kt, qt = (np.repeat(x[row, t], group, axis=0) for x in (k, q))
            a, be, do = np.exp(g[row, t])[:, None, None], beta[row, t][:, None], dout[row, t]
            decayed = before * a
            err = v[row, t] - (decayed * kt[:, :, None]).sum(1)
            d["q"][row, t] += (scale * (after * do[:, None, :]).sum(2)).reshape(hk, group, dk).sum(1)
            ds = ds + scale * qt[:, :, None] * do[:, None, :]
            along = (ds * kt[:, :, None]).sum(1)
            d["beta"][row, t] = (along * err).sum(1)
            derr = be * along
            d["v"][row, t] = derr
            dkt = be * (ds * err[:, None, :]).sum(2) - (decayed * derr[:, None, :]).sum(2)
            d["k"][row, t] += dkt.reshape(hk, group, dk).sum(1)
            ds = ds - kt[:, :, None] * derr[:, None, :]
            d["g"][row, t] = (ds * decayed).sum((1, 2))
            ds = ds * a
        d["h0"][i] = ds
    return d


# ------------------------------------------------------- norm and rotation
def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(x, cos, sin, positions, interleaved, back):
    rot = 2 * cos.shape[1]
    first, second = _pairs(rot, interleaved)
    c, s = cos[positions][:, :, None], sin[positions][:, :, None]
    if back:
        s = -s
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def head_norm(x, w=None, cos=None, sin=None, positions=None, eps=1e-6, l2=False, interleaved=False, dy=None):
    """y of x [b, l, h, d]; with dy: (dx, dw)."""
    b, l, _, dim = x.shape
    share = 1.0 if l2 else 1.0 / dim
    size = np.sqrt((x * x).sum(-1, keepdims=True) * share + eps)
    w = np.ones(dim) if w is None else w
    live = np.ones((b, l), bool)
    if cos is not None:
        positions = np.broadcast_to(np.arange(l), (b, l)) if positions is None else positions
        live = (positions >= 0) & (positions < cos.shape[0])
        positions = np.where(live, positions, 0)
    live = live[:, :, None, None]
    if dy is None:
        y = x / size * w
        return np.where(live, _turn(y, cos, sin, positions, interleaved, False) if cos is not None else y, 0.0)
    d = _turn(dy, cos, sin, positions, interleaved, True) if cos is not None else dy
    d = np.where(live, d, 0.0)
    dw = (d * x / size).sum((0, 1, 2))
    d = d * w
    return d / size - x * (d * x).sum(-1, keepdims=True) * share / size ** 3, dw


# ----------------------------------------------------------------- clipping
def clip(grads, max_norm):
    norm = np.sqrt(sum(float((x * x).sum()) for x in grads))
    f = min(1.0, max_norm / (norm + 1e-6))
    return norm, [x * f for x in grads]
