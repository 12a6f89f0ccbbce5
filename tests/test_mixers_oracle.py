"""The 64-bit definitions of the matrix-state mixers, checked by themselves on
the CPU: gradients against central differences, the norm's lengths, rotations
that keep lengths, and the delta rule's defining property (with full write
strength and no decay a stored pair is read back exactly)."""
import numpy as np
import pytest

from oracle import mixers


def _delta_inputs(seed, b=2, l=5, hk=2, hv=4, dk=3, dv=2, n=None):
    r = np.random.RandomState(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    x = dict(q=r.randn(b, l, hk, dk), k=unit(r.randn(b, l, hk, dk)), v=r.randn(b, l, hv, dv),
             g=-r.rand(b, l, hv), beta=r.rand(b, l, hv))
    return x, r.randn(n or b, hv, dk, dv), r


@pytest.mark.parametrize("reverse,offsets", [(False, None), (True, None), (False, [0, 2, 2, 5]), (True, [0, 4, 5])])
def test_delta_gradients_match_differences(reverse, offsets):
    n = len(offsets) - 1 if offsets else 2
    x, h0, r = _delta_inputs(3, b=1 if offsets else 2, n=n)
    dout, dstate = r.randn(*x["v"].shape), r.randn(*h0.shape)

    def loss(h0=h0, **new):
        out, state, _ = mixers.delta(**{**x, **new}, scale=0.7, h0=h0, reverse=reverse, offsets=offsets)
        return (dout * out).sum() + (dstate * state).sum()

    d = mixers.delta_grad(**x, scale=0.7, dout=dout, h0=h0, dstate=dstate, reverse=reverse, offsets=offsets)
    step = 1e-5                        # error of a central difference: about step^2 and 1e-16 / step
    for name in ("q", "k", "v", "g", "beta", "h0"):
        base = h0 if name == "h0" else x[name]
        for at in [tuple(r.randint(s) for s in base.shape) for _ in range(6)]:
            hi, lo = base.copy(), base.copy()
            hi[at] += step
            lo[at] -= step
            num = (loss(**{name: hi}) - loss(**{name: lo})) / (2 * step)
            assert abs(num - d[name][at]) < 1e-6 * (1 + abs(num)), (name, at)


def test_delta_reads_back_what_it_wrote():
    x, _, _ = _delta_inputs(4, l=3)
    x["g"][:] = 0
    x["beta"][:] = 1
    x["q"] = x["k"]
    out, _, _ = mixers.delta(**x, scale=1.0)
    np.testing.assert_allclose(out, x["v"], atol=1e-12)


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm_gradients_match_differences(l2, interleaved):
    r = np.random.RandomState(5)
    x, w, dy = r.randn(2, 3, 2, 7), r.randn(7), r.randn(2, 3, 2, 7)
    cos, sin = np.cos(r.rand(9, 2) * 6), np.sin(r.rand(9, 2) * 6)
    pos = np.array([[0, 8, -1], [9, 3, 3]])
    more = dict(cos=cos, sin=sin, positions=pos, eps=1e-3, l2=l2, interleaved=interleaved)
    dx, dw = mixers.head_norm(x, w, dy=dy, **more)
    step = 1e-5
    for base, grad, call in ((x, dx, lambda z: mixers.head_norm(z, w, **more)),
                             (w, dw, lambda z: mixers.head_norm(x, z, **more))):
        for at in [tuple(r.randint(s) for s in base.shape) for _ in range(8)]:
            hi, lo = base.copy(), base.copy()
            hi[at] += step
            lo[at] -= step
            num = ((dy * call(hi)).sum() - (dy * call(lo)).sum()) / (2 * step)
            assert abs(num - grad[at]) < 1e-6 * (1 + abs(num))
    y = mixers.head_norm(x, None, **more)
    assert (y[0, 2] == 0).all() and (y[1, 0] == 0).all()        # padding


def test_rotation_keeps_lengths():
    r = np.random.RandomState(6)
    x = r.randn(1, 4, 2, 8)
    angle = r.rand(4, 4) * 6
    for inter in (False, True):
        y = mixers.head_norm(x, None, np.cos(angle), np.sin(angle), l2=True, eps=0.0, interleaved=inter)
        np.testing.assert_allclose((y * y).sum(-1), 1.0, atol=1e-12)


def test_clip():
    norm, got = mixers.clip([np.full(3, 2.0), np.full((1, 2), 2.0)], 1.0)
    assert abs(norm - np.sqrt(20.0)) < 1e-12
    assert abs(np.sqrt(sum((x * x).sum() for x in got)) - 1.0) < 1e-6
    norm, got = mixers.clip([np.full(3, 2.0)], 100.0)
    assert (got[0] == 2.0).all()
