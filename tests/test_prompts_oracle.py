"""The 64-bit definitions against each other and against differences."""
import numpy as np
import pytest

import oracle.prompts as ref

rng = np.random.default_rng(5)


def _differences(f, args, names, grads, eps=1e-6):
    """Central differences of f(**args) against grads, in a random direction of each input."""
    for n in names:
        d = rng.standard_normal(args[n].shape)
        hi, lo = (f(**dict(args, **{n: args[n] + s * eps * d})) for s in (1, -1))
        want, got = (hi - lo) / (2 * eps), float((grads[n] * d).sum())
        assert abs(got - want) <= 1e-6 * (abs(want) + 1), n


@pytest.mark.parametrize("offsets", [None, np.array([0, 3, 3, 5])])
def test_scan_gradients_are_those_of_its_outputs(offsets):
    b, l, d, n = (2, 5, 3, 4) if offsets is None else (1, 5, 3, 4)
    k = b if offsets is None else 3
    a = dict(u=rng.standard_normal((b, l, d)), delta=rng.standard_normal((b, l, d)), A=-rng.random((d, n)) - 0.1,
             B=rng.standard_normal((b, l, n)), C=rng.standard_normal((b, l, n)), D=rng.standard_normal(d),
             bias=rng.standard_normal(d), z=rng.standard_normal((b, l, d)), first=rng.standard_normal((k, d, n)))
    dout, dlast = rng.standard_normal((b, l, d)), rng.standard_normal((k, d, n))

    def loss(**v):
        out, last, _ = ref.scan(**v, offsets=offsets)
        return float((out * dout).sum() + (last * dlast).sum())

    g = ref.scan_grad(**a, dout=dout, dlast=dlast, offsets=offsets)
    g.update(bias=g["delta_bias"], first=g["h0"])
    _differences(loss, a, list(a), g)


@pytest.mark.parametrize("width", [2, 4])
def test_conv_gradients_are_those_of_its_outputs(width):
    offsets = np.array([0, 1, 1, 7])
    a = dict(x=rng.standard_normal((1, 7, 3)), w=rng.standard_normal((3, width)), bias=rng.standard_normal(3),
             first=rng.standard_normal((3, width - 1, 3)))
    dout, dlast = rng.standard_normal((1, 7, 3)), rng.standard_normal((3, width - 1, 3))

    def loss(**v):
        out, last = ref.conv(**v, offsets=offsets)
        return float((out * dout).sum() + (last * dlast).sum())

    g = ref.conv_grad(**a, dout=dout, dlast=dlast, offsets=offsets)
    _differences(loss, a, list(a), dict(g, first=g["h0"]))


def test_a_prompt_in_parts_is_the_whole_prompt():
    l, d, n, w = 9, 4, 3, 4
    u, delta, z = (rng.standard_normal((1, l, d)) for _ in range(3))
    A, B, C = -rng.random((d, n)), rng.standard_normal((1, l, n)), rng.standard_normal((1, l, n))
    whole, last, _ = ref.scan(u, delta, A, B, C, z=z)
    h, parts = np.zeros((1, d, n)), []
    taps = rng.standard_normal((d, w))
    cwhole, _ = ref.conv(u, taps)
    win, cparts = np.zeros((1, w - 1, d)), []
    for lo, hi in ((0, 1), (1, 2), (2, 7), (7, 9)):
        o, h, _ = ref.scan(u[:, lo:hi], delta[:, lo:hi], A, B[:, lo:hi], C[:, lo:hi], z=z[:, lo:hi], first=h)
        parts.append(o)
        o, win = ref.conv(u[:, lo:hi], taps, first=win)
        cparts.append(o)
    assert np.allclose(np.concatenate(parts, 1), whole, rtol=1e-13) and np.allclose(h, last, rtol=1e-13)
    assert np.allclose(np.concatenate(cparts, 1), cwhole, rtol=1e-13)


@pytest.mark.parametrize("center", [False, True])
def test_norm_before_gradients(center):
    a = dict(x=rng.standard_normal((3, 6)), w=rng.standard_normal(6), b=rng.standard_normal(6),
             residual=rng.standard_normal((3, 6)), scale=rng.standard_normal(6))
    dy, dr = rng.standard_normal((3, 6)), rng.standard_normal((3, 6))

    def loss(**v):
        y, r = ref.norm_before(**v, factor=0.7, center=center)
        return float((y * dy).sum() + (r * dr).sum())

    r = ref.norm_before(**a, factor=0.7, center=center)[1]
    g = ref.norm_before_grad(dy, r, a["w"], dr, a["x"], a["scale"], 0.7, center)
    _differences(loss, a, list(a), g)


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("gains", [2, 6])
def test_norm_after_gradients(gate_first, gains):
    a = dict(x=rng.standard_normal((3, 6)), w=rng.standard_normal(gains), z=rng.standard_normal((3, 6)),
             scale=rng.standard_normal(6))
    dout = rng.standard_normal((3, 6))

    def loss(**v):
        return float((ref.norm_after(**v, group=2, factor=0.7, gate_first=gate_first) * dout).sum())

    g = ref.norm_after_grad(dout, a["x"], a["w"], a["z"], 2, a["scale"], 0.7, gate_first)
    _differences(loss, a, list(a), g)
