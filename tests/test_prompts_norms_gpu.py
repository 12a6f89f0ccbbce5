"""The norms before and after a block against their 64-bit definitions."""
import pytest
import torch

import oracle.prompts as ref
import selective_scan_fwd_amd as vm
from _prompts import DEV, DTYPES, close, dev, gen, host, randn, slices, tol_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if DEV is None:
        pytest.fail("GPU test run without a visible GPU")
    vm.load_library()
    print(f"[case] {request.node.name}", flush=True)


DIMS = [(1, 1), (3, 5), (5, 32), (7, 100), (3, 384), (2, 1000), (5, 2048), (3, 2056), (2, 5000), (2, 12000)]
TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("rows,dim", DIMS)
def test_before(rows, dim, center, dtype, rdtype):
    g = gen(dim)
    x, _ = slices([randn(g, rows, dim), randn(g, rows, 3)], DTYPES[dtype], strided=dim % 5 == 0)
    w, b, scale = dev(1 + 0.1 * randn(g, dim)), dev(0.1 * randn(g, dim)), dev(randn(g, dim))
    residual = dev(2 * randn(g, rows, dim) + 1, DTYPES[rdtype])
    use = dict(w=w if dim != 100 else None, b=b if dim % 2 == 0 else None, scale=scale if dim != 1000 else None,
               residual=residual if dim != 384 else None, factor=0.5 if dim != 2048 else 1.0, center=center)
    y, r = vm.vm_norm_before(x, **use)
    h = {k: host(v) if isinstance(v, torch.Tensor) else v for k, v in use.items()}
    wy, wr = ref.norm_before(host(x), **h)
    close(y, wy, tol_of(y), "y")
    close(r, wr, tol_of(r), "r")
    dy, dr = dev(randn(g, rows, dim), x.dtype), dev(randn(g, rows, dim), r.dtype)
    use.pop("residual"), h.pop("residual")
    d = vm.vm_norm_before_bwd(dy, r, dr=dr, x=x, **use)
    h.pop("b")
    want = ref.norm_before_grad(host(dy), host(r), dr=host(dr), x=host(x), **h)
    assert set(d) == {"residual", "x"} | {k for k in ("w", "b", "scale") if use[k] is not None}
    for k, v in d.items():
        close(v, want[k], tol_of(v, sums=k in ("w", "b", "scale")), k)


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("rows,dim,group,gains", [(1, 1, 1, 1), (3, 12, 4, 4), (5, 96, 32, 96), (7, 2048, 128, 128),
                                                  (300, 160, 80, 160), (3, 384, 384, 384), (2, 5000, 1000, 1000),
                                                  (3, 4100, 4100, 4100), (2, 33, 11, 11), (2, 12000, 12000, 12000)])
def test_after(rows, dim, group, gains, gate_first, dtype, rdtype):
    g = gen(dim + group)
    x, z, _ = slices([randn(g, rows, dim), randn(g, rows, dim), randn(g, rows, 7)], DTYPES[dtype], strided=dim % 3 == 0)
    z = None if dim == 33 and not gate_first else z
    use = dict(w=dev(1 + 0.1 * randn(g, gains)) if dim != 96 else None, z=z, group=group,
               scale=dev(randn(g, dim)) if dim != 384 else None, factor=0.5, gate_first=gate_first)
    residual = dev(randn(g, rows, dim), DTYPES[rdtype]) if dim != 2048 or dtype != rdtype else None
    out = vm.vm_norm_after(x, residual=residual, **use)
    h = {k: host(v) if isinstance(v, torch.Tensor) else v for k, v in use.items()}
    close(out, ref.norm_after(host(x), residual=host(residual), **h), tol_of(out), "out")
    dout = dev(randn(g, rows, dim), out.dtype)
    d = vm.vm_norm_after_bwd(dout, x, **use)
    want = ref.norm_after_grad(host(dout), host(x), **h)
    assert set(d) == {"x"} | {k for k in ("w", "z", "scale") if use[k] is not None}
    for k, v in d.items():
        close(v, want[k], tol_of(v, sums=k in ("w", "scale")), k)


def test_before_adds_in_place_and_keeps_nothing():
    g = gen(1)
    x, residual = dev(randn(g, 4, 6, 64), torch.bfloat16), dev(randn(g, 4, 6, 64))
    y0, r0 = vm.vm_norm_before(x, residual=residual)
    again = residual.clone()
    y1, r1 = vm.vm_norm_before(x, residual=again, r=again)
    assert r1 is again and torch.equal(r1, r0) and torch.equal(y1, y0)
    y2, r2 = vm.vm_norm_before(x, residual=residual, want_residual=False)
    assert r2 is None and torch.equal(y2, y0)
    out0 = vm.vm_norm_after(x, residual=residual, group=16)
    out1 = vm.vm_norm_after(x, residual=again.copy_(residual), group=16, out=again)
    assert out1 is again and torch.equal(out1, out0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_by_themselves(dtype):
    """A row of NaN or infinities, and a row of zeros, leave every other row alone."""
    g = gen(2)
    x, z = dev(randn(g, 6, 96), DTYPES[dtype]), dev(randn(g, 6, 96), DTYPES[dtype])
    bad = x.clone()
    bad[1], bad[4] = float("nan"), float("inf")
    bad[2] = 0
    keep = [0, 3, 5]
    for f in (lambda v: vm.vm_norm_before(v)[0], lambda v: vm.vm_norm_before(v, center=True)[0],
              lambda v: vm.vm_norm_after(v, z=z, group=32)):
        a, b = f(x), f(bad)
        assert torch.equal(a[keep], b[keep])
        assert (b[2] == 0).all() and torch.isnan(b[1]).all()


def test_a_mixer_between_its_norms():
    """norm before -> gated delta rule -> gated norm by heads, added to the residual: the gradients of the whole
    block against differences of its outputs in a random direction."""
    g = gen(5)
    b, l, h, d = 2, 70, 2, 16
    dim = h * d
    x, res = dev(randn(g, b, l, dim)), dev(randn(g, b, l, dim))
    w1, w2, scale = dev(1 + 0.1 * randn(g, dim)), dev(1 + 0.1 * randn(g, d)), dev(0.5 + 0.1 * randn(g, dim))
    W = [dev(randn(g, dim, dim) / dim ** 0.5) for _ in range(4)]
    gate, beta = dev(-randn(g, b, l, h).abs()), torch.sigmoid(dev(randn(g, b, l, h)))
    dout = dev(randn(g, b, l, dim))

    def forward(x):
        y, r = vm.vm_norm_before(x, w1, residual=res, scale=scale, factor=0.7)
        q, k, v, z = (y @ m for m in W)
        heads = lambda t: t.view(b, l, h, d)
        q, k = vm.vm_head_norm_rope(heads(q), heads(k), l2=True)
        o, _ = vm.vm_gated_delta_fwd(q, k, heads(v), gate, beta)
        return vm.vm_norm_after(o.view(b, l, dim), w2, z, group=d, residual=r), (y, r, q, k, v, z, o)

    out, (y, r, q, k, v, z, o) = forward(x)
    heads = lambda t: t.view(b, l, h, d)
    d2 = vm.vm_norm_after_bwd(dout, o.view(b, l, dim), w2, z, group=d)
    dd = vm.vm_gated_delta_bwd(q, k, heads(v), gate, beta, heads(d2["x"]))
    yq, yk = heads(y @ W[0]), heads(y @ W[1])
    dq, dk, _, _ = vm.vm_head_norm_rope_bwd(dd["q"], dd["k"], yq, yk, l2=True)
    dy = sum(t.reshape(b, l, dim) @ m.t() for t, m in zip((dq, dk, dd["v"], d2["z"]), W))
    got = vm.vm_norm_before_bwd(dy, r, w1, dr=dout, x=x, scale=scale, factor=0.7)
    way = dev(randn(g, b, l, dim))
    eps = 1e-2
    hi, lo = ((forward(x + s * eps * way)[0].double() * dout).sum() for s in (1, -1))
    diff, want = float((hi - lo) / (2 * eps)), float((got["x"].double() * way).sum())
    # the difference's own error: eps^2 of the third derivative and fp32 outputs (1e-6 of
    # sums of 4480 terms) over eps
    size = float(got["x"].norm() * way.norm()) / (b * l * dim) ** 0.5
    assert abs(diff - want) <= 2e-2 * size, (diff, want, size)
