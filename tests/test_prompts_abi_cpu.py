"""Argument checks of the prompt and token operators: each refusal is made on the host,
before any device is touched (the pointers here are addresses that nothing reads)."""
import ctypes

import pytest

import selective_scan_fwd_amd as vm

NULL, SHAPE, DTYPE, FLAG, ALIAS, UNSUPPORTED, ALLOC = 1, 2, 3, 4, 5, 6, 8
G = 1 << 32                       # addresses far apart


def at(i):
    return (i + 1) * G


@pytest.fixture(scope="module")
def lib():
    return vm.load_library()


def rows(**kw):
    base = dict(u=at(0), delta=at(1), A=at(2), B=at(3), C=at(4), D=at(5), delta_bias=at(6), z=at(7), u_stride=0,
                delta_stride=0, B_stride=0, C_stride=0, z_stride=0)
    base.update(kw)
    return vm.VmScanRows(*(base[k] for k, _ in vm.VmScanRows._fields_))


def scan(lib, p=None, q=None, h0=None, state=None, out=at(10), batch=2, L=8, dim=32, n=16, dtype=0, options=1, ws=None, wn=0):
    return lib.vm_prompt_scan(p if p is not None else rows(), q, h0, state, out, batch, L, dim, n, dtype, options, ws, wn, None)


def scan_bwd(lib, p=None, q=None, h0=None, dout=at(20), dstate=None, batch=2, L=8, dim=32, n=16, dtype=0, options=1, ws=None,
             wn=0, **kw):
    g = dict(du=at(21), ddelta=at(22), dA=at(23), dB=at(24), dC=at(25), dD=at(26), ddelta_bias=at(27), dz=at(28), dh0=None)
    g.update(kw)
    return lib.vm_prompt_scan_bwd(p if p is not None else rows(), q, h0, dout, dstate,
                                  vm.VmRowsGrad(*(g[k] for k, _ in vm.VmRowsGrad._fields_)), batch, L, dim, n, dtype, options,
                                  ws, wn, None)


def sequences(offsets=None, slots=None, fresh=None, n=2, n_slots=0):
    return vm.VmSequences(offsets, slots, fresh, n, n_slots)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=2)), (FLAG, dict(options=2)), (FLAG, dict(options=4)), (NULL, dict(p=rows(u=None))),
    (NULL, dict(p=rows(A=None))), (NULL, dict(p=rows(C=None))), (NULL, dict(out=None)), (SHAPE, dict(batch=0)),
    (SHAPE, dict(L=-1)), (SHAPE, dict(dim=0)), (SHAPE, dict(n=0)), (SHAPE, dict(p=rows(u_stride=31))),
    (SHAPE, dict(p=rows(B_stride=15))), (SHAPE, dict(p=rows(z_stride=-1))), (UNSUPPORTED, dict(n=17)),
    (UNSUPPORTED, dict(p=rows(delta_stride=1 << 23))), (UNSUPPORTED, dict(dim=(1 << 22) + 1)),
    (SHAPE, dict(q=sequences(n=3))), (SHAPE, dict(q=sequences(offsets=at(30)))), (SHAPE, dict(q=sequences(n=0))),
    (SHAPE, dict(q=sequences(slots=at(30), n_slots=0), state=at(11))),
    (ALIAS, dict(out=at(0))), (ALIAS, dict(out=at(2) + 64)), (ALIAS, dict(state=at(10) + 4)), (ALIAS, dict(state=at(4))),
    (ALIAS, dict(h0=at(11), state=at(11) + 64)), (ALIAS, dict(q=sequences(slots=at(10), n_slots=4), state=at(11))),
    (UNSUPPORTED, dict(batch=1 << 24, L=1)), (UNSUPPORTED, dict(batch=1 << 20, L=1, dim=4096)),
    (ALLOC, dict(batch=1, L=1 << 14, dim=16, ws=at(40), wn=1024)),
    (ALLOC, dict(batch=1, L=1 << 14, dim=16, ws=at(40) + 16, wn=1 << 30)),
])
def test_scan_refuses(lib, want, kw):
    assert scan(lib, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(dout=None)), (NULL, dict(du=None)), (NULL, dict(dA=None)), (NULL, dict(dB=None)), (NULL, dict(dz=None)),
    (NULL, dict(p=rows(z=None))), (FLAG, dict(options=2)), (FLAG, dict(q=sequences(slots=at(30), n_slots=2))),
    (FLAG, dict(q=sequences(fresh=at(30)))), (ALIAS, dict(du=at(0))), (ALIAS, dict(dB=at(25) + 4)), (ALIAS, dict(dD=at(5))),
    (ALIAS, dict(h0=at(31), dh0=at(31))), (ALLOC, dict(ws=at(40), wn=64)), (UNSUPPORTED, dict(n=17)),
])
def test_scan_backward_refuses(lib, want, kw):
    assert scan_bwd(lib, **kw) == want


def test_step_refuses(lib):
    def step(p=None, state=at(10), slots=at(11), out=at(12), batch=4, n_slots=6, dim=32, n=16, dtype=1, options=1):
        return lib.vm_token_scan(p if p is not None else rows(), state, slots, out, batch, n_slots, dim, n, dtype, options, None)

    assert step(state=None) == NULL and step(out=None) == NULL and step(p=rows(B=None)) == NULL
    assert step(slots=None, batch=7) == SHAPE and step(n_slots=0) == SHAPE and step(batch=0) == SHAPE
    assert step(out=at(10)) == ALIAS and step(state=at(0)) == ALIAS and step(state=at(11)) == ALIAS
    assert step(n=17) == UNSUPPORTED and step(options=2) == FLAG and step(dtype=5) == DTYPE
    assert step(batch=1 << 20, n_slots=1 << 20, dim=4096, n=1) == UNSUPPORTED


def test_conv_refuses(lib):
    def conv(q=None, x=at(0), xs=0, w=at(1), bias=at(2), h0=None, state=None, out=at(3), batch=2, L=8, dim=32, width=4, silu=1,
             dtype=0):
        return lib.vm_prompt_conv(q, x, xs, w, bias, h0, state, out, batch, L, dim, width, silu, dtype, None)

    assert conv(x=None) == NULL and conv(w=None) == NULL and conv(out=None) == NULL
    assert conv(dtype=-1) == DTYPE and conv(silu=2) == FLAG
    assert conv(width=1) == UNSUPPORTED and conv(width=5) == UNSUPPORTED and conv(dim=(1 << 22) + 1) == UNSUPPORTED
    assert conv(xs=16) == SHAPE and conv(L=0) == SHAPE and conv(q=sequences(n=5)) == SHAPE
    assert conv(out=at(0)) == ALIAS and conv(out=at(1)) == ALIAS and conv(state=at(0) + 8) == ALIAS
    assert conv(h0=at(5), state=at(5) + 8) == ALIAS
    assert conv(batch=1 << 18, L=1, dim=1 << 20) == UNSUPPORTED

    def bwd(q=None, x=at(0), dout=at(3), dstate=None, h0=None, ws=None, wn=0, width=4, **kw):
        g = dict(dx=at(4), dw=at(5), dbias=at(6), dh0=None)
        g.update(kw)
        return lib.vm_prompt_conv_bwd(q, x, 0, at(1), at(2), h0, dout, dstate, vm.VmConvGrad(g["dx"], g["dw"], g["dbias"], g["dh0"]),
                                      2, 8, 32, width, 1, 0, ws, wn, None)

    assert bwd(dout=None) == NULL and bwd(dx=None) == NULL and bwd(dw=None) == NULL
    assert bwd(q=sequences(slots=at(9), n_slots=2)) == FLAG and bwd(q=sequences(fresh=at(9))) == FLAG
    assert bwd(dx=at(3)) == ALIAS and bwd(dw=at(6)) == ALIAS and bwd(dh0=at(4)) == ALIAS
    assert bwd(ws=at(9), wn=16) == ALLOC and bwd(width=9) == UNSUPPORTED

    def step(x=at(0), state=at(1), slots=at(2), out=at(3), batch=2, n_slots=3, dim=32, width=4):
        return lib.vm_token_conv(x, 0, at(4), at(5), state, slots, out, batch, n_slots, dim, width, 1, 0, None)

    assert step(x=None) == NULL and step(state=None) == NULL and step(width=1) == UNSUPPORTED
    assert step(slots=None, batch=4) == SHAPE and step(n_slots=0) == SHAPE
    assert step(out=at(1)) == ALIAS and step(state=at(4)) == ALIAS


def test_norms_refuse(lib):
    def norm(**kw):
        base = dict(x=at(0), w=at(1), b=None, scale=at(2), z=None, x_stride=0, z_stride=0, w_dim=0, group=0, eps=1e-5,
                    factor=1.0, options=0)
        base.update(kw)
        return vm.VmBlockNorm(*(base[k] for k, _ in vm.VmBlockNorm._fields_))

    def before(p, residual=at(3), y=at(4), r=at(5), n=4, dim=64, dtype=1, rdtype=0):
        return lib.vm_norm_before(p, residual, y, r, n, dim, dtype, rdtype, None)

    def after(p, residual=at(3), out=at(4), n=4, dim=64, dtype=1, rdtype=0):
        return lib.vm_norm_after(p, residual, out, n, dim, dtype, rdtype, None)

    inf = float("inf")
    assert before(norm(x=None)) == NULL and before(norm(), y=None) == NULL and before(None) == NULL
    assert before(norm(), dtype=0, rdtype=1) == DTYPE and before(norm(), dtype=3) == DTYPE
    assert before(norm(options=8)) == FLAG and before(norm(z=at(9))) == FLAG and before(norm(group=32)) == FLAG
    assert before(norm(x_stride=63)) == SHAPE and before(norm(), n=0) == SHAPE
    assert before(norm(eps=-1.0)) == UNSUPPORTED and before(norm(eps=float("nan"))) == UNSUPPORTED
    assert before(norm(factor=inf)) == UNSUPPORTED and before(norm(), dim=16385) == UNSUPPORTED
    assert before(norm(), y=at(0)) == ALIAS and before(norm(), r=at(4)) == ALIAS and before(norm(), r=at(3) + 16) == ALIAS
    assert after(norm(options=4)) == FLAG and after(norm(b=at(9))) == FLAG and after(norm(options=8)) == NULL
    assert after(norm(group=48)) == SHAPE and after(norm(group=-1)) == SHAPE and after(norm(group=32, w_dim=16)) == SHAPE
    assert after(norm(), out=at(0)) == ALIAS and after(norm(z=at(9)), out=at(9) + 8) == ALIAS
    assert after(norm(), n=1 << 30, dim=64) == UNSUPPORTED

    def back(p, r=at(3), dy=at(4), dr=at(5), ws=None, wn=0, **kw):
        g = dict(dx=at(10), dresidual=at(11), dz=None, dw=at(12), db=None, dscale=at(13))
        g.update(kw)
        return lib.vm_norm_before_bwd(p, r, dy, dr, vm.VmNormGrad(*(g[k] for k, _ in vm.VmNormGrad._fields_)), 4, 64, 1, 0, ws, wn,
                                      None)

    assert back(norm(), r=None) == NULL and back(norm(), dy=None) == NULL and back(norm(), db=at(14)) == NULL
    assert back(norm(), dx=None, dresidual=None) == NULL and back(norm(w=None)) == NULL and back(norm(x=None)) == NULL
    assert back(norm(), dz=at(15)) == NULL and back(norm(), dx=at(4)) == ALIAS and back(norm(), dw=at(13)) == ALIAS
    assert back(norm(), ws=at(20), wn=8) == ALLOC

    def aback(p, dout=at(4), ws=None, wn=0, **kw):
        g = dict(dx=at(10), dresidual=None, dz=at(11), dw=at(12), db=None, dscale=at(13))
        g.update(kw)
        return lib.vm_norm_after_bwd(p, dout, vm.VmNormGrad(*(g[k] for k, _ in vm.VmNormGrad._fields_)), 4, 64, 1, 0, ws, wn, None)

    assert aback(norm()) == NULL and aback(norm(z=at(9)), dz=None) == NULL and aback(norm(z=at(9)), dresidual=at(14)) == NULL
    assert aback(norm(z=at(9)), dout=None) == NULL and aback(norm(z=at(9)), dx=at(9)) == ALIAS
    assert aback(norm(z=at(9), scale=None)) == NULL and aback(norm(z=at(9)), ws=at(20) + 1, wn=1 << 20) == ALLOC


def test_workspaces(lib):
    f = lib.vm_prompt_scan_workspace
    assert f(0, 8, 1, 8, 8, 0, 0) == -SHAPE and f(2, 8, 3, 8, 8, 0, 0) == -SHAPE and f(2, 8, 3, 8, 8, 1, 0) == -SHAPE
    assert f(1, 8, 3, 8, 17, 1, 1) == -UNSUPPORTED
    assert f(1, 8, 3, 8, 16, 1, 0) == 0 and f(1, 8, 3, 8, 16, 1, 1) > 0 and f(1, 1 << 14, 1, 16, 16, 0, 0) > 0
    assert lib.vm_prompt_conv_workspace(1, 8, 1, 8, 5, 0, 0) == -UNSUPPORTED
    assert lib.vm_prompt_conv_workspace(1, 8, 2, 8, 4, 0, 0) == -SHAPE and lib.vm_prompt_conv_workspace(1, 8, 2, 8, 4, 0, 1) > 0
    assert lib.vm_block_norm_workspace(4, 64, 48) == -SHAPE and lib.vm_block_norm_workspace(4, 1 << 15, 0) == -UNSUPPORTED
    assert lib.vm_block_norm_workspace(4, 64, 0) > 0


def test_structures_match_the_header():
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "vm_scan.h")).read()
    for cls, name in ((vm.VmSequences, "vm_sequences"), (vm.VmConvGrad, "vm_conv_grad"), (vm.VmScanRows, "vm_scan_rows"),
                      (vm.VmRowsGrad, "vm_rows_grad"), (vm.VmBlockNorm, "vm_block_norm"), (vm.VmNormGrad, "vm_norm_grad")):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        fields = re.findall(r"(\w+);", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
        assert fields == [k for k, _ in cls._fields_], name
        assert all(t in (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int32) for _, t in cls._fields_)
