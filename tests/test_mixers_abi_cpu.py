"""Refusals of the matrix-state mixers' C ABI and of the Python binding: every
documented status, before anything is launched (no GPU is touched)."""
import ctypes
import os

import pytest
import torch

import selective_scan_fwd_amd as vm

FAKE = 1 << 40          # plausible-looking but never dereferenced device addresses
WIN = 1 << 32           # each tensor in a window of its own
NAN, INF = float("nan"), float("inf")
OK_SHAPE = dict(batch=2, L=5, n=2, hk=2, hv=4, dk=8, dv=6)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(vm.LIB_PATH):
        from selective_scan_fwd_amd import build
        build.build()
    return vm.load_library()


def _at(k):
    return FAKE + k * WIN


def _delta(h0=None, offsets=None, strides=(0, 0, 0), **null):
    p = vm.VmDelta(_at(0), _at(1), _at(2), _at(3), _at(4), h0, offsets, *strides)
    for k in null:
        setattr(p, k, None)
    return p


def _fwd(lib, p=None, out=_at(9), state=None, scale=1.0, dtype=0, reverse=0, ws=(None, 0), **more):
    s = {**OK_SHAPE, **more}
    return lib.vm_gated_delta_fwd(ctypes.byref(p if p is not None else _delta()), out, state, scale, s["batch"], s["L"],
                                  s["n"], s["hk"], s["hv"], s["dk"], s["dv"], dtype, reverse, *ws, None)


def _bwd(lib, p=None, dout=_at(10), dstate=None, g=None, scale=1.0, dtype=0, reverse=0, ws=(None, 0), **more):
    s = {**OK_SHAPE, **more}
    g = vm.VmDeltaGrad(*(_at(11 + i) for i in range(6))) if g is None else g
    return lib.vm_gated_delta_bwd(ctypes.byref(p if p is not None else _delta()), dout, dstate, ctypes.byref(g), scale,
                                  s["batch"], s["L"], s["n"], s["hk"], s["hv"], s["dk"], s["dv"], dtype, reverse, *ws, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_delta_refusals(lib, call):
    for name in ("q", "k", "v", "g", "beta"):
        assert call(lib, _delta(**{name: None})) == 1
    assert call(lib, dtype=2) == 3
    assert call(lib, reverse=2) == 4
    assert call(lib, scale=NAN) == 6 and call(lib, scale=INF) == 6
    for name in ("batch", "L", "hk", "hv", "dk", "dv", "n"):
        assert call(lib, **{name: 0}) == 2
        assert call(lib, **{name: -1}) == 2
    assert call(lib, hv=5) == 2                                     # not a multiple of the key heads
    assert call(lib, n=3) == 2                                      # sequences without offsets
    assert call(lib, _delta(offsets=_at(8)), batch=2) == 2          # packed sequences take batch 1
    assert call(lib, dk=129) == 6 and call(lib, dv=129) == 6
    assert call(lib, batch=1 << 24, n=1 << 24, L=1) == 6            # past the grid
    assert call(lib, batch=1 << 20, n=1 << 20, L=1 << 20) == 2      # elements overflow
    assert call(lib, _delta(strides=(15, 0, 0))) == 2               # shorter than a token's heads
    assert call(lib, _delta(strides=(0, -16, 0))) == 2
    assert call(lib, _delta(strides=(0, 0, 23))) == 2


def test_delta_forward_aliases(lib):
    assert _fwd(lib, out=None) == 1
    for k in range(5):
        assert _fwd(lib, out=_at(k)) == 5
        assert _fwd(lib, state=_at(k)) == 5
    assert _fwd(lib, state=_at(9) + 8) == 5                         # the outputs on each other
    assert _fwd(lib, _delta(h0=_at(7)), out=_at(7)) == 5
    assert _fwd(lib, _delta(h0=_at(7)), state=_at(7) + 4) == 5      # h0 in place only as a whole
    assert _fwd(lib, _delta(offsets=_at(8)), out=_at(8), batch=1) == 5
    # a strided row reaches past its dense size
    far = _at(2) + 4 * (9 * 1000)
    assert _fwd(lib, _delta(strides=(0, 0, 1000)), out=far) == 5


def test_delta_backward_aliases(lib):
    assert _bwd(lib, dout=None) == 1
    for name in ("dq", "dk", "dv", "dg", "dbeta"):
        g = vm.VmDeltaGrad(*(_at(11 + i) for i in range(6)))
        setattr(g, name, None)
        assert _bwd(lib, g=g) == 1
    for name in ("dq", "dk", "dv", "dg", "dbeta", "dh0"):
        for target in (_at(0), _at(3), _at(10), _at(11 if name != "dq" else 12)):
            g = vm.VmDeltaGrad(*(_at(11 + i) for i in range(6)))
            setattr(g, name, target)
            assert _bwd(lib, g=g) == 5, name


def _step(lib, dtype=0, scale=1.0, ptrs=None, batch=2, n_slots=3, hk=2, hv=4, dk=8, dv=6, **null):
    names = ["q", "k", "v", "g", "beta", "state", "slots", "out"]
    p = {n: _at(i) for i, n in enumerate(names)}
    p.update(ptrs or {})
    p.update(null)
    return lib.vm_gated_delta_step(*(p[n] for n in names), scale, batch, n_slots, hk, hv, dk, dv, dtype, None)


def test_step_refusals(lib):
    for name in ("q", "k", "v", "g", "beta", "state", "out"):
        assert _step(lib, **{name: None}) == 1
    assert _step(lib, dtype=-1) == 3
    for name in ("batch", "n_slots", "hk", "hv", "dk", "dv"):
        assert _step(lib, **{name: 0}) == 2
    assert _step(lib, hv=3) == 2
    assert _step(lib, slots=None, batch=4) == 2                     # more rows than states
    assert _step(lib, dk=129) == 6 and _step(lib, dv=200) == 6 and _step(lib, scale=NAN) == 6
    for name in ("q", "k", "v", "g", "beta", "slots", "out"):
        assert _step(lib, state=_step_at(name)) == 5
    for name in ("q", "k", "v", "g", "beta", "slots"):
        assert _step(lib, out=_step_at(name)) == 5


def _step_at(name):
    return _at(["q", "k", "v", "g", "beta", "state", "slots", "out"].index(name))


def _norm(lib, back=False, batch=2, L=3, hq=4, hk=2, dim=8, eps=1e-6, options=0, dtype=0, rot=4, table=9, stride=0,
          ws=(None, 0), **ptr):
    p = dict(q=_at(0), k=_at(1), wq=_at(2), wk=_at(3), cos=_at(4), sin=_at(5), positions=_at(6), qo=_at(7), ko=_at(8),
             dq=_at(9), dk=_at(10), dwq=_at(11), dwk=_at(12))
    p.update(ptr)
    h = vm.VmHeadNorm(p["q"], p["k"], p["wq"], p["wk"], p["cos"], p["sin"], p["positions"], stride, 0, table, rot)
    tail = (batch, L, hq, hk, dim, eps, options, dtype, None)
    if back:
        return lib.vm_head_norm_rope_bwd(ctypes.byref(h), p["qo"], p["ko"], p["dq"], p["dk"], p["dwq"], p["dwk"], *tail[:-1], *ws, None)
    return lib.vm_head_norm_rope(ctypes.byref(h), p["qo"], p["ko"], *tail)


@pytest.mark.parametrize("back", [False, True])
def test_head_norm_refusals(lib, back):
    assert _norm(lib, back, q=None) == 1 and _norm(lib, back, k=None) == 1 and _norm(lib, back, hk=0) == 1
    assert _norm(lib, back, qo=None) == 1 and _norm(lib, back, ko=None) == 1
    assert _norm(lib, back, cos=None) == 1 and _norm(lib, back, sin=None) == 1
    assert _norm(lib, back, dtype=5) == 3
    assert _norm(lib, back, options=4) == 4 and _norm(lib, back, options=-1) == 4
    for name in ("batch", "L", "hq", "dim"):
        assert _norm(lib, back, **{name: 0}) == 2
    assert _norm(lib, back, hk=-1) == 2
    assert _norm(lib, back, rot=3) == 2 and _norm(lib, back, rot=10) == 2 and _norm(lib, back, rot=-2) == 2
    assert _norm(lib, back, table=0) == 2
    assert _norm(lib, back, stride=31) == 2
    assert _norm(lib, back, dim=513) == 6
    assert _norm(lib, back, eps=NAN) == 6 and _norm(lib, back, eps=-1.0) == 6 and _norm(lib, back, eps=INF) == 6
    outs = ("dq", "dk", "dwq", "dwk") if back else ("qo", "ko")
    for name in outs:
        for k in range(7):
            assert _norm(lib, back, **{name: _at(k)}) == 5, (name, k)
    if back:
        assert _norm(lib, back, dq=None) == 1 and _norm(lib, back, dk=None) == 1
        assert _norm(lib, back, wq=None) == 1 and _norm(lib, back, wk=None) == 1    # a gain's gradient without it
        assert _norm(lib, back, dq=_at(7)) == 5 and _norm(lib, back, dq=_at(10)) == 5
    else:
        assert _norm(lib, back, qo=_at(8)) == 5


def test_clip_refusals(lib):
    def call(tensors, most=1.0, norm=_at(9), count=None, ws=(None, 0)):
        arr = (vm.VmGradTensor * max(1, len(tensors)))(*(vm.VmGradTensor(*t) for t in tensors))
        return lib.vm_clip_grad_norm(arr, len(tensors) if count is None else count, most, norm, *ws, None)

    good = (_at(0), _at(1), 10, 0)
    assert call([good], norm=None) == 1
    assert lib.vm_clip_grad_norm(None, 1, 1.0, _at(9), None, 0, None) == 1
    assert call([(None, _at(1), 10, 0)]) == 1
    assert call([good], count=-1) == 2
    assert call([(_at(0), _at(1), -1, 0)]) == 2
    assert call([(_at(0), _at(1), 10, 2)]) == 3
    assert call([good], most=-1.0) == 6 and call([good], most=NAN) == 6
    assert call([good], count=65537) == 6
    assert call([(_at(0), _at(0) + 8, 10, 0)]) == 5                 # partly on its own input
    assert call([good], norm=_at(1) + 4) == 5
    assert call([good], norm=_at(0)) == 5


def test_workspaces(lib):
    """Sizes from the _workspace functions; a workspace that is too small or not
    aligned is refused before anything is launched."""
    size = lib.vm_gated_delta_workspace(2, 5, 2, 4, 8, 6, 0, 0, 0)
    back = lib.vm_gated_delta_workspace(2, 5, 2, 4, 8, 6, 0, 0, 1)
    assert 0 < size < back
    assert lib.vm_gated_delta_workspace(1, 128, 3, 4, 8, 6, 0, 1, 0) > lib.vm_gated_delta_workspace(1, 128, 1, 4, 8, 6, 0, 0, 0)
    assert lib.vm_gated_delta_workspace(2, 0, 2, 4, 8, 6, 0, 0, 0) == -2
    assert _fwd(lib, ws=(_at(40), size - 1)) == 8 and _fwd(lib, ws=(_at(40) + 16, size + 64)) == 8
    assert _bwd(lib, ws=(_at(40), back - 1)) == 8 and _bwd(lib, ws=(_at(40) + 128, back + 128)) == 8
    size = lib.vm_head_norm_rope_workspace(8)
    assert size > 0
    assert _norm(lib, True, ws=(_at(40), size - 1)) == 8
    size = lib.vm_clip_grad_workspace(300)
    assert size >= lib.vm_clip_grad_workspace(0) > 0
    arr = (vm.VmGradTensor * 1)(vm.VmGradTensor(_at(0), _at(1), 10, 0))
    assert lib.vm_clip_grad_norm(arr, 1, 1.0, _at(9), _at(40), 7, None) == 8


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(1, 2, 1, 4)
    gate = torch.zeros(1, 2, 1)
    with pytest.raises(ValueError):
        vm.vm_gated_delta_fwd(x, x, x, gate, gate)
    with pytest.raises(ValueError):
        vm.vm_gated_delta_bwd(x, x, x, gate, gate, x)
    with pytest.raises(ValueError):
        vm.vm_gated_delta_step(x[0], x[0], x[0], gate[0], gate[0], torch.zeros(2, 1, 4, 4))
    with pytest.raises(ValueError):
        vm.vm_head_norm_rope(x)
    with pytest.raises(ValueError):
        vm.vm_head_norm_rope_bwd(x, None, x)
    with pytest.raises(ValueError):
        vm.vm_clip_grad_norm([x], 1.0)
    with pytest.raises(ValueError):
        vm.vm_clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        vm.vm_head_norm_rope(x[0])
    with pytest.raises(ValueError):
        vm.vm_gated_delta_fwd(x[0], x, x, gate, gate)
