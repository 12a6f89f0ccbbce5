"""The documented limits of the gated delta rule's calls, on both sides, without a
GPU: a size that is taken gets as far as its workspace, which is too small here
(VM_ERR_ALLOC, nothing launched); one past a limit is VM_ERR_UNSUPPORTED."""
import ctypes
import os

import pytest

import selective_scan_fwd_amd as vm

TAKEN, REFUSED = 8, 6
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(vm.LIB_PATH):
        from selective_scan_fwd_amd import build
        build.build()
    return vm.load_library()


def _at(k):
    return (k + 1) << 42                   # never dereferenced; far apart


def _call(lib, back, n, hv, dk, dv, dtype, packed=False, L=1, hk=1, shift=0):
    p = vm.VmDelta(_at(0) + shift, _at(1), _at(2), _at(3), _at(4), None, _at(5) if packed else None, 0, 0, 0)
    shape = (1 if packed else n, n * L if packed else L, n, hk, hv, dk, dv, dtype, 0, _at(30), 256, None)
    if not back:
        return lib.vm_gated_delta_fwd(ctypes.byref(p), _at(6), None, 1.0, *shape)
    g = vm.VmDeltaGrad(*(_at(7 + i) for i in range(5)), None)
    return lib.vm_gated_delta_bwd(ctypes.byref(p), _at(20), None, ctypes.byref(g), 1.0, *shape)


def _size(lib, back, n, hv, dk, dv, dtype):
    return lib.vm_gated_delta_workspace(n, 1, n, hv, dk, dv, dtype, 0, int(back))


# the backward scans of bf16 rows in whole pieces, keys past 64: n hv ceil(dv / 32) below 2^22
@pytest.mark.parametrize("n,hv,dv,status", [
    (2 ** 18, 4, 104, REFUSED), (2 ** 18 - 1, 4, 104, TAKEN), (2 ** 20, 1, 128, REFUSED), (2 ** 20 - 1, 1, 128, TAKEN),
    (1398102, 1, 96, REFUSED), (1398101, 1, 96, TAKEN), (2 ** 21 - 8, 1, 64, TAKEN), (2 ** 21 - 7, 1, 64, REFUSED)])
def test_backward_work_items(lib, n, hv, dv, status):
    assert _call(lib, True, n, hv, 72, dv, BF16) == status
    size = _size(lib, True, n, hv, 72, dv, BF16)
    assert size == -REFUSED if status == REFUSED else size > 0


def test_backward_work_items_of_packed_sequences(lib):
    # (heads in whole rounds of 8)
    assert _call(lib, True, 2 ** 20 - 8, 1, 72, 104, BF16, packed=True) == TAKEN
    assert _call(lib, True, 2 ** 20 - 7, 1, 72, 104, BF16, packed=True) == REFUSED
    assert _call(lib, True, 2 ** 21 - 8, 1, 72, 104, F32, packed=True) == TAKEN


@pytest.mark.parametrize("back,dk,dtype,shift", [(False, 128, BF16, 0), (False, 128, F32, 0), (False, 64, BF16, 0),
                                                 (True, 64, BF16, 0), (True, 128, F32, 0), (True, 72, BF16, 2),
                                                 (True, 70, BF16, 0)])
def test_other_scans_hold_the_whole_range(lib, back, dk, dtype, shift):
    assert _call(lib, back, 2 ** 21 - 8, 1, dk, 128, dtype, shift=shift) == TAKEN
    assert _call(lib, back, 2 ** 21 - 7, 1, dk, 128, dtype, shift=shift) == REFUSED


def test_workspace_refuses_what_the_calls_refuse(lib):
    size = lib.vm_gated_delta_workspace
    for back in (0, 1):
        assert size(2 ** 21, 1, 2 ** 21, 1, 8, 8, F32, 0, back) == -6          # scans
        assert size(1, 5, 1, 65536, 1, 1, F32, 0, back) == -6                  # heads
        assert size(1, (2 ** 23 - 1) * 64 + 1, 1, 1, 8, 8, F32, 0, back) == -6   # chunks
        assert size(1, (2 ** 23 - 1) * 64, 1, 1, 8, 8, F32, 0, back) > 0
        assert size(3, 5, 2, 1, 8, 8, F32, 0, back) == -2                      # n without offsets
        assert size(2, 5, 2, 1, 8, 8, F32, 1, back) == -2                      # packed rows
