"""Refusals at the edges of the prompt and token operators: made on the host, before any
device is touched (the pointers here are addresses that nothing reads)."""
import pytest

import selective_scan_fwd_amd as vm

NULL, FLAG, ALIAS, UNSUPPORTED = 1, 4, 5, 6


def at(i):
    return (i + 1) << 32          # addresses far apart


@pytest.fixture(scope="module")
def lib():
    return vm.load_library()


def rows(**kw):
    base = dict(u=at(0), delta=at(1), A=at(2), B=at(3), C=at(4), D=at(5), delta_bias=at(6), z=at(7), u_stride=0,
                delta_stride=0, B_stride=0, C_stride=0, z_stride=0)
    base.update(kw)
    return vm.VmScanRows(*(base[k] for k, _ in vm.VmScanRows._fields_))


def token_scan(lib, p, out=at(12), options=1):
    return lib.vm_token_scan(p, at(10), at(11), out, 4, 6, 32, 16, 1, options, None)


def test_the_rest_of_a_packed_row_is_cleared_only_where_there_is_one(lib):
    clear = vm.VM_CLEAR_REST

    def scan(options, out):
        return lib.vm_prompt_scan(rows(), None, None, None, out, 2, 8, 32, 16, 0, options, None, 0, None)

    def conv(silu, out):
        return lib.vm_prompt_conv(None, at(0), 0, at(1), at(2), None, None, out, 2, 8, 32, 4, silu, 0, None)

    # (taken by the calls on prompts, whose next check then fails; refused by those on single tokens)
    assert scan(clear, None) == NULL and scan(1 | clear, None) == NULL and scan(2 | clear, None) == FLAG
    assert conv(clear, None) == NULL and conv(1 | clear, None) == NULL and conv(2 | clear, None) == FLAG
    assert token_scan(lib, rows(), options=clear) == FLAG and token_scan(lib, rows(), options=1 | clear) == FLAG
    assert lib.vm_token_conv(at(0), 0, at(4), at(5), at(1), at(2), at(3), 2, 3, 32, 4, 1 | clear, 0, None) == FLAG


def test_rows_of_single_tokens_may_lie_far_apart(lib):
    """Only prompts have a limit on token strides (the call then fails at its next check, that of overlaps)."""
    for name in ("u_stride", "delta_stride", "B_stride", "C_stride", "z_stride"):
        far = rows(**{name: 1 << 27})
        assert token_scan(lib, far, out=at(10)) == ALIAS
        assert lib.vm_prompt_scan(far, None, None, None, at(12), 2, 8, 32, 16, 0, 1, None, 0, None) == UNSUPPORTED
    # the rows' whole extent is what must not meet an output
    assert token_scan(lib, rows(u_stride=1 << 30), out=at(0) + 2 * 3 * (1 << 30)) == ALIAS
