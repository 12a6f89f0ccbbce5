"""Clipping of long lists, whose tensors go to the kernels 120 at a time."""
import ctypes

import pytest
import torch

import selective_scan_fwd_amd as vm
from oracle import mixers
from test_mixers_gpu import BF16, DEV, F32, _case, close, host

pytestmark = pytest.mark.gpu


# few and small tensors first, then more, and the other way round: each launch has
# another number of workgroups
@pytest.mark.parametrize("order", [1, -1])
def test_launches_of_different_sizes(order):
    _case(f"clip launches of different sizes, order {order}")
    g = torch.Generator(device=DEV).manual_seed(71)
    sizes = ([3] * 120 + [70000] * 120 + [5000] * 125)[::order]
    grads = [torch.randn(n, generator=g, device=DEV).to(BF16 if i % 4 == 1 else F32) for i, n in enumerate(sizes)]
    rn, rc = mixers.clip([host(x) for x in grads], 2.5)
    again = [x.clone() for x in grads]
    norm = vm.vm_clip_grad_norm(grads, 2.5)
    assert abs(float(norm) - rn) <= 1e-6 * rn                       # (the sums are fp64, the result fp32)
    for x, r in zip(grads, rc):
        close(x, r, "clipped", tol=4e-3 if x.dtype == BF16 else 1e-6)
    assert torch.equal(norm, vm.vm_clip_grad_norm(again, 2.5)) and all(torch.equal(x, y) for x, y in zip(grads, again))


def test_a_list_takes_no_longer_than_its_parts():
    """6000 gradients of 2^20 elements (one buffer, counted again and again) in one
    call, against 50 calls over 120: the same work and as many launches.  Three
    times as long would mean launches that leave most of the card idle."""
    _case("clip of a long list against its parts")
    lib = vm.load_library()
    x = torch.randn(1 << 20, device=DEV)

    def calls(count, times):
        norm = torch.zeros((), device=DEV)
        arr = (vm.VmGradTensor * count)(*[vm.VmGradTensor(x.data_ptr(), None, x.numel(), vm.VM_F32)] * count)
        ws = torch.empty(lib.vm_clip_grad_workspace(count), dtype=torch.uint8, device=DEV)
        s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        best = float("inf")
        for _ in range(4):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(times):
                assert lib.vm_clip_grad_norm(arr, count, 1.0, norm.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end))
        want = float(x.double().norm()) * count ** 0.5
        assert abs(float(norm) / want - 1) < 1e-6
        return best

    parts, whole = calls(120, 50), calls(6000, 1)
    print(f"parts {parts:.2f} ms, whole {whole:.2f} ms")
    assert whole < 3 * parts
