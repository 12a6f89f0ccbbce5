"""The prompt and token operators at infinities, partial tiles and rows of no sequence, against their 64-bit
definitions: where those are infinite or no number, so are the outputs, and nowhere else.

Finite values are held to the tolerances of the other tests (their derivation stands beside them); the places of
infinities and of NaN have to be the same."""
import numpy as np
import pytest
import torch

import selective_scan_fwd_amd as vm
from _prompts import BF16, DEV, F32, SUMS, Scan, dev, host

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _need_gpu(request):
    if DEV is None:
        pytest.fail("GPU test run without a visible GPU")
    vm.load_library()
    print(f"[case] {request.node.name}", flush=True)


def same(got, want, tol, what):
    """Infinities and NaN in the same places; the rest close by Euclidean norms."""
    want, got = np.asarray(want, dtype=np.float64), host(got)
    assert got.shape == want.shape, what
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), f"{what}: {got[odd][:8]} for {want[odd][:8]}"
    assert np.isfinite(got[~odd]).all(), f"{what}: {(~np.isfinite(got[~odd])).sum()} finite values are not"
    size = np.sqrt((want[~odd] ** 2).sum())
    err = np.sqrt(((got[~odd] - want[~odd]) ** 2).sum())
    assert err <= tol * size, f"{what}: {err / size:.2e} > {tol:.1e}"


def tol(t, sums=False):
    return (BF16 if t.dtype == torch.bfloat16 else 0) + (SUMS if sums else F32)


def mild(s, rate=0.25):
    """Positive B and C (infinite states do not cancel in the read-out) and decays that no step takes below 2^-126."""
    s.a = dict(s.a, A=s.a["A"] * rate, B=s.a["B"].abs(), C=s.a["C"].abs())
    return s


def put(s, name, where, value):
    t = s.a[name].clone()
    t[where] = value
    s.a[name] = t


def check_forward(s, **kw):
    out, state = vm.vm_prompt_scan(**s.a, h0=s.h0, want_state=True, offsets=s.offsets)
    with np.errstate(all="ignore"):
        want, last, _ = s.ref(list(host(s.h0)))
    same(out, want, tol(out), "out")
    same(state, last, F32, "state")


def check_backward(s):
    d = vm.vm_prompt_scan_bwd(**s.a, dout=s.dout, h0=s.h0, dstate=s.dstate, offsets=s.offsets)
    with np.errstate(all="ignore"):
        want = s.ref_grad(list(host(s.h0)), list(host(s.dstate)))
    for k, v in d.items():
        same(v, want[k], tol(v, True), "d" + k)


# ----------------------------------------------------- chunks of a long row
def test_an_infinite_state_stays_infinite_over_chunks():
    """A chunk's decays may round to 0 together where no single one does: an infinite state before it stays."""
    assert vm.load_library().vm_prompt_scan_workspace(1, 700, 1, 16, 16, 0, 0) > 0
    s = mild(Scan(21, 1, 700, 16, 16, "f32", bias=False))
    s.a["A"] = torch.full((16, 16), -8.0, device=DEV)
    put(s, "u", (0, 3, 5), INF)
    check_forward(s)
    check_backward(s)
    s = mild(Scan(22, 1, 700, 16, 16, "f32", bias=False))
    s.a["A"] = torch.full((16, 16), -8.0, device=DEV)
    s.dstate[0, 4] = INF
    check_backward(s)
