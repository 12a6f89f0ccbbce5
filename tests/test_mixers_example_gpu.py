"""The mixer operators together, as examples/gated_delta_mixer.py runs them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_delta_mixer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_delta_mixer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trains_and_serves(example):
    print("[case] mixer example", flush=True)
    layer, losses, norms = example.train(20)
    assert all(x > 0 and x == x for x in norms)
    assert sum(losses[-5:]) < 0.9 * sum(losses[:5])
    # bf16 outputs are rounded to 8 bits before the projection back, once each way
    assert example.serve(layer) < 2 ** -6


def test_gradients_agree_with_differences(example):
    """The whole layer in fp32: the loss along one direction of all weights, by
    central differences, against the gradients through the operators.  Step h:
    the loss's rounding of 2^-22 relative over 2 h, and h^2 of curvature."""
    print("[case] mixer example differences", flush=True)
    layer = example.Mixer(32, hk=1, hv=2, dk=16, dv=12, positions=70, dtype=torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(2, 70, 32, device="cuda", generator=gen)
    aim = torch.randn(2, 70, 32, device="cuda", generator=gen)
    weights = list(layer.w.values())
    way = [torch.randn(w.shape, device="cuda", generator=gen) / w.numel() ** 0.5 for w in weights]
    for reverse in (False, True):
        loss = lambda: (layer.forward(x, reverse).double() * aim.double()).mean()
        grads = torch.autograd.grad(loss(), weights)
        along = sum(float((g.double() * d.double()).sum()) for g, d in zip(grads, way))
        h, ends = 2e-3, []
        with torch.no_grad():
            for sign in (1, -1):
                for w, d in zip(weights, way):
                    w += sign * h * d
                ends.append(float(loss()))
                for w, d in zip(weights, way):
                    w -= sign * h * d
        assert abs((ends[0] - ends[1]) / (2 * h) - along) < 2e-2 * abs(along) + 1e-5
