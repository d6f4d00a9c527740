"""The example trains (GPU): the linear layer's forward and backward with the
Muon step and with the Orth-Dion step lower the loss of a fixed teacher
problem.  A factor of two in 60 steps is far from either optimizer's rate
there and cannot be met by a gradient of the wrong sign, scale or layer."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_mlp.py")


@pytest.mark.parametrize("optimizer", ["muon", "dion"])
def test_example_trains(gpu_lib, optimizer):
    spec = importlib.util.spec_from_file_location("train_mlp", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(optimizer, steps=60)
    assert all(l == l for l in losses)
    assert sum(losses[-5:]) <= 0.5 * sum(losses[:5]), losses
    again = mod.train(optimizer, steps=8)
    assert again == losses[:8]      # the same bits from the same seed
