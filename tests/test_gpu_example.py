"""The example runs training, clipping and generation together: the loss falls,
and the decode step agrees with the batch layer to bf16's rounding (2e-2 of the
largest value, the layer tests' tolerance)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_train_and_generate():
    import train_and_generate as example
    losses, states, off = example.main(["--steps", "40", "--tokens", "6", "--sequences", "3"])
    assert losses[-1] < losses[0]
    assert states.shape == (7, 3, example.D) and torch.isfinite(states.float()).all()
    assert off <= 2e-2
