"""The fine-tuning example learns: its loss falls well below the frozen
layer's, which the base's quantization alone (a share of about 2^-4.5 of each
weight, squared) does not explain away."""
import pytest

from examples.finetune_8bit import finetune
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu


def test_example_learns():
    say("finetune example")
    losses = finetune(steps=60, tokens=256, features=256, rank=8)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.35 * losses[0], losses
