"""The example model: decoding step by step agrees with the whole prompt, and training steps lower the loss."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    import recurrent_model
    return recurrent_model


@pytest.mark.parametrize("kinds", [("delta",), ("ssm",), ("delta", "ssm", "ssm", "delta")])
def test_decoding_goes_on_from_packed_prompts(example, kinds):
    # bf16 activations between two orders of the same sums, an e4m3 step (2^-4 of a value) where a rounding falls on the
    # other side: a few percent of the largest logit
    gap, top = example.decode_gap(example.Model(kinds))
    assert gap <= 0.05 * top


def test_training_lowers_the_loss(example):
    losses = example.train(example.Model(), steps=30)
    assert all(torch.isfinite(torch.tensor(losses))) and losses[-1] < 0.8 * losses[0]

