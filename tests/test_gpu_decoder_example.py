"""The example decoder: products, cache, attention, experts and log probabilities
together; decoding by single tokens agrees with the prompt."""
import os
import runpy

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layers.py")


def test_decoding_agrees_with_the_prompt():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required")
    # fp16 activations through two layers and the head: some tens of roundings of 2^-11 on logits of a few units.
    assert runpy.run_path(PATH)["main"](prompts=(70, 5, 33), steps=3) < 0.1
