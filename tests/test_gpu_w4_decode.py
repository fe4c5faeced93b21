"""The 4-bit operators together: the decoding example at small sizes."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(gpu_lib):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "w4_decode.py")
    spec = importlib.util.spec_from_file_location("w4_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens", [1, 3, 20])
def test_decode_steps(example, tokens):
    """Two layers round their results and the normalised x to bf16, each 2^-9 of its values
    in the mean, and pass that on: ten such steps at most, added up.  A router logit is off
    by as much of the logits' spread (about 1), and so is a probability of itself."""
    off, missed, out = example.main(["--tokens", str(tokens), "--steps", "4", "--layers", "2", "--hidden",
                             "256", "--inter", "160", "--experts", "12", "--topk", "3", "--vocab",
                             "1000", "--group", "64"])
    assert off <= 10 * 2.0 ** -9
    assert missed <= 2 * 10 * 2.0 ** -9
    assert out.shape == (4, tokens) and (out >= 0).all() and (out < 1000).all()


def test_decode_is_what_steps_by_hand_give(example):
    model = example.Model(2, 256, 96, 8, 2, 500, 32)
    tokens, _ = example.decode(model, 5, 3)
    ids, plan = torch.arange(5, device="cuda"), model.plan(5)
    for i in range(3):
        ids = model.step(ids, plan).argmax(-1)
        assert torch.equal(ids, tokens[i])
