"""examples/adapted_block.py end to end: the loss falls, the checkpoint is half
of bf16, and the block served in 8 bits agrees with the trained one up to the
8-bit rounding of its weight rows."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [12, 333])
def test_adapted_block(tokens):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("adapted_block", os.path.join(ROOT, "examples", "adapted_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out = m.main(tokens=tokens, steps=15)
    assert out["last_loss"] < 0.9 * out["first_loss"]
    assert out["bytes_kept"] == tokens * (1024 + 4) and out["bytes_bf16"] == tokens * 2048
    # a weight row's 8-bit step is a 127th of its largest of 1024 Gaussians
    # (about 3.3 standard deviations, so at most 5): an error of a step over
    # sqrt(12), 5 / 127 / 3.46 = 1.1 % of the row, and bf16 roundings
    assert out["served_rel_difference"] < 0.02
