"""The example that runs the 4-bit operators, the distillation loss and the ZeRO step together learns."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("distill_mx4", os.path.join(ROOT, "examples", "distill_mx4.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(tokens=300, dim=256, vocab=1001, top=16, steps=40, report=lambda _: None)
    assert all(x == x for x in losses)
    assert losses[-1] < 0.7 * losses[0], losses  # the first step's logits know nothing of the teacher
