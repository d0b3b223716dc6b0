"""What the post-training example refuses before it takes up the GPU."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_fewer_tokens_than_a_pair_has():
    spec = importlib.util.spec_from_file_location("policy_mx4", os.path.join(ROOT, "examples", "policy_mx4.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    with pytest.raises(ValueError, match="32 tokens"):
        example.train(loss="preference", tokens=31)
