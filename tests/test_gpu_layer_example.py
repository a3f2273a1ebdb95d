"""The example that runs the layer operators and the rule together: whole prompts and
prompts in pieces beside decode rows give every token the same bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_hybrid_layers():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_layers.py")
    spec = importlib.util.spec_from_file_location("hybrid_layers", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    dev = torch.device("cuda", 0)
    whole, pieces = example.serve(dev, split=False), example.serve(dev, split=True)
    for a, b in zip(whole, pieces):
        assert torch.isfinite(a).all() and torch.equal(a, b)
