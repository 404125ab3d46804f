"""The example model's caches: a prompt in pieces gives what the whole prompt gives."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_model.py")


def test_prompts_in_pieces():
    spec = importlib.util.spec_from_file_location("hybrid_model", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    torch.manual_seed(0)
    model = ex.Model()
    with torch.no_grad():
        for mixer in model.mixers:  # (as initialised the mixers hardly show beside the embedding)
            mixer.out.weight.mul_(20)
    tokens = ex.batch(2, 60, 64, torch.Generator().manual_seed(3))
    with torch.no_grad():
        whole = model(tokens)
        states = [{} for _ in model.mixers]
        parts = [model(tokens[:, a:b], None, states) for a, b in ((0, 25), (25, 58), (58, 59), (59, 60))]
    got = torch.cat(parts, 1).float()
    # bf16 activations through three blocks, in two orders of summation: some twenty roundings of 2^-9
    assert float((got - whole.float()).norm() / whole.float().norm()) < 0.05
