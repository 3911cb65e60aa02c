"""The example model runs the operators together: it learns, and its single-token path gives the logits
of its whole-sequence path."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hybrid():
    spec = importlib.util.spec_from_file_location("hybrid_block", os.path.join(ROOT, "examples", "hybrid_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype,bound", [
    (torch.float32, 1e-3),   # four layers at the delta rule's fp32 bound (1e-4) with room for their products
    (torch.bfloat16, 8e-2),  # activations rounded to 2^-8 at about 20 places in a row: sqrt(20) * 2^-8 = 1.7e-2, times up to 4 layers
])
def test_trained_model_serves_what_it_computes(hybrid, dtype, bound):
    torch.manual_seed(0)
    model = hybrid.HybridModel(dtype=dtype).cuda()
    losses = hybrid.train(model, 60, 64)
    assert all(l == l for l in losses) and sum(losses[-3:]) < 0.7 * sum(losses[:3])
    _, diff = hybrid.serve(model, 64)
    assert diff <= bound
