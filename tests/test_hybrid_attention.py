"""The example model with attention layers: its single-token path gives the logits of its whole-sequence path, and the attention
mixer's gradients are those of the same mixer written in plain torch in 64 bits."""
import importlib.util
import math
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
@pytest.mark.parametrize("every", [1, 2])
def test_steps_are_the_whole_sequences(hybrid, dtype, bound, every):
    torch.manual_seed(0)
    model = hybrid.HybridModel(dtype=dtype, attention=every).cuda()
    losses = hybrid.train(model, 3, 64)
    assert all(math.isfinite(x) for x in losses)
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in model.parameters())
    seq, diff = hybrid.serve(model, 64)
    assert seq.shape == (5, 61) and diff <= bound


def plain(mixer, x):
    """AttentionMixer.forward from its definition."""
    B, T, _ = x.shape
    q, k, v = (x @ mixer.proj.weight.double().T).unflatten(-1, (-1, mixer.D)).split(mixer.sizes, -2)
    angle = torch.arange(T, device=x.device).double()[:, None, None] * mixer.freqs
    n = len(mixer.freqs)

    def turn(t):
        a, b = t[..., :n], t[..., n:2 * n]
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin(), t[..., 2 * n:]], -1)

    q, k, v = (t.repeat_interleave(mixer.Hq // t.shape[2], 2).transpose(1, 2) for t in (turn(q), turn(k), v))
    s = q @ k.transpose(-1, -2) / math.sqrt(mixer.D)
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=x.device).triu(1), -math.inf)
    return (s.softmax(-1) @ v).transpose(1, 2).flatten(-2) @ mixer.out.weight.double().T


def test_gradients_of_the_attention_mixer(hybrid):
    torch.manual_seed(1)
    mixer = hybrid.AttentionMixer(64, 2, 32).cuda()
    x, dy = torch.randn(3, 75, 64, device="cuda", requires_grad=True), torch.randn(3, 75, 64, device="cuda")
    leaves = [x, mixer.proj.weight, mixer.out.weight]
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        y = mixer(x)
        got = torch.autograd.grad(y, leaves, dy)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = old
    xd = x.detach().double().requires_grad_()
    ref = plain(mixer, xd)
    want = torch.autograd.grad(ref, [xd, mixer.proj.weight, mixer.out.weight], dy.double())
    # sums of up to 225 terms in 32 bits behind three products: 1e-5 of the largest value
    for a, b in zip((y, *got), (ref, *want)):
        assert (a.double() - b).abs().max() <= 1e-5 * b.abs().max()
