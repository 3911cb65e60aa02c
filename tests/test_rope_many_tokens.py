"""Rotary positions where the threads that pass features on are more than 32 bits count, though those that rotate are not."""
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr

pytestmark = pytest.mark.gpu


def test_the_last_tokens_features_are_passed_on():
    """Two features of 1024 are turned, so that 511 threads of a token pass the others on: 2^32 and more of them."""
    D, tokens, tail = 1024, (1 << 32) // 511 + 5000, 6000
    q = torch.ones(1, tokens, 1, D, dtype=torch.bfloat16, device="cuda")
    stale = torch.full((1, tokens, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    q[:, -tail:] = torch.randn(1, tail, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    freqs, _ = gdr.rope_frequencies(2)
    del stale  # the output comes to lie there
    out, none = gdr.rope_forward(q, None, freqs)
    assert none is None
    same = [bool((a[..., 2:] == b[..., 2:]).all()) for a, b in zip(out.split(1 << 20, 1), q.split(1 << 20, 1))]
    assert all(same)
    few, _ = gdr.rope_forward(q[:, -tail:], None, freqs, torch.arange(tokens - tail, tokens, dtype=torch.int32, device="cuda")[None])
    assert torch.equal(out[:, -tail:], few)
