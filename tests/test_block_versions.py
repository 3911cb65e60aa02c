"""Steps change their pools in place, and autograd can tell: a pool that it has saved is not differentiated at
values that it no longer has."""
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr

pytestmark = pytest.mark.gpu


def steps():
    """name: (a pool, a step on it)."""
    x, w = torch.ones(2, 16, device="cuda"), torch.ones(16, 4, device="cuda")
    A, bc = -torch.ones(16, 4, device="cuda"), torch.ones(2, 1, 4, device="cuda")
    q, g = torch.ones(2, 1, 16, device="cuda") / 4, torch.zeros(2, 1, device="cuda")
    return {"conv_step": (torch.ones(3, 3, 16, device="cuda"), lambda p: gdr.conv_step(x, p, w)),
            "ssm_step": (torch.ones(3, 16, 4, device="cuda"), lambda p: gdr.ssm_step(x, x, A, bc, bc, p)),
            "step": (torch.ones(3, 1, 16, 16, device="cuda"), lambda p: gdr.step(q, q, q, g, g, p))}


@pytest.mark.parametrize("name", ["conv_step", "ssm_step", "step"])
def test_a_saved_pool_is_missed(name):
    pool, call = steps()[name]
    was = pool._version
    scale = torch.ones((), device="cuda", requires_grad=True)
    loss = (pool * scale).sum()
    call(pool)
    assert pool._version > was
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("name", ["conv_step", "ssm_step", "step"])
def test_a_pool_of_inference_mode_has_no_version(name):
    with torch.inference_mode():
        pool, call = steps()[name]
        call(pool)
    call(pool)  # outside of it, too
    assert pool.is_inference()
