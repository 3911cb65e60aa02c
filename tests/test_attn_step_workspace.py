"""The status of a step can be asked for, as that of the attention mixer's other calls: in a workspace of the caller's."""
import ctypes

import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr

F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32


def test_sizes():
    q, cache, table = torch.zeros(3, 8, 64, dtype=BF), torch.zeros(5, 16, 2, 64, dtype=BF), torch.zeros(3, 4, dtype=I32)
    ws = gdr.attn_step_workspace(q, cache, table)
    p = gdr.gdr_cache_problem(3, 1, 8, 2, 64, 5, 16, 4, None, gdr.GDR_DTYPE_BF16)
    assert ws.numel() == gdr.load().gdr_attn_step_workspace_bytes(ctypes.byref(p)) > 256 and not ws[:256].any()


def rows(dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, generator=g).to(dtype).cuda()
    table = torch.randperm(40, generator=g).to(I32).view(2, 20).cuda()
    return [r(2, 8, 64), r(2, 2, 64), r(2, 2, 64), r(40, 16, 2, 64), r(40, 16, 2, 64), table, torch.tensor([300, 7], dtype=I32).cuda()]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_the_status_is_the_last_calls(dtype):
    args = rows(dtype, 1)
    want = gdr.attn_step(*args)
    ws = gdr.attn_step_workspace(args[0], args[3], args[5])
    for _ in range(2):
        assert torch.equal(gdr.attn_step(*args, workspace=ws), want)
        assert gdr.gdr_workspace_status(ws) == (gdr.GDR_OK, 0)
    ws[:4].view(I32).fill_(2)  # what a wait that ran out in an earlier call left
    assert gdr.gdr_workspace_status(ws)[0] != gdr.GDR_OK
    assert torch.equal(gdr.attn_step(*args, workspace=ws), want)
    assert gdr.gdr_workspace_status(ws) == (gdr.GDR_OK, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdr.attn_step(*args, stream=side, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_a_small_or_other_workspace_is_refused():
    args = rows(BF, 2)
    before = args[3].clone()
    ws = gdr.attn_step_workspace(args[0], args[3], args[5])
    with pytest.raises(gdr.GDRError) as error:
        gdr.attn_step(*args, workspace=ws[:-1])
    assert error.value.status == gdr.GDR_ERR_WORKSPACE
    with pytest.raises(ValueError, match="^workspace: expected a contiguous CUDA tensor"):
        gdr.attn_step(*args, workspace=ws.cpu())
    assert torch.equal(args[3], before)
