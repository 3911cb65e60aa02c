"""The workspace that a packed call is handed tells, after it, whether its cu_seqlens was well formed."""
import ctypes

import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr

BF = torch.bfloat16


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_workspace_sizes(backward, packed):
    """What the helpers allocate is what the library asks for, and its status word is clear."""
    lib, way = gdr.load(), "bwd" if backward else "fwd"
    B = 1 if packed else 3
    cu = torch.tensor([0, 5, 40], dtype=torch.int32) if packed else None
    n, at = (2, cu.data_ptr()) if packed else (3, None)
    x, w, Bm = torch.zeros(B, 40, 24, dtype=BF), torch.zeros(24, 4), torch.zeros(B, 40, 2, 16, dtype=BF)
    for ws, p, name in ((gdr.conv_workspace(x, w, cu, backward), gdr.gdr_conv_problem(B, 40, 24, 4, n, at, 1), "conv"),
                        (gdr.ssm_workspace(x, Bm, cu, backward), gdr.gdr_ssm_problem(B, 40, 24, 16, 2, n, at, 1), "ssm")):
        need = getattr(lib, f"gdr_{name}_{way}_workspace_bytes")(ctypes.byref(p))
        assert ws.dtype == torch.uint8 and ws.numel() == max(need, 256) and not ws[:256].any()


def calls(cu):
    """name: (the call, its workspace), on tensors of ones."""
    x, w = torch.ones(1, 10, 8, device="cuda"), torch.ones(8, 4, device="cuda")
    A, bc = -torch.ones(8, 4, device="cuda"), torch.ones(1, 10, 1, 4, device="cuda")
    p = gdr.gdr_ssm_problem(1, 10, 8, 4, 1, cu.numel() - 1, cu.data_ptr(), 0)
    saved = torch.zeros(gdr.load().gdr_ssm_saved_bytes(ctypes.byref(p)) // 4, device="cuda")
    return {
        "conv_forward": (lambda ws: gdr.conv_forward(x, w, cu_seqlens=cu, workspace=ws), gdr.conv_workspace(x, w, cu)),
        "conv_backward": (lambda ws: gdr.conv_backward(x, w, None, x, cu_seqlens=cu, workspace=ws), gdr.conv_workspace(x, w, cu, True)),
        "causal_conv": (lambda ws: gdr.causal_conv(x, w, cu_seqlens=cu, workspace=ws), gdr.conv_workspace(x, w, cu)),
        "ssm_forward": (lambda ws: gdr.ssm_forward(x, x, A, bc, bc, cu_seqlens=cu, workspace=ws), gdr.ssm_workspace(x, bc, cu)),
        "ssm_backward": (lambda ws: gdr.ssm_backward(x, x, A, bc, bc, saved, x, cu_seqlens=cu, workspace=ws), gdr.ssm_workspace(x, bc, cu, True)),
        "selective_scan": (lambda ws: gdr.selective_scan(x, x, A, bc, bc, cu_seqlens=cu, workspace=ws), gdr.ssm_workspace(x, bc, cu)),
    }


NAMES = ["conv_forward", "conv_backward", "causal_conv", "ssm_forward", "ssm_backward", "selective_scan"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_a_malformed_cu_seqlens_can_be_seen(name):
    for cu, well in (([0, 5, 10], True), ([0, 5, 3, 10], False), ([1, 5, 10], False), ([0, 5, 9], False)):
        call, ws = calls(torch.tensor(cu, dtype=torch.int32, device="cuda"))[name]
        call(ws)
        status, flags = gdr.gdr_workspace_status(ws)
        assert (status, flags & 1) == ((gdr.GDR_OK, 0) if well else (gdr.GDR_ERR_INVALID_ARG, 1)), cu


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_the_workspace_handed_in_changes_no_result(name):
    call, ws = calls(torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda"))[name]
    for a, b in zip(call(ws), call(None)):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


@pytest.mark.gpu
def test_workspace_refusals():
    x, w = torch.ones(1, 10, 8, device="cuda"), torch.ones(8, 4, device="cuda")
    cu = torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda")
    ws = gdr.conv_workspace(x, w, cu)
    with pytest.raises(gdr.GDRError) as e:
        gdr.conv_forward(x, w, cu_seqlens=cu, workspace=ws[:255])
    assert e.value.status == gdr.GDR_ERR_WORKSPACE
    with pytest.raises(gdr.GDRError) as e:
        gdr.conv_backward(x, w, None, x, cu_seqlens=cu, workspace=gdr.conv_workspace(x, w, cu, True)[16:])
    assert e.value.status == gdr.GDR_ERR_ALIGNMENT
    with pytest.raises(ValueError, match="workspace: expected a contiguous CUDA tensor"):
        gdr.conv_forward(x, w, cu_seqlens=cu, workspace=ws.cpu())
    # a fixed-length call has no cu_seqlens to check: the status stays clear
    gdr.conv_forward(x, w, workspace=ws)
    assert gdr.gdr_workspace_status(ws) == (gdr.GDR_OK, 0)
