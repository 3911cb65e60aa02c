"""Delay injection for the hand-overs of the attention mixer that test_attn_delay's cases leave out: the step's copies, warps and joins in a
stage, the tiles that a cluster's blocks share, and the fp32 kernels."""
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr
from chunked_gated_delta_04_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def delay_lib():
    return gbuild.build(delay=True)


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


STEPS = [  # lengths, page size, query heads, key heads, D, window, off 16 bytes
    ([5000], 64, 4, 1, 128, 0, False),                               # a unit in many blocks
    ([(53 * i) % 400 for i in range(200)], 16, 4, 2, 64, 0, False),  # many units in a block
    ([700, 0, 1, 63, 64, 65, 3000], 100, 40, 2, 96, 0, False),       # three units of a key head
    ([1500, 90, 4000], 32, 6, 2, 128, 333, False),
    ([300, 17, 64], 7, 4, 2, 48, 0, True),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths,size,Hq,Hk,D,window,off", STEPS)
def test_delayed_steps_give_bitwise_identical_results(delay_lib, dtype, lengths, size, Hq, Hk, D, window, off):
    g = torch.Generator().manual_seed(2)
    r = lambda *shape: torch.randn(*shape, generator=g).to(dtype).cuda()
    B, wide = len(lengths), max(lengths) // size + 1
    table = torch.randperm(B * wide, generator=g).view(B, wide).to(torch.int32).cuda()
    lens = torch.tensor(lengths, dtype=torch.int32).cuda()
    new = [r(B, Hq, D), r(B, Hk, D), r(B, Hk, D)]
    if off:
        new = [torch.empty(t.numel() + 1, dtype=dtype, device="cuda")[1:].view(t.shape).copy_(t) for t in new]
    held = r(B * wide, size, Hk, D), r(B * wide, size, Hk, D)

    def run():
        kc, vc = (t.clone() for t in held)
        ws = gdr.attn_step_workspace(new[0], kc, table)
        o = gdr.attn_step(*new, kc, vc, table, lens, window=window, workspace=ws)
        assert gdr.gdr_workspace_status(ws) == (gdr.GDR_OK, 0)
        return o, kc, vc

    want = run()
    assert torch.isfinite(want[0]).all()
    with gdr.library(delay_lib):
        for _ in range(3):
            assert all(same_bits(a, b) for a, b in zip(run(), want))


@pytest.mark.parametrize("dtype,n,m,Hq,Hk,D,window,lens", [
    (BF, 1, 3000, 2, 1, 64, 0, None), (BF, 640, 640, 8, 1, 128, 0, None), (BF, 515, 1800, 8, 8, 64, 700, None),
    (BF, 0, 0, 2, 1, 96, 0, [300, 0, 900]), (F32, 700, 900, 4, 2, 64, 0, None), (F32, 300, 300, 40, 20, 64, 0, None),
    (F32, 500, 500, 2, 1, 128, 200, None), (F32, 0, 0, 2, 1, 80, 0, [300, 1, 0, 430])])
def test_delayed_blocks_give_bitwise_identical_results(delay_lib, dtype, n, m, Hq, Hk, D, window, lens):
    g = torch.Generator().manual_seed(3)
    n, m = (sum(lens), sum(lens)) if lens else (n, m)
    q, k, v, do = (torch.randn(1, t, h, D, generator=g).to(dtype).cuda() for t, h in ((n, Hq), (m, Hk), (m, Hk), (n, Hq)))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if lens else None
    how = dict(cu_seqlens=cu, window=window)

    def run():
        ws = gdr.attn_workspace(q, k, cu), gdr.attn_workspace(q, k, cu, backward=True)
        o, lse = gdr.attn_forward(q, k, v, **how, workspace=ws[0])
        grads = gdr.attn_backward(q, k, v, o, lse, do, **how, workspace=ws[1])
        assert [gdr.gdr_workspace_status(w) for w in ws] == [(gdr.GDR_OK, 0)] * 2
        return [o, lse, *grads]

    want = run()
    with gdr.library(delay_lib):
        for _ in range(3):
            assert all(same_bits(a, b) for a, b in zip(run(), want))
