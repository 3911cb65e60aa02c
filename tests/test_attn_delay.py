"""Delay injection for the attention kernels (see test_delay_injection): one role late at each hand-off changes no bit, and no
wait runs out.  A step's gradients of the scores may be ready before the product of the step before has been issued: a barrier
that both steps share would then be two phases on when it is waited for, which never ends."""
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr
from chunked_gated_delta_04_gb300 import build as gbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def delay_lib():
    return gbuild.build(delay=True)


CASES = [  # queries, keys, query heads, key heads, D, window, lengths of a packed batch
    (1500, 1500, 4, 4, 128, 0, None), (700, 900, 8, 2, 64, 0, None), (1000, 1000, 2, 1, 96, 200, None), (300, 300, 64, 16, 128, 0, None),
    (0, 0, 4, 2, 128, 0, [700, 1, 0, 130, 512])]


@pytest.mark.parametrize("n,m,Hq,Hk,D,window,lens", CASES)
def test_delayed_roles_give_bitwise_identical_results(delay_lib, n, m, Hq, Hk, D, window, lens):
    g = torch.Generator().manual_seed(1)
    B, n, m = (1, sum(lens), sum(lens)) if lens else (2, n, m)
    q, k, v, do = (torch.randn(B, t, h, D, generator=g).bfloat16().cuda() for t, h in ((n, Hq), (m, Hk), (m, Hk), (n, Hq)))
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
            assert all(torch.equal(a, b) for a, b in zip(run(), want))
