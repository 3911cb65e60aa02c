"""Which tensors have to be aligned to 16 bytes: the header says so, the library refuses them otherwise, and the Python
calls copy the ones that they only read."""
import ctypes
import os
import re

import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: every call here is refused
FWD = ["x", "dt", "A", "Bm", "Cm", "Dskip", "dt_bias", "S0", "y", "S_T", "h_saved"]
BWD = ["x", "dt", "A", "Bm", "Cm", "Dskip", "dt_bias", "h_saved", "dy", "dS_T", "dx", "ddt", "dA", "dBm", "dCm", "dDskip", "ddt_bias",
       "dS0"]
STEP = ["x", "dt", "A", "Bm", "Cm", "Dskip", "dt_bias", "pool", "slots", "y"]
DELTA = ["q", "k", "v", "g", "beta", "pool"]


def test_the_header_names_what_is_refused():
    text = " ".join(re.sub(r"\n \*", " ", open(os.path.join(ROOT, "include", "gdr_block.h")).read()).split())
    named = re.search(r"unless they are aligned to 16: ([\w, ]+) and the pools of gdr_ssm_step and gdr_step\.", text)
    assert named is not None
    named = named.group(1).split(", ")
    lib, R = gdr.load(), ctypes.byref
    p = gdr.gdr_ssm_problem(2, 40, 16, 16, 1, 2, None, 0, 1)
    one = gdr.gdr_ssm_problem(2, 1, 16, 16, 1, 2, None, 0, 1, num_slots=4)
    d = gdr.make_problem(2, 1, 2, 4, 128, 128, torch.float32)
    for name in named:
        assert name in FWD + BWD
        off = {n: FAKE + 4 * (n == name) for n in FWD + BWD}
        if name in FWD:
            assert lib.gdr_ssm_fwd(R(p), *[off[n] for n in FWD], FAKE, 1 << 40, 0) == gdr.GDR_ERR_ALIGNMENT, name
        if name in BWD:
            assert lib.gdr_ssm_bwd(R(p), *[off[n] for n in BWD], FAKE, 1 << 40, 0) == gdr.GDR_ERR_ALIGNMENT, name
    assert lib.gdr_ssm_step(R(one), *[FAKE + 4 * (n == "pool") for n in STEP], 0) == gdr.GDR_ERR_ALIGNMENT
    assert lib.gdr_step(R(d), *[FAKE + 4 * (n == "pool") for n in DELTA], 4, FAKE, FAKE, 0) == gdr.GDR_ERR_ALIGNMENT
    assert set(named) == {"A", "S0", "S_T", "h_saved", "dS_T", "dS0"}


def between(t):
    """The same values as a view of a flat buffer that begins 4 bytes past a 16-byte boundary."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:] = t.flatten()
    return buf[1:].view(t.shape)


@pytest.mark.gpu
def test_views_of_a_flat_buffer():
    gen = torch.Generator().manual_seed(2)

    def rand(*shape):
        return torch.randn(*shape, generator=gen).cuda()

    B, T, D, N = 2, 37, 24, 8
    x, dt, Bm, Cm, dy = rand(B, T, D), rand(B, T, D) * 0.3, rand(B, T, 1, N), rand(B, T, 1, N), rand(B, T, D)
    A, S0, dS, skip = -torch.exp(rand(D, N)), rand(B, D, N), rand(B, D, N), rand(D)

    def run(f):
        y, S, saved = gdr.ssm_forward(x, dt, f(A), Bm, Cm, f(skip), None, f(S0))
        grads = gdr.ssm_backward(x, dt, f(A), Bm, Cm, f(saved), dy, f(skip), None, f(dS))
        pool = S0.clone()
        return y, S, *grads, gdr.ssm_step(x[:, 0], dt[:, 0], f(A), Bm[:, 0], Cm[:, 0], pool, f(skip)), pool

    for a, b in zip(run(lambda t: t), run(between)):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    leaf = between(A).requires_grad_()
    gdr.selective_scan(x, dt, leaf, Bm, Cm)[0].sum().backward()
    assert torch.isfinite(leaf.grad).all()
    with pytest.raises(gdr.GDRError) as e:  # a pool is changed in place: a copy would lose that
        gdr.ssm_step(x[:, 0], dt[:, 0], A, Bm[:, 0], Cm[:, 0], between(S0))
    assert e.value.status == gdr.GDR_ERR_ALIGNMENT
