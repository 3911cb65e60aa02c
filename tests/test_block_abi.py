"""Host-side tests of include/gdr_block.h (no GPU): exports, size queries, and that bad arguments are
refused with a status before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr
from chunked_gated_delta_04_gb300 import build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced
R = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdr.load()


def test_exports_every_declared_function(lib):
    hdr = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gdr_block.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(gdr_[a-z0-9_]+)\s*\(", hdr))
    assert names == set(gdr.BLOCK_EXPORTS) and names <= set(gdr.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def conv(**kw):
    a = dict(B=2, T=8, C=16, W=4, num_seqs=2, cu_seqlens=None, dtype=1, silu=1, ld_x=0, ld_dy=0, num_slots=4)
    a.update(kw)
    return gdr.gdr_conv_problem(*a.values())


def ssm(**kw):
    a = dict(B=2, T=40, D=16, N=16, G=1, num_seqs=2, cu_seqlens=None, dtype=1, dt_softplus=1, ld_x=0, ld_dt=0, ld_b=0, ld_c=0,
             ld_dy=0, num_slots=4)
    a.update(kw)
    return gdr.gdr_ssm_problem(*a.values())


def norm(**kw):
    a = dict(tokens=4, heads=2, D=64, dtype=1, res_dtype=1, eps=1e-6, ld_x=0, ld_gate=0)
    a.update(kw)
    return gdr.gdr_norm_problem(*a.values())


def conv_fwd(lib, p, **kw):
    a = dict(x=FAKE, w=FAKE, b=None, state=None, y=FAKE, last=None, ws=FAKE, n=1 << 30, s=0)
    a.update(kw)
    return lib.gdr_conv_fwd(R(p), *a.values())


def ssm_fwd(lib, p, **kw):
    a = dict(x=FAKE, dt=FAKE, A=FAKE, Bm=FAKE, Cm=FAKE, D=None, bias=None, S0=None, y=FAKE, S_T=None, saved=None, ws=FAKE,
             n=1 << 40, s=0)
    a.update(kw)
    return lib.gdr_ssm_fwd(R(p), *a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(C=0), gdr.GDR_ERR_INVALID_ARG), (dict(W=5), gdr.GDR_ERR_UNSUPPORTED), (dict(W=1), gdr.GDR_ERR_UNSUPPORTED),
    (dict(dtype=2), gdr.GDR_ERR_INVALID_ARG), (dict(silu=2), gdr.GDR_ERR_INVALID_ARG),
    (dict(ld_x=15), gdr.GDR_ERR_INVALID_ARG), (dict(num_seqs=3), gdr.GDR_ERR_INVALID_ARG),
    (dict(cu_seqlens=FAKE), gdr.GDR_ERR_INVALID_ARG),  # packed tokens need B = 1
    (dict(T=-1), gdr.GDR_ERR_INVALID_ARG), (dict(B=1 << 16, T=1 << 16, num_seqs=1 << 16), gdr.GDR_ERR_UNSUPPORTED)])
def test_conv_refusals(lib, kw, code):
    p = conv(**kw)
    assert conv_fwd(lib, p) == code
    assert lib.gdr_conv_bwd(R(p), *[FAKE] * 11, 1 << 40, 0) == code
    assert lib.gdr_conv_bwd_workspace_bytes(R(p)) == 0


def test_conv_argument_refusals(lib):
    p = conv()
    assert conv_fwd(lib, p, x=None) == gdr.GDR_ERR_INVALID_ARG
    assert conv_fwd(lib, p, w=None) == gdr.GDR_ERR_INVALID_ARG
    assert conv_fwd(lib, p, x=FAKE + 1) == gdr.GDR_ERR_ALIGNMENT
    assert conv_fwd(lib, conv(dtype=0), x=FAKE + 2) == gdr.GDR_ERR_ALIGNMENT
    packed = conv(B=1, num_seqs=3, cu_seqlens=FAKE)
    assert lib.gdr_conv_fwd_workspace_bytes(R(packed)) == 256 and lib.gdr_conv_fwd_workspace_bytes(R(p)) == 0
    assert conv_fwd(lib, packed, ws=None) == gdr.GDR_ERR_WORKSPACE
    assert conv_fwd(lib, packed, ws=FAKE + 16) == gdr.GDR_ERR_ALIGNMENT
    need = lib.gdr_conv_bwd_workspace_bytes(R(p))
    assert lib.gdr_conv_bwd(R(p), *[FAKE] * 11, need - 1, 0) == gdr.GDR_ERR_WORKSPACE
    assert lib.gdr_conv_bwd(None, *[FAKE] * 11, 1 << 40, 0) == gdr.GDR_ERR_INVALID_ARG
    # a step is one token, without cu_seqlens, from a pool
    assert lib.gdr_conv_step(R(conv()), *[FAKE] * 6, 0) == gdr.GDR_ERR_INVALID_ARG
    assert lib.gdr_conv_step(R(conv(T=1, num_slots=-1)), *[FAKE] * 6, 0) == gdr.GDR_ERR_INVALID_ARG
    assert lib.gdr_conv_step(R(conv(T=1)), FAKE, FAKE, None, None, None, FAKE, 0) == gdr.GDR_ERR_INVALID_ARG
    assert lib.gdr_conv_step(R(conv(T=1, B=0)), *[None] * 6, 0) == gdr.GDR_OK


@pytest.mark.parametrize("kw,code", [
    (dict(N=12), gdr.GDR_ERR_UNSUPPORTED), (dict(N=128), gdr.GDR_ERR_UNSUPPORTED), (dict(G=3), gdr.GDR_ERR_INVALID_ARG),
    (dict(D=0), gdr.GDR_ERR_INVALID_ARG), (dict(dtype=5), gdr.GDR_ERR_INVALID_ARG),
    (dict(dt_softplus=3), gdr.GDR_ERR_INVALID_ARG), (dict(ld_b=15), gdr.GDR_ERR_INVALID_ARG),
    (dict(ld_dt=8), gdr.GDR_ERR_INVALID_ARG), (dict(num_seqs=1), gdr.GDR_ERR_INVALID_ARG),
    (dict(B=1 << 15, T=1 << 16, num_seqs=1 << 15), gdr.GDR_ERR_UNSUPPORTED)])
def test_ssm_refusals(lib, kw, code):
    p = ssm(**kw)
    assert ssm_fwd(lib, p) == code
    assert lib.gdr_ssm_bwd(R(p), *[FAKE] * 19, 1 << 40, 0) == code
    assert lib.gdr_ssm_saved_bytes(R(p)) == 0 and lib.gdr_ssm_fwd_workspace_bytes(R(p)) == 0


def test_ssm_sizes_and_argument_refusals(lib):
    p = ssm()
    assert lib.gdr_ssm_saved_bytes(R(p)) == 2 * 3 * 16 * 16 * 4  # ceil(40 / 16) states for each of two sequences
    packed = ssm(B=1, T=100, num_seqs=7, cu_seqlens=FAKE)
    assert lib.gdr_ssm_saved_bytes(R(packed)) == (100 // 16 + 7) * 16 * 16 * 4
    assert ssm_fwd(lib, p, A=None) == gdr.GDR_ERR_INVALID_ARG
    assert ssm_fwd(lib, p, A=FAKE + 4) == gdr.GDR_ERR_ALIGNMENT
    assert ssm_fwd(lib, p, S0=FAKE + 8) == gdr.GDR_ERR_ALIGNMENT
    assert ssm_fwd(lib, p, ws=None) == gdr.GDR_ERR_WORKSPACE
    assert ssm_fwd(lib, p, n=lib.gdr_ssm_fwd_workspace_bytes(R(p)) - 1) == gdr.GDR_ERR_WORKSPACE
    need = lib.gdr_ssm_bwd_workspace_bytes(R(p))
    assert lib.gdr_ssm_bwd(R(p), *[FAKE] * 19, need - 1, 0) == gdr.GDR_ERR_WORKSPACE
    args = [FAKE] * 19
    args[7] = None  # h_saved
    assert lib.gdr_ssm_bwd(R(p), *args, need, 0) == gdr.GDR_ERR_INVALID_ARG
    assert lib.gdr_ssm_step(R(p), *[FAKE] * 10, 0) == gdr.GDR_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(D=0), gdr.GDR_ERR_INVALID_ARG), (dict(D=16385), gdr.GDR_ERR_UNSUPPORTED), (dict(eps=0.0), gdr.GDR_ERR_INVALID_ARG),
    (dict(eps=float("nan")), gdr.GDR_ERR_INVALID_ARG), (dict(dtype=0, res_dtype=1), gdr.GDR_ERR_INVALID_ARG),
    (dict(ld_x=127), gdr.GDR_ERR_INVALID_ARG), (dict(heads=0), gdr.GDR_ERR_INVALID_ARG),
    (dict(tokens=-1), gdr.GDR_ERR_INVALID_ARG)])
def test_norm_refusals(lib, kw, code):
    p = norm(**kw)
    assert lib.gdr_norm_fwd(R(p), *[FAKE] * 8, 0) == code
    assert lib.gdr_norm_bwd(R(p), *[FAKE] * 6, 1, *[FAKE] * 9, 1 << 40, 0) == code
    assert lib.gdr_norm_bwd_workspace_bytes(R(p)) == 0


def test_norm_argument_refusals(lib):
    p = norm()
    inv = gdr.GDR_ERR_INVALID_ARG
    # x alone; a norm in front of a block without a residual but with a gate; a residual without r
    assert lib.gdr_norm_fwd(R(p), FAKE, None, None, None, None, None, FAKE, None, 0) == inv
    assert lib.gdr_norm_fwd(R(p), FAKE, None, FAKE, None, None, FAKE, FAKE, FAKE, 0) == inv
    assert lib.gdr_norm_fwd(R(p), FAKE, None, None, None, FAKE, FAKE, None, FAKE, 0) == inv
    assert lib.gdr_norm_fwd(R(p), FAKE + 1, FAKE, None, None, None, None, FAKE, None, 0) == gdr.GDR_ERR_ALIGNMENT
    need = lib.gdr_norm_bwd_workspace_bytes(R(p))

    def bwd(**kw):
        a = dict(x=FAKE, w_post=FAKE, gate=FAKE, scale=None, r=FAKE, w_pre=FAKE, has=1, dr=FAKE, dy=FAKE, dx=FAKE, dgate=FAKE,
                 dres=FAKE, dpost=FAKE, dscale=None, dpre=FAKE, ws=FAKE, n=need, s=0)
        a.update(kw)
        return lib.gdr_norm_bwd(R(p), *a.values())

    assert bwd(dy=None) == inv and bwd(dr=None, dy=None) == inv and bwd(dgate=None) == inv and bwd(dpost=None) == inv
    assert bwd(dpre=None) == inv and bwd(r=None) == inv and bwd(has=0) == inv
    assert bwd(n=need - 1) == gdr.GDR_ERR_WORKSPACE and bwd(ws=None) == gdr.GDR_ERR_WORKSPACE


def test_step_refusals(lib):
    def call(slots=4, pool=FAKE, q=FAKE, **kw):
        a = dict(B=2, T=1, Hk=2, Hv=4, DK=128, DV=128, dtype=torch.bfloat16, layout="KV")
        a.update(kw)
        return lib.gdr_step(R(gdr.make_problem(**a)), q, FAKE, FAKE, FAKE, FAKE, pool, slots, None, FAKE, 0)

    assert call(T=2) == gdr.GDR_ERR_INVALID_ARG and call(Hv=3) == gdr.GDR_ERR_INVALID_ARG
    assert call(DK=136) == gdr.GDR_ERR_UNSUPPORTED and call(DV=8) == gdr.GDR_ERR_UNSUPPORTED
    assert call(dtype=torch.float16) == gdr.GDR_ERR_INVALID_ARG and call(prologue=8) == gdr.GDR_ERR_INVALID_ARG
    assert call(layout=5) == gdr.GDR_ERR_INVALID_ARG and call(slots=-1) == gdr.GDR_ERR_INVALID_ARG
    assert call(q=None) == gdr.GDR_ERR_INVALID_ARG and call(pool=FAKE + 8) == gdr.GDR_ERR_ALIGNMENT
    assert call(B=70000) == gdr.GDR_ERR_UNSUPPORTED and call(B=0, q=None, pool=None) == gdr.GDR_OK


def test_python_refusals():
    """The helpers name what is wrong before they reach the library."""
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="x: expected a CUDA"):
        gdr.conv_forward(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="x: expected a CUDA"):
        gdr.ssm_forward(x, x, torch.zeros(8, 4), torch.zeros(2, 4, 1, 4), torch.zeros(2, 4, 1, 4))
    with pytest.raises(ValueError, match="x: expected a CUDA"):
        gdr.norm_forward(x, torch.zeros(8))
    with pytest.raises(ValueError, match="q: expected a contiguous CUDA"):
        gdr.step(torch.zeros(1, 1, 16), torch.zeros(1, 1, 16), torch.zeros(1, 1, 16), torch.zeros(1, 1), torch.zeros(1, 1),
                 torch.zeros(1, 1, 16, 16))


def test_token_strides():
    from chunked_gated_delta_04_gb300.block import _ld

    base = torch.zeros(2, 5, 48)
    assert _ld("x", base, 1) == 0 and _ld("x", base[:, :, 8:24], 1) == 48
    assert _ld("x", base.view(2, 5, 4, 12)[:, :, 1:3], 2) == 48
    assert _ld("x", base[:, 3], 1) == 240 and _ld("x", base[:1, ::2], 1) == 96
    for bad in (base.transpose(0, 1), base[:, :4, 8:24], base[:, :, ::2]):
        with pytest.raises(ValueError):
            _ld("x", bad, 1)


def test_token_strides_of_broadcast_rows():
    """A row repeated over tokens or over the batch (stride 0) is no evenly spaced batch of rows."""
    from chunked_gated_delta_04_gb300.block import _ld, _rows_ok

    for t, inner in ((torch.zeros(1, 1, 16).expand(1, 5, 16), 1), (torch.zeros(2, 1, 16).expand(2, 5, 16), 1),
                     (torch.zeros(1, 5, 16).expand(2, 5, 16), 1), (torch.zeros(1, 1, 1).expand(2, 5, 16), 1),
                     (torch.zeros(2, 1, 2, 8).expand(2, 5, 2, 8), 2), (torch.zeros(1, 3, 16).expand(1, 3, 16)[:, :, :8], 1)):
        if 0 in t.stride():
            with pytest.raises(ValueError):
                _ld("x", t, inner)
            assert _rows_ok(t, inner).is_contiguous()
        else:
            assert _ld("x", t, inner) == 16


def test_sizes_beyond_32_bits():
    """A size that an int does not hold is refused, not cut to its low bits (the tensors here are one element)."""
    def big(*shape, dtype=torch.float32):
        return torch.zeros((1,) * len(shape), dtype=dtype).expand(shape)

    n = (1 << 32) + 5
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        gdr.conv_forward(big(1, n, 8), torch.zeros(8, 4))
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        gdr.conv_step(big(2, 8), big(n, 3, 8), torch.zeros(8, 4))
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        gdr.ssm_forward(big(1, n, 8), big(1, n, 8), torch.zeros(8, 4), big(1, n, 1, 4), big(1, n, 1, 4))
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        gdr.norm_forward(big(2, n), big(n))
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        gdr.step(big(1, 1, 16), big(1, 1, 16), big(1, 1, 16), big(1, 1), big(1, 1), big(n, 1, 16, 16))
