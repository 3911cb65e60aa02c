"""Host-side tests of include/gdr_attn.h (no GPU): exports, size queries, and that bad arguments are refused before anything
is launched; what the Python helpers refuse, second derivatives among it."""
import ctypes
import os
import re

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import chunked_gated_delta_04_gb300 as gdr
from chunked_gated_delta_04_gb300 import attn, build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced
R = ctypes.byref
F32, F64, BF, I32 = torch.float32, torch.float64, torch.bfloat16, torch.int32
INV, UNS, ALI, WS = gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED, gdr.GDR_ERR_ALIGNMENT, gdr.GDR_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdr.load()


def test_exports_every_declared_function(lib):
    hdr = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gdr_attn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(gdr_[a-z0-9_]+)\s*\(", hdr))
    assert names == set(gdr.ATTN_EXPORTS) and names <= set(gdr.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def rope(**kw):
    a = dict(B=2, T=8, Hq=4, Hk=2, D=64, R=32, num_seqs=2, cu=None, dtype=1, interleaved=0, inverse=0, scale=1.0, ld_q=0, ld_k=0)
    a.update(kw)
    return gdr.gdr_rope_problem(*a.values())


def att(**kw):
    a = dict(B=2, Tq=8, Tk=16, Hq=4, Hk=2, D=64, num_seqs=2, cu_q=None, cu_k=None, dtype=1, causal=1, window=0, scale=0.0, ld_q=0, ld_k=0,
             ld_v=0, ld_do=0)
    a.update(kw)
    return gdr.gdr_attn_problem(*a.values())


def cache(**kw):
    a = dict(B=2, T=1, Hq=4, Hk=2, D=64, num_pages=8, page_size=16, max_pages=3, cu=None, dtype=1, window=0, scale=0.0, ld_q=0, ld_k=0, ld_v=0)
    a.update(kw)
    return gdr.gdr_cache_problem(*a.values())


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(Hq=0), INV), (dict(Hk=-1), INV), (dict(R=0), INV), (dict(R=3), INV), (dict(R=66), INV), (dict(dtype=2), INV),
    (dict(interleaved=2), INV), (dict(inverse=-1), INV), (dict(scale=NAN), INV), (dict(ld_q=255), INV), (dict(ld_k=-8), INV),
    (dict(num_seqs=3), INV), (dict(cu=FAKE), INV), (dict(cu=FAKE, B=1, num_seqs=0), INV), (dict(D=1040), UNS),
    (dict(B=1 << 16, T=1 << 16, num_seqs=1 << 16), UNS), (dict(Hq=70000), UNS)])
def test_rope_refusals(lib, kw, code):
    assert lib.gdr_rope(R(rope(**kw)), *[FAKE] * 7, 1 << 20, 0) == code
    assert lib.gdr_rope_workspace_bytes(R(rope(**kw))) == 0


def test_rope_argument_refusals(lib):
    def call(p, q=FAKE, k=FAKE, freqs=FAKE, pos=None, qo=FAKE, ko=FAKE, ws=FAKE, n=256):
        return lib.gdr_rope(R(p), q, k, freqs, pos, qo, ko, ws, n, 0)

    assert call(rope(), q=None) == INV and call(rope(), k=None) == INV and call(rope(), freqs=None) == INV and call(rope(), ko=None) == INV
    assert call(rope(), q=FAKE + 1) == ALI and call(rope(), freqs=FAKE + 4) == ALI and call(rope(), pos=FAKE + 2) == ALI
    packed = rope(B=1, cu=FAKE, num_seqs=3)
    assert lib.gdr_rope_workspace_bytes(R(packed)) == 256 and lib.gdr_rope_workspace_bytes(R(rope())) == 0
    assert call(packed, ws=None) == WS and call(packed, n=255) == WS and call(packed, ws=FAKE + 8) == ALI
    assert call(rope(T=0), q=None, k=None, qo=None, ko=None) == gdr.GDR_OK and lib.gdr_rope(None, *[FAKE] * 7, 256, 0) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1, num_seqs=-1), INV), (dict(Tq=-1), INV), (dict(Hq=3), INV), (dict(Hk=0), INV), (dict(D=0), INV), (dict(dtype=3), INV),
    (dict(causal=2), INV), (dict(window=-1), INV), (dict(scale=NAN), INV), (dict(scale=INF), INV), (dict(cu_q=FAKE), INV),
    (dict(B=1, num_seqs=2, cu_q=FAKE), INV), (dict(cu_q=FAKE, cu_k=FAKE), INV), (dict(num_seqs=1), INV), (dict(ld_q=255), INV),
    (dict(ld_v=127), INV), (dict(ld_do=-1), INV), (dict(D=72), UNS), (dict(D=256), UNS), (dict(B=1 << 16, Tq=1 << 15, num_seqs=1 << 16), UNS)])
def test_attn_refusals(lib, kw, code):
    p = att(**kw)
    assert lib.gdr_attn_fwd(R(p), *[FAKE] * 6, 1 << 40, 0) == code
    assert lib.gdr_attn_bwd(R(p), *[FAKE] * 10, 1 << 40, 0) == code
    assert lib.gdr_attn_fwd_workspace_bytes(R(p)) == 0 and lib.gdr_attn_bwd_workspace_bytes(R(p)) == 0


def test_attn_argument_refusals(lib):
    p = att()
    fwd, bwd = lib.gdr_attn_fwd_workspace_bytes(R(p)), lib.gdr_attn_bwd_workspace_bytes(R(p))
    assert fwd >= 256 and bwd >= 256 + 4 * 2 * 8 * 4
    packed = att(B=1, num_seqs=3, cu_q=FAKE, cu_k=FAKE)
    assert lib.gdr_attn_fwd_workspace_bytes(R(packed)) > fwd

    def f(p=p, n=fwd, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, ws=FAKE)
        a.update(kw)
        return lib.gdr_attn_fwd(R(p), *a.values(), n, 0)

    def b(p=p, n=bwd, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE)
        a.update(kw)
        return lib.gdr_attn_bwd(R(p), *a.values(), n, 0)

    for name in ("q", "k", "v", "o", "lse"):
        assert f(**{name: None}) == INV and f(**{name: FAKE + 1}) == ALI, name
    for name in ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv"):
        assert b(**{name: None}) == INV and b(**{name: FAKE + 1}) == ALI, name
    assert f(n=fwd - 1) == WS and f(ws=None) == WS and f(ws=FAKE + 16) == ALI
    assert b(n=bwd - 1) == WS and b(ws=None) == WS and b(ws=FAKE + 16) == ALI
    assert f(att(B=0, num_seqs=0), q=None, k=None, v=None, o=None, lse=None) == gdr.GDR_OK
    assert lib.gdr_attn_fwd(None, *[FAKE] * 6, 1 << 40, 0) == INV and lib.gdr_attn_bwd(None, *[FAKE] * 10, 1 << 40, 0) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(T=2), INV), (dict(cu=FAKE), INV), (dict(Hq=3), INV), (dict(Hk=0), INV), (dict(D=0), INV), (dict(dtype=4), INV),
    (dict(num_pages=-1), INV), (dict(page_size=0), INV), (dict(max_pages=-1), INV), (dict(window=-1), INV), (dict(scale=INF), INV),
    (dict(ld_q=255), INV), (dict(ld_k=100), INV), (dict(D=40), UNS), (dict(D=144), UNS), (dict(max_pages=1 << 20, page_size=1 << 12), UNS),
    (dict(B=1 << 29, Hq=8, Hk=8), UNS)])
def test_step_refusals(lib, kw, code):
    p = cache(**kw)
    assert lib.gdr_attn_step(R(p), *[FAKE] * 9, 1 << 40, 0) == code and lib.gdr_attn_step_workspace_bytes(R(p)) == 0


def test_step_and_write_argument_refusals(lib):
    p = cache()
    need = lib.gdr_attn_step_workspace_bytes(R(p))

    def step(p=p, n=need, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lengths=FAKE, o=FAKE, ws=FAKE)
        a.update(kw)
        return lib.gdr_attn_step(R(p), *a.values(), n, 0)

    for name in ("q", "k", "v", "kc", "vc", "table", "lengths", "o"):
        assert step(**{name: None}) == INV, name
    assert step(q=FAKE + 1) == ALI and step(kc=FAKE + 8) == ALI and step(table=FAKE + 2) == ALI and step(ws=FAKE + 8) == ALI
    assert step(n=need - 1) == WS and step(ws=None) == WS and step(cache(B=0), q=None) == gdr.GDR_OK

    def write(p, ws=None, n=0, **kw):
        a = dict(k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, table=FAKE, starts=None)
        a.update(kw)
        return lib.gdr_cache_write(R(p), *a.values(), ws, n, 0)

    p = cache(T=5, Hq=0)
    for name in ("k", "v", "kc", "vc", "table"):
        assert write(p, **{name: None}) == INV, name
    assert write(p, k=FAKE + 1) == ALI and write(p, vc=FAKE + 4) == ALI and write(p, starts=FAKE + 1) == ALI
    assert write(cache(T=-1)) == INV and write(cache(T=5, D=24)) == UNS and write(cache(T=1 << 16, B=1 << 16)) == UNS
    packed = cache(T=5, cu=FAKE)
    assert lib.gdr_cache_write_workspace_bytes(R(packed)) == 256 and lib.gdr_cache_write_workspace_bytes(R(p)) == 0
    assert write(packed) == WS and write(packed, ws=FAKE + 8, n=256) == ALI and write(cache(B=0, T=5, cu=FAKE), ws=FAKE, n=256) == INV
    assert write(cache(T=0), k=None, v=None) == gdr.GDR_OK


# name: (shape, dtype) of the calls' tensors, the first being the one that the others have to join
ATTN = dict(q=((1, 6, 4, 16), BF), k=((1, 9, 2, 16), BF), v=((1, 9, 2, 16), BF))
CACHE = dict(k_cache=((4, 8, 2, 16), BF), v_cache=((4, 8, 2, 16), BF), block_table=((2, 3), I32))
CALLS = {
    "rope_forward": dict(q=((1, 6, 4, 16), BF), k=((1, 6, 2, 16), BF), freqs=((8,), F64), positions=((1, 6), I32), cu_seqlens=((3,), I32)),
    "rope_backward": dict(dq=((1, 6, 4, 16), BF), dk=((1, 6, 2, 16), BF), freqs=((8,), F64), positions=((1, 6), I32)),
    "attn_forward": dict(ATTN, cu_seqlens=((3,), I32), cu_seqlens_k=((3,), I32)),
    "attn_backward": dict(ATTN, o=((1, 6, 4, 16), BF), lse=((1, 4, 6), F32), do=((1, 6, 4, 16), BF), cu_seqlens=((3,), I32)),
    "attn_step": dict(q=((2, 4, 16), BF), k=((2, 2, 16), BF), v=((2, 2, 16), BF), **CACHE, lengths=((2,), I32)),
    "cache_write": dict(k=((1, 6, 2, 16), BF), v=((1, 6, 2, 16), BF), **CACHE, starts=((2,), I32), cu_seqlens=((3,), I32)),
}
INNER = {"dk": "k", "dq": "q"}  # what the library calls them


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake devices")
@pytest.mark.parametrize("call,name", [(c, n) for c, args in CALLS.items() for n in list(args)[1:]])
def test_a_tensor_on_another_device_is_refused(call, name):
    with FakeTensorMode():
        args = {n: torch.empty(shape, dtype=dtype, device="cuda:1" if n == name else "cuda:0") for n, (shape, dtype) in CALLS[call].items()}
        with pytest.raises(ValueError, match=f"^{INNER.get(name, name)}: on cuda:1, the call's first tensor on cuda:0"):
            getattr(gdr, call)(**args)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake devices")
@pytest.mark.parametrize("call", list(CALLS))
def test_shapes_and_types_are_checked(call):
    """Each tensor of a call with another type, and with one more row, is named."""
    for name, (shape, dtype) in CALLS[call].items():
        for wrong in (dict(dtype=torch.int64), dict(shape=(*shape[:-1], shape[-1] + 1))):
            if "shape" in wrong and name in (list(CALLS[call])[0], "k_cache", "block_table", "freqs", "cu_seqlens"):
                continue  # sizes that the others are measured by
            with FakeTensorMode():
                args = {n: torch.empty(s, dtype=d, device="cuda:0") for n, (s, d) in CALLS[call].items()}
                args[name] = torch.empty(wrong.get("shape", shape), dtype=wrong.get("dtype", dtype), device="cuda:0")
                with pytest.raises(ValueError):
                    getattr(gdr, call)(**args)


def test_python_refusals():
    x = torch.zeros(2, 4, 2, 16)
    with pytest.raises(ValueError, match="q: expected a CUDA"):
        gdr.attn_forward(x, x, x)
    with pytest.raises(ValueError, match="q: expected a CUDA"):
        gdr.rope_forward(x, None, torch.zeros(8, dtype=F64))
    with pytest.raises(ValueError, match="single tokens"):
        gdr.rope_forward(x[0], None, torch.zeros(8, dtype=F64))
    with pytest.raises(ValueError, match="scale 0"):
        gdr.attn_forward(x, x, x, scale=0)
    with pytest.raises(ValueError, match="scale nan"):
        gdr.attn_step(x[0], x[0], x[0], x, x, x, x, scale=NAN)
    with pytest.raises(TypeError, match="k: expected a tensor"):
        gdr.attn_forward(x, 3, x)
    with pytest.raises(ValueError, match="v: expected a tensor, got None"):
        gdr.attn_forward(x, x, None)
    with pytest.raises(ValueError, match="k: expected a CUDA"):
        gdr.cache_write(x, x, x, x, x)
    with FakeTensorMode():
        q, k = torch.empty(1, 6, 4, 16, dtype=BF, device="cuda"), torch.empty(1, 9, 2, 16, dtype=BF, device="cuda")
        cu = torch.empty(3, dtype=I32, device="cuda")
        with pytest.raises(ValueError, match="cu_seqlens_k needs cu_seqlens"):
            gdr.attn_forward(q, k, k, cu_seqlens_k=cu)
        with pytest.raises(ValueError, match="cu_seqlens_k: expected 3 entries"):
            gdr.attn_forward(q, k, k, cu_seqlens=cu, cu_seqlens_k=torch.empty(4, dtype=I32, device="cuda"))
        with pytest.raises(ValueError, match="window: -1"):
            gdr.attn_forward(q, k, k, window=-1)
        with pytest.raises(ValueError, match="evenly spaced"):
            gdr.attn_forward(q.expand(2, 6, 4, 16), k.expand(2, 9, 2, 16).contiguous(), k.expand(2, 9, 2, 16).contiguous())


@pytest.mark.parametrize("scale", [1e-50, 1e-40, -1.0, 1e39, INF])
def test_scales_beyond_32_bits(scale):
    """What rounds to 0 as a 32-bit number would otherwise be taken for the default."""
    x = torch.zeros(2, 4, 2, 16)
    with pytest.raises(ValueError, match="scale"):
        gdr.attn_forward(x, x, x, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        gdr.attn_step(x[0], x[0], x[0], x, x, x, x, scale=scale)


def test_token_counts_at_the_limit(lib):
    """The end of the last tile has to be a 32-bit number."""
    for name in ("Tq", "Tk"):
        assert lib.gdr_attn_fwd_workspace_bytes(R(att(B=1, num_seqs=1, **{name: (1 << 31) - 1000}))) == 0
        assert lib.gdr_attn_fwd_workspace_bytes(R(att(B=1, num_seqs=1, Hq=1, Hk=1, **{name: (1 << 31) - 1025}))) == 256


def test_sizes_beyond_32_bits():
    def big(*shape, dtype=F32):
        return torch.zeros((1,) * len(shape), dtype=dtype).expand(shape)

    n = (1 << 32) + 5
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        gdr.attn_forward(big(1, n, 2, 16), big(1, 4, 2, 16), big(1, 4, 2, 16))
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        gdr.rope_forward(big(1, n, 2, 16), None, big(8, dtype=F64))
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        gdr.attn_step(big(n, 2, 16), big(n, 2, 16), big(n, 2, 16), big(1, 16, 2, 16), big(1, 16, 2, 16), big(n, 1, dtype=I32), big(n, dtype=I32))


@pytest.mark.parametrize("kind", ["rope", "attention"])
def test_second_derivatives_are_refused(monkeypatch, kind):
    """The library's calls are replaced by cubes, whose gradients are known."""
    monkeypatch.setattr(attn, "_rows_ok", lambda t, inner: t)
    monkeypatch.setattr(attn, "rope_forward", lambda q, k, *a, **kw: (q * 3, None))
    monkeypatch.setattr(attn, "rope_backward", lambda dq, dk, *a, **kw: (dq * 3, None))
    monkeypatch.setattr(attn, "attn_forward", lambda q, k, v, *a, **kw: (q ** 3, q.sum()))
    monkeypatch.setattr(attn, "attn_backward", lambda q, k, v, o, lse, do, *a: (3 * do * q ** 2, torch.zeros_like(k), torch.zeros_like(v)))
    x = torch.randn(1, 5, 2, 4, dtype=F64, generator=torch.Generator().manual_seed(1)).requires_grad_()
    freqs = torch.ones(2, dtype=F64)

    def f(x):
        return gdr.rope(x, None, freqs)[0] if kind == "rope" else gdr.attention(x, x.detach(), x.detach())

    g, = torch.autograd.grad((x * f(x)).sum(), x, create_graph=True)
    want = 6 * x if kind == "rope" else 4 * x ** 3
    assert torch.allclose(g, want, rtol=1e-13)
    with pytest.raises(RuntimeError, match=f"{kind} has no second derivative"):
        torch.autograd.grad(g.sum(), x)


def test_workspace_sizes(lib):
    q, k = torch.zeros(1, 40, 4, 16, dtype=BF), torch.zeros(1, 50, 2, 16, dtype=BF)
    cu, cu_k = torch.tensor([0, 5, 40], dtype=I32), torch.tensor([0, 9, 50], dtype=I32)
    for backward in (False, True):
        ws = gdr.attn_workspace(q, k, cu, cu_k, backward=backward)
        p = att(B=1, Tq=40, Tk=50, D=16, num_seqs=2, cu_q=cu.data_ptr(), cu_k=cu_k.data_ptr())
        need = getattr(lib, f"gdr_attn_{'bwd' if backward else 'fwd'}_workspace_bytes")(R(p))
        assert ws.numel() == need > 256 and not ws[:256].any()
    assert gdr.rope_workspace(q, cu).numel() == 256 and gdr.cache_write_workspace(k, cu_k).numel() == 256
