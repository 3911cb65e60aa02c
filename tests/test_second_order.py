"""Second derivatives of the autograd entry points are refused: the gradients are computed outside autograd, and
a second derivative without the terms through them would be wrong.  On the CPU the calls that the Functions make are
replaced by cubes, whose gradients are known."""
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr
from chunked_gated_delta_04_gb300 import block

F64 = torch.float64


def cube(x, *rest):
    return x ** 3


@pytest.fixture
def cubes(monkeypatch):
    """conv, scan and norm of cubes: y = x^3 (the scan's final state: S0^3)."""
    monkeypatch.setattr(block, "_rows_ok", lambda t, inner: t)
    monkeypatch.setattr(block, "conv_forward", lambda x, w, b, st, *a, **k: (x ** 3, x[:, -3:].clone()))
    monkeypatch.setattr(block, "conv_backward",
                        lambda x, w, b, dy, st, *a: (3 * dy * x ** 2, torch.zeros_like(w), None, None if st is None else torch.zeros_like(st)))
    monkeypatch.setattr(block, "ssm_forward", lambda x, dt, A, B, C, D, bias, S0, *a, **k: (x ** 3, S0 + 1 if S0 is not None else A + 1, x ** 2))
    monkeypatch.setattr(block, "ssm_backward", lambda x, dt, A, B, C, saved, dy, D, bias, dS, *a, want_dS0:
                        (3 * dy * saved, *[torch.zeros_like(t) for t in (dt, A, B, C)], None, None, torch.zeros_like(dS) if want_dS0 else None))
    monkeypatch.setattr(block, "norm_forward", lambda x, post, gate, scale, res, pre, eps: (x ** 3 + (0 if res is None else res), None))
    monkeypatch.setattr(block, "norm_backward", lambda x, post, gate, scale, r, pre, dr, dy, eps:
                        (3 * dr * x ** 2, None, None if r is None else dr, None, None, None))


def entries(x):
    one = torch.ones(x.shape[-1], 4, dtype=x.dtype, device=x.device)
    bc = torch.ones(*x.shape[:2], 1, 4, dtype=x.dtype, device=x.device)
    return {"causal_conv": lambda x: gdr.causal_conv(x, one)[0],
            "selective_scan": lambda x: gdr.selective_scan(x, x.detach(), -one, bc, bc)[0],
            "block_norm": lambda x: gdr.block_norm(x, one[:, 0].contiguous())[0]}


def losses(f, x):
    """The gradient that comes in depends on x, and does not."""
    return {"product": lambda: (x * f(x)).sum(), "sum": lambda: (x ** 2).sum() + f(x).sum()}


@pytest.mark.parametrize("name", ["causal_conv", "selective_scan", "block_norm"])
@pytest.mark.parametrize("loss", ["product", "sum"])
def test_second_derivatives_are_refused(cubes, monkeypatch, name, loss):
    monkeypatch.setattr(torch.Tensor, "float", lambda t: t)  # the weights stay in 64 bits
    x = torch.randn(2, 5, 3, dtype=F64, generator=torch.Generator().manual_seed(1)).requires_grad_()
    f = entries(x)[name]
    run, plain = losses(f, x)[loss], losses(cube, x)[loss]
    g, = torch.autograd.grad(run(), x, create_graph=True)
    assert torch.equal(g, torch.autograd.grad(plain(), x)[0]) or torch.allclose(g, torch.autograd.grad(plain(), x)[0], rtol=1e-14)
    with pytest.raises(RuntimeError, match=f"{name} has no second derivative"):
        torch.autograd.grad(g.sum(), x)
    with pytest.raises(RuntimeError, match=f"{name} has no second derivative"):
        torch.autograd.grad(run(), x, create_graph=True)[0].sum().backward()


def test_an_initial_state_counts_too(cubes, monkeypatch):
    """A scan's gradients depend on its initial state, although it is not kept: it may be changed in place."""
    monkeypatch.setattr(torch.Tensor, "float", lambda t: t)
    x, S = torch.randn(2, 5, 3, dtype=F64).requires_grad_(), torch.randn(2, 3, 4, dtype=F64).requires_grad_()
    one, bc = torch.ones(3, 4, dtype=F64), torch.ones(2, 5, 1, 4, dtype=F64)

    def run(state):
        y, last = gdr.selective_scan(x, x.detach(), -one, bc, bc, initial_state=state)
        return y.sum() + last.sum()

    g, = torch.autograd.grad(run(S), x, create_graph=True)
    with pytest.raises(RuntimeError, match="selective_scan has no second derivative"):
        torch.autograd.grad(g.sum(), S)
    state = S * 1  # not a leaf
    loss = run(state)
    state.zero_()
    loss.backward()
    assert torch.allclose(x.grad, 3 * x.detach() ** 2, rtol=1e-14)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["causal_conv", "selective_scan", "block_norm"])
@pytest.mark.parametrize("loss", ["product", "sum"])
def test_second_derivatives_are_refused_on_the_gpu(name, loss):
    x = torch.randn(2, 5, 8, device="cuda").requires_grad_()
    run = losses(entries(x)[name], x)[loss]
    first, = torch.autograd.grad(run(), x)
    g, = torch.autograd.grad(run(), x, create_graph=True)
    assert torch.equal(g, first)
    with pytest.raises(RuntimeError, match=f"{name} has no second derivative"):
        torch.autograd.grad(g.sum(), x)


def delta_inputs(B, T, H, D, **kw):
    gen = torch.Generator().manual_seed(3)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, dtype=kw["dtype"]).to(kw["device"])

    q, k, v = rand(B, T, H, D), torch.nn.functional.normalize(rand(B, T, H, D), dim=-1), rand(B, T, H, D)
    return q, k, v, -rand(B, T, H).abs(), torch.sigmoid(rand(B, T, H)), rand(B, H, D, D)


@pytest.mark.parametrize("loss", ["product", "sum"])
def test_second_derivatives_of_the_delta_rule_are_refused(monkeypatch, loss):
    q, k, v, g, beta, S0 = delta_inputs(2, 5, 1, 3, dtype=F64, device="cpu")
    monkeypatch.setattr(gdr, "forward", lambda q, k, v, g, beta, S0, *a, **kw: (v ** 3, S0 + 1, v ** 2))
    monkeypatch.setattr(gdr, "backward", lambda q, k, v, g, beta, saved, do, dS, *a, **kw:
                        (*[torch.zeros_like(t) for t in (q, k)], 3 * do * saved, torch.zeros_like(g), torch.zeros_like(beta), dS))
    x, S0 = v.requires_grad_(), S0.requires_grad_()
    run = losses(lambda x: gdr.chunk_gated_delta_rule(q, k, x, g, beta, S0)[0], x)[loss]
    grad, = torch.autograd.grad(run(), x, create_graph=True)
    assert torch.allclose(grad, torch.autograd.grad(losses(cube, x)[loss](), x)[0], rtol=1e-14)
    for of in (x, S0):  # the state counts too
        with pytest.raises(RuntimeError, match="chunk_gated_delta_rule has no second derivative"):
            torch.autograd.grad(grad.sum(), of, retain_graph=True)
    state = S0 * 1
    total = gdr.chunk_gated_delta_rule(q, k, x, g, beta, state)[0].sum()
    state.zero_()  # its owner may change it: it is not kept
    assert torch.allclose(torch.autograd.grad(total, x)[0], 3 * x.detach() ** 2, rtol=1e-14)


@pytest.mark.gpu
@pytest.mark.parametrize("loss", ["product", "sum"])
def test_second_derivatives_of_the_delta_rule_are_refused_on_the_gpu(loss):
    q, k, v, g, beta, S0 = delta_inputs(1, 20, 2, 16, dtype=torch.float32, device="cuda")
    x, S0 = v.requires_grad_(), S0.requires_grad_()
    run = losses(lambda x: gdr.chunk_gated_delta_rule(q, k, x, g, beta, S0)[0], x)[loss]
    first, = torch.autograd.grad(run(), x)
    grad, = torch.autograd.grad(run(), x, create_graph=True)
    assert torch.equal(grad, first)
    for of in (x, S0):
        with pytest.raises(RuntimeError, match="chunk_gated_delta_rule has no second derivative"):
            torch.autograd.grad(grad.sum(), of, retain_graph=True)
