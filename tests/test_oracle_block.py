"""Pins of the fp64 references of the operators around the gated delta rule (CPU): hand-worked
values, closed forms, and every gradient against central differences (step 1e-6 in fp64: truncation
~1e-12 relative to the third derivative, rounding ~1e-10; bound 1e-6)."""
import numpy as np
import pytest

from oracle import block as ob


def directional(f, args, grads, rng, eps=1e-6):
    """max over the arguments of |difference quotient - gradient . direction|, relative."""
    worst = 0.0
    for k, g in grads.items():
        d = rng.standard_normal(args[k].shape)
        up, dn = dict(args), dict(args)
        up[k], dn[k] = args[k] + eps * d, args[k] - eps * d
        num, ana = (f(**up) - f(**dn)) / (2 * eps), float((g * d).sum())
        worst = max(worst, abs(num - ana) / max(abs(ana), 1e-3))
    return worst


def test_conv_by_hand():
    # one channel, taps (1, 10, 100), state (2, 3), tokens 4, 5: 100*4 + 10*3 + 2 and 100*5 + 10*4 + 3
    r = ob.conv(np.array([[4.0], [5.0]]), np.array([[1.0, 10.0, 100.0]]), np.array([0.5]), np.array([[[2.0], [3.0]]]),
                [2], silu=False, dy=np.array([[1.0], [1.0]]))
    assert r["y"][:, 0].tolist() == [432.5, 543.5] and r["last"][0, :, 0].tolist() == [4.0, 5.0]
    assert r["dx"][:, 0].tolist() == [110.0, 100.0] and r["dstate"][0, :, 0].tolist() == [1.0, 11.0]
    assert r["dw"][0].tolist() == [5.0, 7.0, 9.0] and r["db"].tolist() == [2.0]


@pytest.mark.parametrize("W,silu", [(2, True), (3, False), (4, True)])
def test_conv_gradients(W, silu):
    rng = np.random.default_rng(W)
    lens, C = [3, 0, 1, 6], 5
    T = sum(lens)
    a = dict(x=rng.standard_normal((T, C)), w=rng.standard_normal((C, W)), bias=rng.standard_normal(C),
             state=rng.standard_normal((4, W - 1, C)))
    dy, dl = rng.standard_normal((T, C)), rng.standard_normal((4, W - 1, C))
    r = ob.conv(**a, lens=lens, silu=silu, dy=dy, dlast=dl)

    def loss(**k):
        o = ob.conv(**k, lens=lens, silu=silu)
        return (o["y"] * dy).sum() + (o["last"] * dl).sum()

    assert directional(loss, a, dict(x=r["dx"], w=r["dw"], bias=r["db"], state=r["dstate"]), rng) < 1e-6


def test_ssm_closed_form():
    # constant inputs, no softplus: h_t = a h + c, a geometric sum
    T, A = 7, -0.3
    one = np.ones((T, 1))
    r = ob.ssm(2 * one, 0.5 * one, np.array([[A]]), one[:, None], 3 * one[:, None], np.array([0.25]), None, None, [T],
               with_softplus=False)
    a = np.exp(0.5 * A)
    h = [sum(a ** i for i in range(t + 1)) for t in range(T)]
    assert np.allclose(r["y"][:, 0], 3 * np.array(h) + 0.5, rtol=1e-14)


@pytest.mark.parametrize("soft", [True, False])
def test_ssm_gradients(soft):
    rng = np.random.default_rng(3)
    lens, D, G, N = [4, 0, 1, 5], 6, 2, 4
    T = sum(lens)
    a = dict(x=rng.standard_normal((T, D)), dt=rng.standard_normal((T, D)) * 0.5, A=-np.exp(rng.standard_normal((D, N)) * 0.3),
             Bm=rng.standard_normal((T, G, N)), Cm=rng.standard_normal((T, G, N)), Dskip=rng.standard_normal(D),
             dt_bias=rng.standard_normal(D) * 0.1, S0=rng.standard_normal((4, D, N)))
    dy, dS = rng.standard_normal((T, D)), rng.standard_normal((4, D, N))
    r = ob.ssm(**a, lens=lens, with_softplus=soft, dy=dy, dS_T=dS)

    def loss(**k):
        o = ob.ssm(**k, lens=lens, with_softplus=soft)
        return (o["y"] * dy).sum() + (o["S_T"] * dS).sum()

    g = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", Dskip="dD", dt_bias="ddt_bias", S0="dS0")
    assert directional(loss, a, {k: r[v] for k, v in g.items()}, rng) < 1e-6
    assert np.array_equal(r["dS0"][1], dS[1]) and np.array_equal(r["S_T"][1], a["S0"][1])  # the empty sequence


@pytest.mark.parametrize("post,gate,scale,res,pre", [(1, 1, 0, 0, 0), (0, 0, 0, 1, 1), (1, 1, 1, 1, 1), (0, 0, 0, 0, 1),
                                                     (0, 1, 1, 1, 0)])
def test_norm_gradients(post, gate, scale, res, pre):
    rng = np.random.default_rng(7)
    R, D = 4, 9
    a = dict(x=rng.standard_normal((R, D)))
    for on, k, shape in ((post, "w_post", (D,)), (gate, "z", (R, D)), (scale, "scale", (D,)), (res, "residual", (R, D)),
                         (pre, "w_pre", (D,))):
        if on:
            a[k] = rng.standard_normal(shape)
    dr = rng.standard_normal((R, D)) if res or not pre else None
    dy = rng.standard_normal((R, D)) if pre else None

    def loss(**k):
        r, y = ob.norm(**k)
        return ((r * dr).sum() if dr is not None else 0.0) + ((y * dy).sum() if dy is not None else 0.0)

    r, _ = ob.norm(**a)
    ins = {k: v for k, v in a.items() if k != "residual"}
    g = ob.norm_grad(**ins, r=r, dr=dr, dy=dy) if pre or res else ob.norm_grad(**ins, dr=dr)
    names = {"x": "dx", "w_post": "dw_post", "z": "dz", "scale": "dscale", "residual": "dresidual", "w_pre": "dw_pre"}
    assert directional(loss, a, {k: g[names[k]] for k in a}, rng) < 1e-6


def test_step_is_the_recurrence():
    """One step equals the token recurrence of the operator's own reference at T = 1."""
    import torch

    import oracle
    from chunked_gated_delta_04_gb300.inputs import make_inputs, small_workload

    w = small_workload("step", torch.float32, B=3, T=1, Hk=2, Hv=4, DK=16, DV=32, layout="VK")
    inp = make_inputs(w)
    ref = oracle.reference(inp, "VK")
    n = {k: v.double().numpy() for k, v in inp.items() if k in ("q", "k", "v", "g", "beta", "S0")}
    o, S = ob.step(n["q"][:, 0], n["k"][:, 0], n["v"][:, 0], n["g"][:, 0], n["beta"][:, 0], n["S0"])
    assert np.allclose(o, ref["o"][:, 0], rtol=1e-12, atol=1e-12) and np.allclose(S, ref["S_T"], rtol=1e-12, atol=1e-12)
