"""fp64 references of the operators around the gated delta rule (``include/gdr_block.h``), written
from their formulas in numpy, token by token.  Used by the tests only; shares no code with the CUDA
path.  ``lens`` lists the sequence lengths of a packed batch: activations are [tokens, ...].
"""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    out = np.empty_like(x)
    pos = x >= 0
    out[pos] = 1.0 / (1.0 + np.exp(-x[pos]))
    e = np.exp(x[~pos])
    out[~pos] = e / (1.0 + e)
    return out


def softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int)


# ---------------------------------------------------------------------------------- convolution
def conv(x, w, bias, state, lens, silu=True, dy=None, dlast=None):
    """dict of y, last and, with dy, dx, dw, db, dstate."""
    W, C = w.shape[1], w.shape[0]
    at = starts(lens)
    y, last = np.zeros_like(x), np.zeros((len(lens), W - 1, C))
    dx, dstate, dw, db = np.zeros_like(x), np.zeros_like(last), np.zeros_like(w), np.zeros(C)
    for n, L in enumerate(lens):
        X = np.concatenate([state[n] if state is not None else np.zeros((W - 1, C)), x[at[n]:at[n + 1]]])
        dX = np.zeros_like(X)
        last[n] = X[L:]
        if dlast is not None:
            dX[L:] += dlast[n]
        for t in range(L):
            pre = (w.T * X[t:t + W]).sum(0) + (bias if bias is not None else 0.0)
            s = sigmoid(pre)
            y[at[n] + t] = pre * s if silu else pre
            if dy is not None:
                d = dy[at[n] + t] * (s * (1 + pre * (1 - s)) if silu else 1.0)
                dX[t:t + W] += w.T * d
                dw += (d * X[t:t + W]).T
                db += d
        dx[at[n]:at[n + 1]] = dX[W - 1:]
        dstate[n] = dX[:W - 1]
    out = {"y": y, "last": last}
    if dy is not None:
        out.update(dx=dx, dw=dw, db=db, dstate=dstate)
    return out


# ------------------------------------------------------------------------------- selective scan
def ssm(x, dt, A, Bm, Cm, Dskip, dt_bias, S0, lens, with_softplus=True, dy=None, dS_T=None):
    """x, dt [tokens, D], Bm, Cm [tokens, G, N]: dict of y, S_T, states (in front of every token) and,
    with dy, dx, ddt, dA, dB, dC, dD, ddt_bias, dS0."""
    T, D = x.shape
    G, N = Bm.shape[1:]
    group = np.arange(D) // (D // G)
    raw = dt + (dt_bias if dt_bias is not None else 0.0)
    delta = softplus(raw) if with_softplus else raw
    skip = Dskip if Dskip is not None else np.zeros(D)
    at = starts(lens)
    y, before, S_T = np.zeros_like(x), np.zeros((T, D, N)), np.zeros((len(lens), D, N))
    for n in range(len(lens)):
        h = S0[n].copy() if S0 is not None else np.zeros((D, N))
        for t in range(at[n], at[n + 1]):
            before[t] = h
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * Bm[t, group]
            y[t] = (h * Cm[t, group]).sum(-1) + skip * x[t]
        S_T[n] = h
    out = {"y": y, "S_T": S_T, "states": before}
    if dy is None:
        return out
    dx, ddelta, dA = np.zeros_like(x), np.zeros_like(x), np.zeros_like(A)
    dB, dC, dS0 = np.zeros_like(Bm), np.zeros_like(Cm), np.zeros_like(S_T)
    for n in range(len(lens)):
        dh = dS_T[n].copy() if dS_T is not None else np.zeros((D, N))
        for t in range(at[n + 1] - 1, at[n] - 1, -1):
            a = np.exp(delta[t][:, None] * A)
            b, c = Bm[t, group], Cm[t, group]
            h = a * before[t] + (delta[t] * x[t])[:, None] * b
            dh = dh + dy[t][:, None] * c
            for g in range(G):
                ch = group == g
                dC[t, g] = (dy[t][ch, None] * h[ch]).sum(0)
                dB[t, g] = (dh[ch] * (delta[t] * x[t])[ch, None]).sum(0)
            dlog = dh * a * before[t]
            dA += dlog * delta[t][:, None]
            into = (dh * b).sum(-1)
            dx[t] = into * delta[t] + skip * dy[t]
            ddelta[t] = (dlog * A).sum(-1) + into * x[t]
            dh = a * dh
        dS0[n] = dh
    ddt = ddelta * (sigmoid(raw) if with_softplus else 1.0)
    out.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dy * x).sum(0), ddt_bias=ddt.sum(0), dS0=dS0)
    return out


# ---------------------------------------------------------------------------------- block norms
def norm(x, w_post=None, z=None, scale=None, residual=None, w_pre=None, eps=1e-6, store=lambda v: v):
    """(r, y); store rounds r as the caller's type does."""
    u = x
    if w_post is not None:
        u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * w_post
    if z is not None:
        u = u * z * sigmoid(z)
    if scale is not None:
        u = u * scale
    r = store(u + residual) if residual is not None else u
    y = None
    if w_pre is not None:
        y = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * w_pre
    return r, y


def norm_grad(x, w_post=None, z=None, scale=None, r=None, w_pre=None, dr=None, dy=None, eps=1e-6):
    """dict of dx, dz, dresidual, dw_post, dscale, dw_pre; r is the stored stream."""
    out = {}
    du = np.zeros_like(x) if dr is None else dr
    if w_pre is not None:
        rs = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
        rh, t = r * rs, dy * w_pre
        du = du + rs * (t - rh * (t * rh).mean(-1, keepdims=True))
        out["dw_pre"] = (dy * rh).sum(0)
    out["dresidual"] = du
    rx = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * rx if w_post is not None else x
    n = xh * w_post if w_post is not None else xh
    s = sigmoid(z) if z is not None else None
    act = z * s if z is not None else 1.0
    sc = scale if scale is not None else 1.0
    out["dscale"] = (du * n * act).sum(0)
    if z is not None:
        out["dz"] = du * sc * n * s * (1 + z * (1 - s))
    t = du * sc * act
    if w_post is not None:
        out["dw_post"] = (t * xh).sum(0)
        t = t * w_post
        t = rx * (t - xh * (t * xh).mean(-1, keepdims=True))
    out["dx"] = t
    return out


# ----------------------------------------------------------------- the delta rule, one token each
def step(q, k, v, g, beta, S, scale=None, l2norm=False, logsigmoid=False, sig=False):
    """q, k [B, Hk, DK], v [B, Hv, DV], S [B, Hv, DV, DK]: (o, S after the token)."""
    B, Hk, DK = q.shape
    Hv = v.shape[1]
    if l2norm:
        q, k = (t / np.sqrt((t * t).sum(-1, keepdims=True) + 1e-6) for t in (q, k))
    if logsigmoid:
        g = -softplus(-g)
    if sig:
        beta = sigmoid(beta)
    o, S = np.zeros_like(v), S.copy()
    for b in range(B):
        for h in range(Hv):
            kh, qh = k[b, h // (Hv // Hk)], q[b, h // (Hv // Hk)]
            M = S[b, h]
            M = np.exp(g[b, h]) * (M - beta[b, h] * np.outer(M @ kh, kh)) + beta[b, h] * np.outer(v[b, h], kh)
            S[b, h] = M
            o[b, h] = (1 / np.sqrt(DK) if scale is None else scale) * (M @ qh)
    return o, S
