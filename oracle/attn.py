"""fp64 references of the attention mixer (``include/gdr_attn.h``), written from its formulas in numpy, head by head.
Used by the tests only; shares no code with the CUDA path.

Besides the values ``attention`` and ``step`` give an elementwise bound of the error that their arithmetic allows:
every input is exact, products and sums run in 32 bits, and for 16-bit problems the probabilities, the gradients of the scores
and the outputs are rounded by at most ``u`` (half a step, relative).
"""
from __future__ import annotations

import math

import numpy as np

E = 2.0 ** -24  # half a step of fp32


# -------------------------------------------------------------------------------- rotary positions
def rope(x, freqs, positions, interleaved=False, scale=1.0, inverse=False):
    """x [tokens, H, D], positions [tokens]: rotated by position * freq, pair by pair."""
    y, R = x.copy(), 2 * len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        t = positions.astype(np.float64) * f * (-1 if inverse else 1)
        c, s = (np.cos(t) * scale)[:, None], (np.sin(t) * scale)[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


# --------------------------------------------------------------------------------------- attention
def sees(n, m, causal, window):
    """[n, m]: query i sees key j."""
    i, j = np.arange(n)[:, None] + (m - n), np.arange(m)[None]
    on = np.ones((n, m), bool)
    if causal:
        on &= j <= i
    if window:
        on &= j > i - window
    return on


def _softmax(s, on):
    top = np.where(on, s, -np.inf).max(-1, initial=-np.inf)
    base = np.where(np.isneginf(top), 0.0, top)
    e = np.where(on, np.exp(np.where(on, s - base[..., None], 0.0)), 0.0)
    l = e.sum(-1)
    with np.errstate(divide="ignore"):
        lse = np.log(l) + base
    return e / np.where(l == 0, 1.0, l)[..., None], lse


def _score_error(q, k, scale, s, lse, on, D):
    """Relative error of a probability from its score: a sum of D products (each partial sum off by E of its size), the
    score's distance from the maximum and from lse (a few roundings of numbers up to |s| + |lse|), exp2 itself (2^-22)."""
    mag = scale * (np.abs(q) @ np.abs(k).T)
    ref = np.where(np.isfinite(lse), np.abs(lse), 0.0)[:, None]
    each = (D + 4) * E * mag + 6 * E * (np.abs(s) + ref) + 4 * 2.0 ** -22
    return 2 * np.where(on, each, 0.0).max(-1, keepdims=True, initial=0.0) + 0 * s


def attention(q, k, v, q_lens, k_lens, causal=True, window=0, scale=None, do=None, u=0.0):
    """q, do [tokens, Hq, D], k, v [tokens, Hk, D], packed by q_lens and k_lens: dict of o, lse [Hq, tokens] and, with do, dq, dk,
    dv; and dict of their bounds."""
    (Tq, Hq, D), (Tk, Hk, _) = q.shape, k.shape
    G = Hq // Hk
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = {"o": np.zeros_like(q), "lse": np.full((Hq, Tq), -np.inf), "dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    tol = {name: np.zeros_like(a) for name, a in out.items()}
    tol["lse"] = np.zeros((Hq, Tq))
    a = b = 0
    for n, m in zip(q_lens, k_lens):
        on = sees(n, m, causal, window)
        for h in range(Hq):
            Q, K, V = q[a:a + n, h], k[b:b + m, h // G], v[b:b + m, h // G]
            s = scale * (Q @ K.T)
            p, lse = _softmax(s, on)
            e = _score_error(Q, K, scale, s, lse, on, D)
            rows = (m + 8) * E  # of a sum over the keys
            o = p @ V
            out["o"][a:a + n, h], out["lse"][h, a:a + n] = o, lse
            # the sum that o is divided by is off as the probabilities are
            o_tol = ((u + 2 * e + 2 * rows) * p) @ np.abs(V) * (1 + u)
            tol["o"][a:a + n, h] = o_tol + (u + E) * np.abs(o)
            tol["lse"][h, a:a + n] = np.where(np.isfinite(lse), e.max(-1, initial=0.0) + rows + 4 * E * np.abs(lse), 0.0)
            if do is None:
                continue
            g = do[a:a + n, h]
            dp = g @ V.T
            delta = (g * o).sum(-1, keepdims=True)
            ds = np.where(on, p * (dp - delta), 0.0)
            # delta from the o that was stored, dp from its sums
            delta_tol = (np.abs(g) * (o_tol + u * np.abs(o))).sum(-1, keepdims=True) + (D + 4) * E * (np.abs(g) * np.abs(o)).sum(-1, keepdims=True)
            ds_tol = np.where(on, (u + 3 * e) * np.abs(ds) + p * (1 + u) * (delta_tol + (D + 4) * E * (np.abs(g) @ np.abs(V).T)), 0.0)
            out["dv"][b:b + m, h // G] += p.T @ g
            tol["dv"][b:b + m, h // G] += ((u + 3 * e + (n * G + 8) * E) * p).T @ np.abs(g)
            out["dq"][a:a + n, h] = scale * ds @ K
            tol["dq"][a:a + n, h] = scale * (ds_tol + rows * np.abs(ds)) @ np.abs(K) + (u + 2 * E) * np.abs(scale * ds @ K)
            out["dk"][b:b + m, h // G] += scale * ds.T @ Q
            tol["dk"][b:b + m, h // G] += scale * (ds_tol + (n * G + 8) * E * np.abs(ds)).T @ np.abs(Q)
        a, b = a + n, b + m
    for name in ("dk", "dv"):
        tol[name] += (u + 2 * E) * np.abs(out[name])
    if do is None:
        for name in ("dq", "dk", "dv"):
            del out[name], tol[name]
    return out, tol


# ----------------------------------------------------------------------------------- a paged cache
def write(k, v, k_cache, v_cache, table, starts, lens):
    """k, v [tokens, Hk, D], packed by lens, into copies of the caches; what has no place is left out."""
    kc, vc = k_cache.copy(), v_cache.copy()
    pages, size = kc.shape[:2]
    t = 0
    for n, L in enumerate(lens):
        for i in range(L):
            pos = int(starts[n]) + i
            if 0 <= pos < table.shape[1] * size and 0 <= table[n, pos // size] < pages:
                kc[table[n, pos // size], pos % size], vc[table[n, pos // size], pos % size] = k[t], v[t]
            t += 1
    return kc, vc


def step(q, k, v, k_cache, v_cache, table, lengths, window=0, scale=None, u=0.0):
    """One token per row: (o, its bound, k_cache, v_cache)."""
    pages, size = k_cache.shape[:2]
    room = table.shape[1] * size
    live = [0 <= n < room for n in lengths]
    kc, vc = k_cache.copy(), v_cache.copy()
    for b, n in enumerate(lengths):
        if live[b]:
            kc, vc = write(k[b:b + 1], v[b:b + 1], kc, vc, table[b:b + 1], [n], [1])
    o, tol = np.zeros_like(q), np.zeros_like(q)
    for b, n in enumerate(lengths):
        if not live[b]:
            continue
        at = np.arange(max(0, n + 1 - window) if window else 0, n + 1)
        page = table[b, at // size]
        if (page < 0).any() or (page >= pages).any():
            continue
        r, t = attention(q[b:b + 1], kc[page, at % size], vc[page, at % size], [1], [len(at)], True, 0, scale, u=u)
        o[b], tol[b] = r["o"][0], t["o"][0]
    return o, tol, kc, vc
