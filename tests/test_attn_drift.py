"""The running softmax over many tiles: while the maximum stays where it is, what has been summed stays what it is.

Scores are exact in 32 bits and large, the largest lie in the first tile, and every block takes a whole row of tiles, so that what a
tile does wrong to the sums before it adds up.  A feature of V is 1 at one key and 0 at all others: its output is that key's weight,
without a sum over the keys.  Bounds, relative, each of them of arithmetic in 32 bits (E = 2^-24):
  weight   the exponent's rounding and log2(e)'s, E times its size each (11 at most, the scores lie 7.5 apart), times ln 2, and exp2, 2^-22
  sum      of N tiles: N roundings and 40 more within a tile, over warps and parts, each E of it, and the weights' own
  output   1 / l, its product and the parts' weights: 8 roundings; bf16: the weight and the output to 2^-8 each
  lse      the maximum times log2(e) / sqrt(D) is rounded once, and so is the result: 3 E of it, and the sum's relative error
"""
import math

import numpy as np
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
E, U = 2.0 ** -24, {F32: 0.0, BF: 2.0 ** -8}
SCALE = 0.25  # a power of two


def keys(m, D, far):
    """Feature 0 sets the scores' size, the next 15 their distances, the first 64 keys' the largest."""
    g = torch.Generator().manual_seed(m)
    k = torch.zeros(m, D)
    k[:, 0] = far
    k[:, 1:16] = torch.randint(-1, 2, (m, 15), generator=g).float()
    k[:64, 1:16] = 1
    return k


def queries(count, D):
    """Multiples of 1/16 from 8 to 16 for feature 0: exact in bf16, as their products are in 32 bits."""
    q = torch.zeros(count, D)
    q[:, 0] = 8 + (torch.arange(count) * 37 % 128) / 16
    q[:, 1:16] = 1
    return q


def values(m, D):
    at = torch.linspace(0, m - 1, D).long()
    v = torch.zeros(m, D)
    v[at, torch.arange(D)] = 1
    return v, at


def reference(q, k, at):
    """Of the queries [n, D]: weights of the keys `at`, and lse."""
    s = SCALE * (q[:128].double() @ k.double().T).numpy()  # every 128th query is the same
    top = s.max(-1, keepdims=True)
    e = np.exp(s - top)
    l = e.sum(-1, keepdims=True)
    each = np.arange(len(q)) % 128
    return (e / l)[:, at.numpy()][each], (np.log(l) + top)[each, 0]


def bounds(tiles, dtype):
    weight = 22 * E * math.log(2) + 2.0 ** -22
    total = (tiles + 40) * E + weight
    return weight + total + 8 * E + (1 + U[dtype]) ** 2 - 1, total


@pytest.mark.parametrize("D,far,m", [(16, 64.0, 8192), (16, 512.0, 8192), (80, 512.0, 8192), (64, 512.0, 32768)])
def test_forward(D, far, m):
    """320 heads of one tile of queries: more tiles than the GPU holds blocks, so that none is shared."""
    H, n = 320, 3
    q, k = queries(H * n, D), keys(m, D, far)
    v, at = values(m, D)
    o, lse = gdr.attn_forward(q.view(1, n, H, D).cuda(), k.view(1, m, 1, D).cuda(), v.view(1, m, 1, D).cuda(), causal=False, scale=SCALE)
    w, ref = reference(q, k, at)
    rel, total = bounds(m // 64, F32)
    assert (np.abs(o.double().cpu().numpy().reshape(-1, D) - w) <= rel * w).all()
    got = lse[0].T.reshape(-1).double().cpu().numpy()
    assert (np.abs(got - ref) <= total + 3 * E * np.abs(ref)).all()


@pytest.mark.parametrize("dtype,G,m,far", [(F32, 1, 8192, 64.0), (F32, 1, 8192, 512.0), (F32, 4, 16384, 512.0), (F32, 8, 8192, 512.0),
                                           (BF, 1, 65536, 512.0), (BF, 5, 65536, 512.0)])
@pytest.mark.parametrize("B", [304, 1])
def test_step(dtype, G, m, far, B):
    """304 rows that share their pages but for the last one: a row for each block.  One row: every block has a part of it."""
    D, size = 64, 64
    q, k = queries(B * G, D), keys(m, D, far)
    v, at = values(m, D)
    pages = m // size
    table = torch.arange(pages).repeat(B, 1)
    table[:, -1] = pages - 1 + torch.arange(B)
    rows = lambda t: torch.cat([t[:-size].view(-1, size, 1, D), t[-size:].view(1, size, 1, D).expand(B, -1, -1, -1)]).to(dtype).cuda()
    last = lambda t: t[-1].expand(B, 1, D).to(dtype).cuda().contiguous()
    o = gdr.attn_step(q.view(B, G, D).to(dtype).cuda(), last(k), last(v), rows(k), rows(v), table.to(torch.int32).cuda(),
                      torch.full((B,), m - 1, dtype=torch.int32).cuda(), scale=SCALE)
    w, _ = reference(q, k, at)
    rel, _ = bounds(m // (64 if dtype == BF else 32), dtype)
    assert (np.abs(o.double().cpu().numpy().reshape(-1, D) - w) <= rel * w).all()
