"""GPU parity of the attention mixer with its fp64 references.  The references bound the error of every element from the
arithmetic (``oracle/attn.py``); u is half a step of the output's type."""
import math

import numpy as np
import pytest
import torch

import chunked_gated_delta_04_gb300 as gdr
from oracle import attn as oa

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
U = {F32: 0.0, BF: 2.0 ** -8}


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *shape, dtype=F32: torch.randn(*shape, generator=g).to(dtype).cuda()


def npy(t):
    return t.detach().double().cpu().numpy()


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()


def check(got, ref, tol, name):
    got = npy(got).reshape(ref.shape)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), name
    fine = np.isfinite(ref)
    assert np.isfinite(got[fine]).all(), name
    over = np.abs(got - ref, where=fine, out=np.zeros_like(ref)) - tol
    assert not (over[fine] > 0).any(), (name, float(over[fine].max()), float(np.abs(got - ref)[fine].max()), np.argwhere((over > 0) & fine)[:5].tolist())


# -------------------------------------------------------------------------------- rotary positions
def rope_bound(x, dtype, scale):
    """Angle off by 2^-25 turns of half a turn's sine argument (2e-7 with its rounding) and sines by 2^-22; two products and a sum."""
    pair = np.abs(x).max(-1, keepdims=True) * 2 * abs(scale)
    return pair * 8e-7 + np.zeros_like(x)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (80, 80), (64, 32), (48, 38), (32, 2), (10, 6)])
def test_rope(dtype, interleaved, D, R):
    r = gen(R)
    qkv = r(2, 37, 9, D, dtype=dtype)  # a projection that q and k are slices of
    q, k = qkv[:, :, :5], qkv[:, :, 5:7]
    freqs, _ = gdr.rope_frequencies(R)
    pos = torch.randint(-5, 1 << 20, (2, 37), dtype=torch.int32).cuda()
    for positions in (None, pos):
        at = npy(torch.arange(37).expand(2, 37) if positions is None else positions).reshape(-1)
        for way in (gdr.rope_forward, gdr.rope_backward):
            a, b = way(q, k, freqs, positions, interleaved=interleaved, scale=1.25)
            for got, x in ((a, q), (b, k)):
                ref = oa.rope(npy(x).reshape(74, -1, D), npy(freqs), at, interleaved, 1.25, way is gdr.rope_backward)
                check(got, ref, rope_bound(npy(x).reshape(ref.shape), dtype, 1.25) + U[dtype] * np.abs(ref), "rope")
                assert torch.equal(got[..., R:], x[..., R:]) and got.is_contiguous()


def test_rope_far_positions():
    """The last int32 positions: fp32 angles would be off by whole turns."""
    r = gen(3)
    q = r(4, 2, 64)
    freqs, _ = gdr.rope_frequencies(64)
    pos = torch.tensor([2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, 123456789], dtype=torch.int32).cuda()
    got, none = gdr.rope_forward(q, None, freqs, pos)
    assert none is None
    ref = oa.rope(npy(q), npy(freqs), npy(pos))
    # here the reference's own angle is rounded: position * freq to 2^-53 of up to 2^31 radians
    check(got, ref, rope_bound(npy(q), F32, 1.0) + np.abs(npy(q)).max() * 2 * 2.0 ** 31 * 2.0 ** -52, "rope")


def test_rope_packed_places_and_views():
    r = gen(4)
    lens = [3, 0, 1, 40]
    q, k = r(1, 44, 3, 64, dtype=BF), r(1, 44, 1, 64, dtype=BF)
    freqs, _ = gdr.rope_frequencies(32)
    at = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()[None]
    one = gdr.rope_forward(q, k, freqs, cu_seqlens=cu_of(lens))
    two = gdr.rope_forward(q, k, freqs, at)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    flat = torch.empty(q.numel() + 1, dtype=BF, device="cuda")  # not aligned to 16 bytes: the same values
    odd = flat[1:].view(q.shape).copy_(q)
    assert torch.equal(gdr.rope_forward(odd, k, freqs, at)[0], two[0])
    row = gdr.rope_forward(q[0], k[0], freqs, at[0])
    assert torch.equal(row[0], two[0][0])


def test_rope_autograd():
    r = gen(5)
    q, k = r(2, 9, 4, 32).requires_grad_(), r(2, 9, 2, 32).requires_grad_()
    freqs, scale = gdr.rope_frequencies(32, scaling="yarn", factor=8.0)
    a, b = gdr.rope(q, k, freqs, scale=scale)
    ga = r(2, 9, 4, 32)
    gq, gk = torch.autograd.grad(a, (q, k), ga, retain_graph=True)
    ref = oa.rope(npy(ga).reshape(18, 4, 32), npy(freqs), np.tile(np.arange(9), 2), scale=scale, inverse=True)
    check(gq, ref, rope_bound(npy(ga).reshape(ref.shape), F32, scale), "dq")
    assert not gk.any()
    gq, gk = torch.autograd.grad(b.sum(), (q, k))
    assert not gq.any() and gk.any()


def test_rope_frequencies():
    plain, one = gdr.rope_frequencies(64, device="cpu")
    assert one == 1.0 and plain.dtype == torch.float64 and torch.allclose(plain, 10000.0 ** -(torch.arange(32).double() / 32), rtol=1e-15)
    lin, _ = gdr.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(lin, plain / 4)
    ntk, _ = gdr.rope_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and torch.allclose(ntk[-1], plain[-1] / 4, rtol=1e-13)
    yarn, s = gdr.rope_frequencies(64, scaling="yarn", factor=16.0, original_length=4096, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(yarn[turns >= 32], plain[turns >= 32]) and torch.equal(yarn[turns <= 1], plain[turns <= 1] / 16)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (yarn[mid] < plain[mid]).all() and (yarn[mid] > plain[mid] / 16).all() and abs(s - 1.27725887) < 1e-8
    for bad in (dict(rotary_dim=7), dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, scaling="other"),
                dict(rotary_dim=8, scaling="yarn", beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(ValueError):
            gdr.rope_frequencies(**bad, device="cpu")


# --------------------------------------------------------------------------------------- attention
def attn_case(dtype, q_lens, k_lens, Hq, Hk, D, causal=True, window=0, scale=None, packed=True, train=True, seed=0, same_cu=False):
    r = gen(seed)
    B = 1 if packed else len(q_lens)
    Tq, Tk = (sum(q_lens), sum(k_lens)) if packed else (q_lens[0], k_lens[0])
    q, k, v, do = r(B, Tq, Hq, D, dtype=dtype), r(B, Tk, Hk, D, dtype=dtype), r(B, Tk, Hk, D, dtype=dtype), r(B, Tq, Hq, D, dtype=dtype)
    how = dict(causal=causal, window=window, scale=scale)
    if packed:
        how.update(cu_seqlens=cu_of(q_lens), cu_seqlens_k=None if same_cu else cu_of(k_lens))
    o, lse = gdr.attn_forward(q, k, v, **how)
    ref, tol = oa.attention(*[npy(t).reshape(-1, *t.shape[2:]) for t in (q, k, v)], q_lens, k_lens, causal, window, scale,
                            npy(do).reshape(-1, Hq, D) if train else None, U[dtype])
    got = {"o": o, "lse": lse if packed else lse.transpose(0, 1).reshape(Hq, -1)}
    if train:
        got.update(zip(("dq", "dk", "dv"), gdr.attn_backward(q, k, v, o, lse, do, **how)))
    for name, t in got.items():
        check(t, ref[name].reshape(npy(t).shape), tol[name].reshape(npy(t).shape), name)
    return q, k, v, do, how, got


SHAPES = [  # queries and keys of the sequences
    ([1], [1]), ([64], [64]), ([65], [65]), ([128], [128]), ([129], [129]), ([300], [300]), ([257], [513]), ([513], [200]), ([7], [700]), ([700], [7])]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,m", SHAPES)
def test_attention_lengths(dtype, D, n, m):
    attn_case(dtype, n * 2, m * 2, 4, 2, D, packed=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [16, 32, 48, 80, 96, 112])
def test_attention_head_sizes(dtype, D):
    attn_case(dtype, [150], [170], 3, 1, D, packed=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [0, 1, 60, 128, 333])
def test_attention_masks(dtype, causal, window):
    attn_case(dtype, [290, 290], [400, 400], 2, 2, 64, causal, window, packed=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 1), (8, 2), (6, 6)])
def test_attention_heads(dtype, Hq, Hk):
    attn_case(dtype, [200], [200], Hq, Hk, 128, scale=0.3, packed=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D,n,m,Hq,Hk,B", [(128, 150, 150, 20, 20, 4), (64, 260, 129, 32, 16, 3), (80, 129, 400, 24, 24, 2)])
def test_attention_many_tiles(dtype, D, n, m, Hq, Hk, B):
    """Tiles enough that no two blocks share one, and that blocks take several."""
    attn_case(dtype, [n] * B, [m] * B, Hq, Hk, D, packed=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,m,Hq,Hk", [(1, 5000, 2, 1), (100, 3001, 1, 1), (2000, 2000, 3, 1), (640, 640, 16, 2), (129, 1500, 6, 2)])
def test_attention_few_tiles(dtype, n, m, Hq, Hk):
    """Few tiles of many steps, which blocks share."""
    attn_case(dtype, [n], [m], Hq, Hk, 64, packed=False)
    attn_case(dtype, [n], [m], Hq, Hk, 128, window=700, packed=False, train=n > 1)


PACKED = [([130, 1, 0, 257, 64], None), ([100, 0, 33, 5], [300, 40, 0, 2]), ([0, 0], [5, 0]), ([20, 30, 300], [0, 0, 0]), ([128, 128, 1], None),
          ([3] * 40, [5] * 40)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("q_lens,k_lens", PACKED)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
def test_attention_packed(dtype, q_lens, k_lens, causal, window):
    attn_case(dtype, q_lens, k_lens or q_lens, 4, 2, 64, causal, window, same_cu=k_lens is None)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_attention_of_a_projection(dtype):
    """Slices of one projection, and ones that are not aligned to 16 bytes, give what contiguous tensors give."""
    r = gen(11)
    qkv = r(2, 150, 8, 64, dtype=dtype)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    do = r(2, 150, 6, 64, dtype=dtype)[:, :, 1:5]
    o, lse = gdr.attn_forward(*[t.contiguous() for t in (q, k, v)])
    assert torch.equal(gdr.attn_forward(q, k, v)[0], o)
    want = gdr.attn_backward(*[t.contiguous() for t in (q, k, v)], o, lse, do.contiguous())
    for a, b in zip(gdr.attn_backward(q, k, v, o, lse, do), want):
        assert torch.equal(a, b)
    flat = torch.empty(q.numel() + 1, dtype=dtype, device="cuda")
    odd = flat[1:].view(q.shape).copy_(q)
    got = [gdr.attn_forward(odd, k, v)[0], *gdr.attn_backward(odd, k, v, o, lse, do)]
    for a, b in zip(got, (o, *want)):
        assert (a.float() - b.float()).abs().max() <= 3 * max(U[dtype], 1e-5) * b.float().abs().max()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_attention_is_reproducible(dtype):
    *_, a = attn_case(dtype, [500, 3, 700], [500, 3, 700], 4, 2, 128, seed=5)
    *_, b = attn_case(dtype, [500, 3, 700], [500, 3, 700], 4, 2, 128, seed=5)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (80, 40)])  # tiles that blocks share, and tiles enough
def test_sequences_do_not_reach_one_another(dtype, packed, Hq, Hk):
    """NaN and infinities in one sequence leave the others' results bit for bit what they are."""
    lens = [100, 60, 170] if packed else [100, 100, 100]
    r = gen(12)
    shape = (1, sum(lens)) if packed else (3, 100)
    ts = [r(*shape, h, 64, dtype=dtype) for h in (Hq, Hk, Hk, Hq)]
    how = dict(cu_seqlens=cu_of(lens)) if packed else {}

    def run(q, k, v, do):
        o, lse = gdr.attn_forward(q, k, v, **how)
        return [o, *gdr.attn_backward(q, k, v, o, lse, do, **how)]

    sound = run(*ts)
    spoilt = [t.clone() for t in ts]
    for t in spoilt:
        view = t.view(-1, *t.shape[2:])[lens[0]:lens[0] + lens[1]]
        view[0], view[-1], view[7] = float("nan"), float("inf"), -float("inf")
    for a, b in zip(run(*spoilt), sound):
        a, b = a.view(-1, *a.shape[2:]), b.view(-1, *b.shape[2:])
        assert torch.equal(a[:lens[0]], b[:lens[0]]) and torch.equal(a[lens[0] + lens[1]:], b[lens[0] + lens[1]:])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,T", [(2, 300), (40, 700)])
def test_a_query_that_is_not_a_number(dtype, H, T):
    """Its row is not a number, and the others are bit for bit what they were."""
    r = gen(15)
    q, k, v = (r(2, T, H, 64, dtype=dtype) for _ in range(3))
    want, lse = gdr.attn_forward(q, k, v)
    bad = q.clone()
    bad[1, 150] = float("nan")
    o, ls = gdr.attn_forward(bad, k, v)
    assert o[1, 150].isnan().all() and ls[1, :, 150].isnan().all()
    keep = torch.ones(2, T, dtype=torch.bool, device="cuda")
    keep[1, 150] = False
    assert torch.equal(o[keep], want[keep]) and torch.equal(ls.transpose(1, 2)[keep], lse.transpose(1, 2)[keep])
    table, lengths = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.tensor([3, 5], dtype=torch.int32).cuda()
    table[1] = 1
    kc, vc = k[:, :16].contiguous(), v[:, :16].contiguous()
    o = gdr.attn_step(bad[:, 150], k[:, 0], v[:, 0], kc, vc, table, lengths)
    assert torch.isfinite(o[0]).all() and o[1].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_sequences(dtype):
    """More sequences than the tile tables' kernel keeps the bounds of."""
    lens = [3] * 1200 + [200] + [0] * 100 + [1] * 50
    attn_case(dtype, lens, lens, 2, 1, 64, same_cu=True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_large_scores(dtype):
    """Scores of a hundred and more: the running maximum moves far, and what lies far below it counts nothing."""
    r = gen(13)
    q, k, v = r(1, 300, 2, 64, dtype=dtype) * 8, r(1, 300, 2, 64, dtype=dtype) * 8, r(1, 300, 2, 64, dtype=dtype)
    k[:, 150:] *= 2
    o, lse = gdr.attn_forward(q, k, v)
    ref, tol = oa.attention(*[npy(t)[0] for t in (q, k, v)], [300], [300], u=U[dtype])
    check(o, ref["o"][None], tol["o"][None], "o")
    check(lse, ref["lse"][None], tol["lse"][None], "lse")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_attention_autograd(dtype):
    q, k, v, do, how, got = attn_case(dtype, [90, 90], [120, 120], 4, 2, 64, packed=False, seed=6)
    ts = [t.clone().requires_grad_() for t in (q, k, v)]
    o = gdr.attention(*ts, **how)
    assert torch.equal(o, got["o"])
    for a, name in zip(torch.autograd.grad(o, ts, do), ("dq", "dk", "dv")):
        assert torch.equal(a, got[name]), name
    g = torch.autograd.grad(gdr.attention(*ts, **how).sum(), ts)  # a gradient that is a broadcast one
    ones = gdr.attn_backward(q, k, v, got["o"], gdr.attn_forward(q, k, v, **how)[1], torch.ones_like(q), **how)
    assert all(torch.equal(a, b) for a, b in zip(g, ones))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_empty_tensors(dtype):
    for B, Tq, Tk in ((0, 5, 5), (2, 0, 5), (2, 5, 0)):
        q, k = torch.ones(B, Tq, 4, 64, dtype=dtype, device="cuda"), torch.ones(B, Tk, 2, 64, dtype=dtype, device="cuda")
        o, lse = gdr.attn_forward(q, k, k)
        dq, dk, dv = gdr.attn_backward(q, k, k, o, lse, q)
        assert not any(t.any() for t in (o, dq, dk, dv)) and (lse == -math.inf).all()


def test_long_sequence():
    """One head at 20000 tokens: a few queries against the reference of their own rows."""
    r = gen(14)
    T, D = 20000, 128
    q, k, v = r(1, T, 2, D, dtype=BF), r(1, T, 1, D, dtype=BF), r(1, T, 1, D, dtype=BF)
    o, lse = gdr.attn_forward(q, k, v)
    for i in (0, 127, 128, 9999, T - 1):
        ref, tol = oa.attention(*[npy(t)[0] for t in (q[:, i:i + 1], k[:, :i + 1], v[:, :i + 1])], [1], [i + 1], u=U[BF])
        check(o[0, i:i + 1], ref["o"], tol["o"], "o")
        check(lse[0, :, i:i + 1], ref["lse"], tol["lse"], "lse")


# ----------------------------------------------------------------------------------- a paged cache
def pages_for(lengths, size, spare, seed):
    g = torch.Generator().manual_seed(seed)
    need = [-(-(max(n, 0) + 1) // size) for n in lengths]
    free = torch.randperm(sum(need) + spare, generator=g)
    table, at = torch.full((len(lengths), max(need) + 1), -1), 0
    for b, n in enumerate(need):
        table[b, :n] = free[at:at + n]
        at += n
    return table.to(torch.int32).cuda(), len(free)


def step_case(dtype, lengths, size, Hq, Hk, D, window=0, seed=0, table=None, unaligned=False):
    r = gen(seed)
    B = len(lengths)
    tab, pages = pages_for(lengths, size, 3, seed)
    tab = tab if table is None else table(tab)
    # what no row holds is not a number, and must not be seen
    kc, vc = (r(pages, size, Hk, D, dtype=dtype) for _ in range(2))
    held = torch.zeros(pages, size, dtype=torch.bool)
    for b, n in enumerate(lengths):
        for p in range(max(n, 0)):
            if p // size < tab.shape[1] and 0 <= tab[b, p // size] < pages:
                held[tab[b, p // size], p % size] = True
    ref_k, ref_v = npy(kc), npy(vc)
    kc[~held.cuda()], vc[~held.cuda()] = float("nan"), float("inf")
    q, k, v = r(B, Hq, D, dtype=dtype), r(B, Hk, D, dtype=dtype), r(B, Hk, D, dtype=dtype)
    if unaligned:
        q, k, v = (torch.empty(t.numel() + 1, dtype=dtype, device="cuda")[1:].view(t.shape).copy_(t) for t in (q, k, v))
    lens = torch.tensor(lengths, dtype=torch.int32).cuda()
    before = kc.clone(), vc.clone()
    o = gdr.attn_step(q, k, v, kc, vc, tab, lens, window=window)
    ref, tol, rk, rv = oa.step(npy(q), npy(k), npy(v), ref_k, ref_v, tab.cpu().numpy(), lengths, window, u=U[dtype])
    check(o, ref, tol, "o")
    # the new tokens are in their places, and nothing else has changed
    wrote = torch.tensor((rk != ref_k).any((2, 3)))
    for cache, old, new in ((kc, before[0], rk), (vc, before[1], rv)):
        assert torch.equal(cache[~wrote.cuda()].nan_to_num(7.0, 8.0), old[~wrote.cuda()].nan_to_num(7.0, 8.0))
        assert np.array_equal(npy(cache)[wrote.numpy()], new[wrote.numpy()])
    return o


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("size", [1, 7, 16, 64, 100])
@pytest.mark.parametrize("lengths", [[0], [63, 0, 64], [700], [5, 31, 32, 33, 127, 128, 511, 1000]])
def test_step_lengths(dtype, size, lengths):
    step_case(dtype, lengths, size, 4, 2, 64)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 128), (4, 4, 16), (8, 1, 80), (5, 1, 48), (32, 2, 64), (40, 2, 128), (17, 1, 112), (12, 3, 96)])
def test_step_heads(dtype, Hq, Hk, D):
    step_case(dtype, [100, 3, 250], 16, Hq, Hk, D)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("window", [1, 2, 64, 65, 300, 5000])
def test_step_window(dtype, window):
    step_case(dtype, [0, 1, 63, 64, 200, 700], 32, 4, 2, 64, window)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_step_unaligned_inputs(dtype):
    assert torch.equal(step_case(dtype, [90, 17], 16, 4, 2, 64, unaligned=True), step_case(dtype, [90, 17], 16, 4, 2, 64))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_step_rows_that_are_skipped(dtype):
    """Negative and full rows, and ones whose pages are outside the pool: zeros, the others as ever."""
    def table(t):
        t = t.clone()
        t[2, 1] = 1000     # a page that the row needs
        t[3, 0] = -5
        t[5, -1] = 99999   # one that it does not
        return t

    o = step_case(dtype, [40, -1, 150, 3, 300, 20], 16, 4, 2, 64, table=table)
    assert not o[1:4].any() and o[0].any() and o[4].any() and o[5].any()
    full = step_case(dtype, [15, 32], 16, 2, 1, 64, table=lambda t: t[:, :2].contiguous())
    assert full[0].any() and not full[1].any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_step_many_rows_and_a_long_one(dtype):
    step_case(dtype, [(37 * i) % 90 for i in range(300)], 16, 2, 1, 64)
    step_case(dtype, [30000, 2], 64, 4, 1, 128)


def test_step_shares_pages():
    """Rows with a common beginning read the same pages."""
    r = gen(21)
    kc, vc = r(6, 16, 2, 64), r(6, 16, 2, 64)
    table = torch.tensor([[0, 1, 2], [0, 1, 3]], dtype=torch.int32).cuda()
    q, k, v = r(2, 4, 64), r(2, 2, 64), r(2, 2, 64)
    ref, tol, rk, _ = oa.step(npy(q), npy(k), npy(v), npy(kc), npy(vc), table.cpu().numpy(), [32, 40])
    check(gdr.attn_step(q, k, v, kc, vc, table, torch.tensor([32, 40], dtype=torch.int32).cuda()), ref, tol, "o")
    assert np.array_equal(npy(kc), rk)


def test_step_empty():
    kc = torch.zeros(2, 16, 1, 64, device="cuda")
    none = torch.zeros(0, 1, 64, device="cuda")
    table = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    assert gdr.attn_step(none, none, none, kc, kc.clone(), table, torch.zeros(0, dtype=torch.int32, device="cuda")).shape == (0, 1, 64)
    one = torch.ones(1, 1, 64, device="cuda")  # no pages at all: every row is full
    o = gdr.attn_step(one, one, one, kc[:0], kc[:0].clone(), torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                      torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert not o.any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("unaligned", [False, True])
def test_cache_write(dtype, unaligned):
    r = gen(22)
    lens, starts, size, Hk, D = [30, 0, 1, 77], [5, 3, -1, 0], 16, 3, 48
    table, pages = pages_for([40, 20, 20, 60], size, 2, 1)  # the last one's end has no room
    table[0, 1] = 500
    kv = r(1, sum(lens), 2 * Hk + 1, D, dtype=dtype)
    k, v = (kv[:, :, :Hk], kv[:, :, Hk:2 * Hk])
    if unaligned:
        flat = torch.empty(kv.numel() + 1, dtype=dtype, device="cuda")[1:].view(kv.shape).copy_(kv)
        k, v = (flat[:, :, :Hk], flat[:, :, Hk:2 * Hk])
    kc, vc = r(pages, size, Hk, D, dtype=dtype), r(pages, size, Hk, D, dtype=dtype)
    rk, rv = oa.write(npy(k)[0], npy(v)[0], npy(kc), npy(vc), table.cpu().numpy(), starts, lens)
    at = torch.tensor(starts, dtype=torch.int32).cuda()
    gdr.cache_write(k, v, kc, vc, table, starts=at, cu_seqlens=cu_of(lens))
    assert np.array_equal(npy(kc), rk) and np.array_equal(npy(vc), rv)
    k, v = r(4, 6, Hk, D, dtype=dtype), r(4, 6, Hk, D, dtype=dtype)  # B sequences of T tokens, from 0 on
    rk, rv = oa.write(npy(k).reshape(24, Hk, D), npy(v).reshape(24, Hk, D), npy(kc), npy(vc), table.cpu().numpy(), [0] * 4, [6] * 4)
    gdr.cache_write(k, v, kc, vc, table)
    assert np.array_equal(npy(kc), rk) and np.array_equal(npy(vc), rv)


# --------------------------------------------------------------------------------- used together
@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompt_then_tokens(dtype):
    """A prompt goes through rope, attention and the cache, then tokens follow one by one: every token's output is that of
    the whole sequence."""
    r = gen(31)
    lens, new, Hq, Hk, D, size = [70, 1, 129], 5, 4, 2, 64, 16
    whole = [n + new for n in lens]
    T = sum(whole)
    qkv = r(1, T, Hq + 2 * Hk, D, dtype=dtype)
    freqs, _ = gdr.rope_frequencies(D // 2)
    q, k = gdr.rope_forward(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], freqs, cu_seqlens=cu_of(whole))
    v = qkv[:, :, Hq + Hk:]
    ref, tol = oa.attention(*[npy(t)[0] for t in (q, k, v)], whole, whole, u=U[dtype])
    first = np.concatenate([[0], np.cumsum(whole)])
    prompt = torch.cat([torch.arange(first[n], first[n] + L) for n, L in enumerate(lens)]).cuda()
    table, pages = pages_for([n + new for n in lens], size, 4, 3)
    kc, vc = (torch.full((pages, size, Hk, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    part = qkv[:, prompt]
    pq, pk = gdr.rope_forward(part[:, :, :Hq], part[:, :, Hq:Hq + Hk], freqs, cu_seqlens=cu_of(lens))
    pv = part[:, :, Hq + Hk:]
    o, _ = gdr.attn_forward(pq, pk, pv, cu_seqlens=cu_of(lens))
    check(o[0], ref["o"][prompt.cpu()], tol["o"][prompt.cpu()], "prompt")
    gdr.cache_write(pk, pv, kc, vc, table, cu_seqlens=cu_of(lens))
    lengths = torch.tensor(lens, dtype=torch.int32).cuda()
    for t in range(new):
        at = torch.tensor([first[n] + L + t for n, L in enumerate(lens)]).cuda()
        row = qkv[0, at]
        q1, k1 = gdr.rope_forward(row[:, :Hq], row[:, Hq:Hq + Hk], freqs, positions=lengths)
        o = gdr.attn_step(q1, k1, row[:, Hq + Hk:], kc, vc, table, lengths)
        check(o, ref["o"][at.cpu()], tol["o"][at.cpu()], t)
        lengths += 1


def test_calls_on_streams_and_in_graphs():
    """On a stream of its own, and captured: replays on new inputs give what calls give."""
    r = gen(32)
    q, k, v, do = r(2, 200, 4, 64, dtype=BF), r(2, 200, 2, 64, dtype=BF), r(2, 200, 2, 64, dtype=BF), r(2, 200, 4, 64, dtype=BF)
    table, pages = pages_for([50, 90], 16, 2, 5)
    kc, vc = r(pages, 16, 2, 64, dtype=BF), r(pages, 16, 2, 64, dtype=BF)
    lengths = torch.tensor([50, 90], dtype=torch.int32).cuda()
    freqs, _ = gdr.rope_frequencies(64)

    def all_of(stream=None):
        q1, k1 = gdr.rope_forward(q, k, freqs, stream=stream)
        o, lse = gdr.attn_forward(q1, k1, v, stream=stream)
        s = gdr.attn_step(q[:, 0], k[:, 0], v[:, 0], kc, vc, table, lengths, stream=stream)
        return [q1, o, s, *gdr.attn_backward(q1, k1, v, o, lse, do, stream=stream)]

    want = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of()
    for t in (q, k, v, do):
        t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(9)).to(BF))
    graph.replay()
    got = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(got, all_of()))


def test_malformed_cu_seqlens_can_be_seen():
    q, k = torch.ones(1, 10, 2, 64, device="cuda"), torch.ones(1, 10, 1, 64, device="cuda")
    freqs, _ = gdr.rope_frequencies(64)
    table = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    for cu, well in (([0, 5, 10, 10], True), ([0, 5, 3, 10], False), ([1, 5, 5, 10], False), ([0, 5, 5, 9], False)):
        cu = torch.tensor(cu, dtype=torch.int32).cuda()
        want = (gdr.GDR_OK, 0) if well else (gdr.GDR_ERR_INVALID_ARG, 1)
        ws = gdr.attn_workspace(q, k, cu)
        o, lse = gdr.attn_forward(q, k, k, cu_seqlens=cu, workspace=ws)
        assert gdr.gdr_workspace_status(ws) == want
        ws = gdr.attn_workspace(q, k, cu, backward=True)
        gdr.attn_backward(q, k, k, q, torch.zeros(1, 2, 10, device="cuda"), q, cu_seqlens=cu, workspace=ws)
        assert gdr.gdr_workspace_status(ws) == want
        ws = gdr.rope_workspace(q, cu)
        gdr.rope_forward(q, k, freqs, cu_seqlens=cu, workspace=ws)
        assert gdr.gdr_workspace_status(ws) == want
        ws, kc = gdr.cache_write_workspace(k, cu), torch.zeros(1, 16, 1, 64, device="cuda")
        gdr.cache_write(k, k, kc, kc.clone(), table, cu_seqlens=cu, workspace=ws)
        assert gdr.gdr_workspace_status(ws) == want and bool(kc.any()) == well


@pytest.mark.parametrize("dtype", [F32, BF])
def test_tokens_beyond_32_bit_offsets(dtype):
    """Token strides that take the last tokens behind 2^31 elements: the same bits as contiguous inputs."""
    T, ld = 2200, 1 << 20
    r = gen(35)
    q, k, v, do = r(1, T, 4, 64, dtype=dtype), r(1, T, 2, 64, dtype=dtype), r(1, T, 2, 64, dtype=dtype), r(1, T, 4, 64, dtype=dtype)
    wide = torch.empty(T * ld, dtype=dtype, device="cuda").view(1, T, ld)
    at, views = 0, []
    for t in (q, k, v, do):
        n = t.shape[2] * 64
        views.append(wide[..., at:at + n].unflatten(-1, (t.shape[2], 64)))
        views[-1].copy_(t)
        at += n
    freqs, _ = gdr.rope_frequencies(64)
    table = torch.arange((T + 15) // 16, dtype=torch.int32).view(1, -1).cuda()

    def all_of(q, k, v, do):
        kc, vc = (torch.zeros(table.shape[1], 16, 2, 64, dtype=dtype, device="cuda") for _ in range(2))
        o, lse = gdr.attn_forward(q, k, v, window=500)
        gdr.cache_write(k, v, kc, vc, table)
        return [*gdr.rope_forward(q, k, freqs), o, lse, *gdr.attn_backward(q, k, v, o, lse, do, window=500), kc, vc]

    assert all(torch.equal(a, b) for a, b in zip(all_of(*views), all_of(q, k, v, do)))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_caches_beyond_32_bit_offsets(dtype):
    """Pages behind 2^31 elements of the pool: the same bits as with a small one."""
    size, Hk, D, lens = 16, 2, 128, [70, 33]
    r = gen(36)
    few, first = 12, (1 << 31) // (size * Hk * D) + 3
    k, v = r(2, 80, Hk, D, dtype=dtype), r(2, 80, Hk, D, dtype=dtype)
    q, k1, v1 = r(2, 4, D, dtype=dtype), r(2, Hk, D, dtype=dtype), r(2, Hk, D, dtype=dtype)
    table = torch.arange(few, dtype=torch.int32).view(2, -1).flip(1).contiguous().cuda()
    lengths = torch.tensor(lens, dtype=torch.int32).cuda()

    def all_of(pages, offset):
        kc, vc = (torch.empty(pages, size, Hk, D, dtype=dtype, device="cuda") for _ in range(2))
        kc[offset:].zero_(), vc[offset:].zero_()
        gdr.cache_write(k, v, kc, vc, table + offset)
        return gdr.attn_step(q, k1, v1, kc, vc, table + offset, lengths), kc[offset:].clone(), vc[offset:].clone()

    assert all(torch.equal(a, b) for a, b in zip(all_of(first + few, first), all_of(few, 0)))


def test_a_call_without_queries_clears_the_status():
    q = torch.ones(1, 10, 2, 64, device="cuda")
    cu = torch.tensor([0, 5, 3, 10], dtype=torch.int32).cuda()
    lse = torch.zeros(1, 2, 10, device="cuda")
    for backward in (False, True):
        ws = gdr.attn_workspace(q, q, cu, backward=backward)
        if backward:
            gdr.attn_backward(q, q, q, q, lse, q, cu_seqlens=cu, workspace=ws)
        else:
            gdr.attn_forward(q, q, q, cu_seqlens=cu, workspace=ws)
        assert gdr.gdr_workspace_status(ws) == (gdr.GDR_ERR_INVALID_ARG, 1)
        none = q[:, :0]
        if backward:
            gdr.attn_backward(none, q, q, none, lse[..., :0].contiguous(), none, workspace=ws)
        else:
            gdr.attn_forward(none, q, q, workspace=ws)
        assert gdr.gdr_workspace_status(ws) == (gdr.GDR_OK, 0)


def test_a_row_with_a_page_outside_the_pool_keeps_its_own_page():
    """The row's result is zero; its token goes to its page where that is in the pool, and nowhere else."""
    kc = torch.zeros(4, 16, 1, 64, device="cuda")
    vc = kc.clone()
    one = torch.ones(2, 1, 64, device="cuda")
    table = torch.tensor([[9, 2], [1, -1]], dtype=torch.int32).cuda()
    o = gdr.attn_step(one, one, one, kc, vc, table, torch.tensor([20, 20], dtype=torch.int32).cuda())
    assert not o.any()
    want = torch.zeros_like(kc)
    want[2, 4] = 1
    assert torch.equal(kc, want) and torch.equal(vc, want)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,heads,packed", [(40, 2, True), (700, 8, False), (1500, 2, True)])
def test_calls_in_a_row_wait_for_each_other(dtype, T, heads, packed):
    """Every call reads what the one before it wrote, its launches begin while that one ends, and memory goes round: the same bits as with
    a synchronisation behind each call."""
    r = gen(34)
    q0, k0, v0 = (r(1, T, heads, 64, dtype=dtype) for _ in range(3))
    freqs, _ = gdr.rope_frequencies(64)
    cu = torch.tensor([0, T // 3, T], dtype=torch.int32).cuda() if packed else None
    pages = (T + 15) // 16 + 2
    table = torch.arange(2 * pages, dtype=torch.int32).view(2, pages).cuda()[:2 if packed else 1].contiguous()

    def chain(after):
        q, k, v, out = q0, k0, v0, []
        kc, vc = torch.zeros(2 * pages, 16, heads, 64, dtype=dtype, device="cuda"), torch.zeros(2 * pages, 16, heads, 64, dtype=dtype, device="cuda")
        lengths = torch.tensor([T // 3, T - T // 3] if packed else [T], dtype=torch.int32).cuda()
        for _ in range(6):
            q, k = after(gdr.rope_forward(q, k, freqs, cu_seqlens=cu))
            o, lse = after(gdr.attn_forward(q, k, v, cu_seqlens=cu))
            dq, dk, dv = after(gdr.attn_backward(q, k, v, o, lse, o, cu_seqlens=cu))
            after(gdr.cache_write(k, v, kc, vc, table, cu_seqlens=cu))
            x = o[0, :lengths.numel()]
            for _ in range(3):
                x = after(gdr.attn_step(x, k[0, :lengths.numel()], x, kc, vc, table, lengths))
            out += [o, lse, dq, dk, dv, x, kc.clone(), vc.clone()]
            q, k, v = q + dq, k + dk, o
        return out

    def synced(x):
        torch.cuda.synchronize()
        return x

    want = chain(synced)
    for _ in range(3):
        got = chain(lambda x: x)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_training_step_in_a_graph():
    """Forward and backward through autograd, captured: replays on new inputs give what eager steps give."""
    r = gen(33)
    q, k, v, do = r(1, 300, 4, 64, dtype=BF), r(1, 300, 2, 64, dtype=BF), r(1, 300, 2, 64, dtype=BF), r(1, 300, 4, 64, dtype=BF)
    freqs, _ = gdr.rope_frequencies(64)
    cu = torch.tensor([0, 170, 300], dtype=torch.int32).cuda()

    def grads(q, k, v):
        q, k, v = (t.detach().requires_grad_() for t in (q, k, v))
        q1, k1 = gdr.rope(q, k, freqs, cu_seqlens=cu)
        o = gdr.attention(q1, k1, v, cu_seqlens=cu, window=100)
        return [o.detach(), *torch.autograd.grad(o, (q, k, v), do)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(q, k, v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = grads(q, k, v)
    for t in (q, k, v, do):
        t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(7)).to(BF))
    graph.replay()
    got = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(got, grads(q, k, v)))


def test_caches_have_versions():
    kc, vc = torch.ones(2, 16, 1, 64, device="cuda"), torch.ones(2, 16, 1, 64, device="cuda")
    was = kc._version, vc._version
    one = torch.ones(1, 1, 64, device="cuda")
    gdr.attn_step(one, one, one, kc, vc, torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert kc._version > was[0] and vc._version > was[1]
    was = kc._version, vc._version
    gdr.cache_write(one[None], one[None], kc, vc, torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
    assert kc._version > was[0] and vc._version > was[1]
