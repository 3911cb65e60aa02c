"""Pins of the fp64 references of the attention mixer: gradients against finite differences, closed forms, the step
against whole sequences."""
import numpy as np
import pytest

from oracle import attn as oa


@pytest.mark.parametrize("q_lens,k_lens,causal,window", [([5], [5], True, 0), ([3, 4], [6, 2], True, 0), ([4], [7], False, 0),
                                                         ([6], [6], True, 3), ([3], [5], False, 2)])
def test_gradients_are_the_differences(q_lens, k_lens, causal, window):
    r = np.random.default_rng(1)
    q, k, v = r.normal(size=(sum(q_lens), 4, 3)), r.normal(size=(sum(k_lens), 2, 3)), r.normal(size=(sum(k_lens), 2, 3))
    do = r.normal(size=q.shape)
    got, _ = oa.attention(q, k, v, q_lens, k_lens, causal, window, 0.7, do)

    def loss(*t):
        return (oa.attention(*t, q_lens, k_lens, causal, window, 0.7)[0]["o"] * do).sum()

    for n, name in enumerate(("dq", "dk", "dv")):
        ts = [q, k, v]
        diff = np.zeros_like(ts[n])
        for i in np.ndindex(diff.shape):
            hi, lo = [t.copy() for t in ts], [t.copy() for t in ts]
            hi[n][i] += 1e-5
            lo[n][i] -= 1e-5
            diff[i] = (loss(*hi) - loss(*lo)) / 2e-5
        assert np.abs(diff - got[name]).max() <= 1e-8 * max(1.0, np.abs(diff).max())


def test_closed_forms():
    r = np.random.default_rng(2)
    v = r.normal(size=(6, 1, 4))
    zero = np.zeros_like(v)
    got, _ = oa.attention(zero, zero, v, [6], [6], True)  # equal scores: running means
    assert np.allclose(got["o"][:, 0], np.cumsum(v[:, 0], 0) / np.arange(1, 7)[:, None], atol=1e-14)
    assert np.allclose(got["lse"][0], np.log(np.arange(1, 7)), atol=1e-14)
    got, _ = oa.attention(v, v, v, [6], [2], True)  # four queries stand before the first key
    assert not got["o"][:4].any() and np.isneginf(got["lse"][0, :4]).all() and np.allclose(got["o"][4], v[0])


def test_a_rotation_is_relative():
    """Products of rotated vectors depend on the difference of their positions; the inverse undoes it."""
    r = np.random.default_rng(3)
    x, y, f = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8)), 10000.0 ** -(np.arange(3) / 3)
    for nb in (False, True):
        def dot(a, b):
            return (oa.rope(x, f, np.array([a]), nb) * oa.rope(y, f, np.array([b]), nb)).sum()
        assert abs(dot(5, 2) - dot(105, 102)) < 1e-12
        back = oa.rope(oa.rope(x, f, np.array([77]), nb, 2.0), f, np.array([77]), nb, 0.5, inverse=True)
        assert np.allclose(back, x, atol=1e-14)


def test_steps_are_the_last_rows():
    r = np.random.default_rng(4)
    lens, size = [5, 9], 4
    q, k, v = r.normal(size=(14, 4, 3)), r.normal(size=(14, 2, 3)), r.normal(size=(14, 2, 3))
    whole, _ = oa.attention(q, k, v, lens, lens, True, 6)
    kc = vc = np.zeros((7, size, 2, 3))
    table = np.array([[3, 0, -1], [6, 2, 5]])
    first = np.r_[0:4, 5:13]
    kc, vc = oa.write(k[first], v[first], kc, vc, table, [0, 0], [4, 8])
    o, _, kc, vc = oa.step(q[[4, 13]], k[[4, 13]], v[[4, 13]], kc, vc, table, [4, 8], 6)
    assert np.allclose(o, whole["o"][[4, 13]], atol=1e-13)
    assert np.array_equal(kc[5, 0], k[13]) and np.array_equal(vc[0, 0], v[4])
