"""Pins of ``oracle.cache_ops`` to facts other than itself: the rotate-half rope, torch's
scaled-dot-product attention over the concatenated tokens, closed forms of the scalings at
their ends, and hand-worked evictions."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops
from oracle.rope import rope_rotate_half

rng = np.random.default_rng(5)


def test_plain_half_rotary_is_the_rotate_half_rope():
    x, pos = rng.standard_normal((3, 2, 16)), [0, 7, 100000]
    got = cache_ops.rotary(x, pos, cache_ops.rotary_frequencies(16, base=10000.0))
    for t, p in enumerate(pos):
        for h in range(2):
            np.testing.assert_allclose(got[t, h], rope_rotate_half(x[t, h], p, 10000.0), rtol=0, atol=1e-9)


def test_layouts_are_a_permutation_and_the_rest_is_copied():
    x, freq = rng.standard_normal((2, 1, 12)), cache_ops.rotary_frequencies(8)
    perm = [0, 2, 4, 6, 1, 3, 5, 7]      # element of the interleaved head at each half-layout place
    il = cache_ops.rotary(x, [3, 9], freq, "interleaved", 1.5)
    half = cache_ops.rotary(x[..., perm + [8, 9, 10, 11]], [3, 9], freq, "half", 1.5)
    np.testing.assert_allclose(il[..., perm], half[..., :8], rtol=1e-14)
    np.testing.assert_array_equal(il[..., 8:], x[..., 8:])
    # norms of pairs grow by the amplitude, position 0 only scales
    np.testing.assert_allclose((il[..., :8]**2).sum(), 2.25 * (x[..., :8]**2).sum())
    np.testing.assert_allclose(cache_ops.rotary(x, [0, 0], freq, "half", 2.0)[..., :8], 2 * x[..., :8])


def test_scalings_at_their_ends():
    plain = cache_ops.rotary_frequencies(64)
    np.testing.assert_allclose(plain, [10000.0**(-i / 32) for i in range(32)])
    np.testing.assert_allclose(cache_ops.rotary_frequencies(64, "linear", factor=4.0), plain / 4)
    ntk = cache_ops.rotary_frequencies(64, "ntk", factor=4.0)
    assert ntk[0] == 1.0                                  # the fastest pair keeps its speed
    np.testing.assert_allclose(ntk[-1], plain[-1] / 4)    # the slowest is stretched by the factor
    for scaling, kw in (("ramp", dict(low=1.0, high=32.0)), ("bands", dict(low=1.0, high=4.0))):
        f = cache_ops.rotary_frequencies(64, scaling, factor=4.0, original_len=4096, **kw)
        assert f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 4)
        assert (np.diff(f) < 0).all() and (f <= plain).all() and (f >= plain / 4 - 1e-15).all()
    # bands: a pair that turns (low + high) / 2 times takes the mean of the two
    n = 2 * math.pi * 2.5 / plain[7]
    f = cache_ops.rotary_frequencies(64, "bands", factor=4.0, original_len=n, low=1.0, high=4.0)
    np.testing.assert_allclose(f[7], plain[7] * (1 + 0.25) / 2)


@pytest.mark.parametrize("bias", [False, True])
def test_shared_attention_is_attention_over_both(bias):
    Hq, Hkv, d, lens, plens, rows = 4, 2, 8, [5, 0, 20], [17, 3], [0, 1, -1]
    kc, vc = rng.standard_normal((9, Hkv, 16, d)), rng.standard_normal((9, Hkv, 16, d))
    tab, ptab = np.array([[4, -1], [-1, -1], [7, 2]]), np.array([[0, 8], [5, -1]])
    q = rng.standard_normal((3, Hq, d))
    add = rng.standard_normal((3, 20)) if bias else None
    if bias:
        add[0, 2] = -np.inf

    def flat(cache, t, n):
        return np.concatenate([cache[b] for b in t if b >= 0] + [np.zeros((Hkv, 0, d))], 1)[:, :n]
    got = cache_ops.shared_attention(q, kc, vc, tab, lens, 0.3, ptab, plens, rows, add)
    for b in range(3):
        m = plens[rows[b]] if rows[b] >= 0 else 0
        kk, vv = (np.concatenate([flat(c, ptab[rows[b]], m) if m else np.zeros((Hkv, 0, d)),
                                  flat(c, tab[b], lens[b])], 1).repeat(2, 0) for c in (kc, vc))
        mask = np.zeros(m + lens[b])
        if bias:
            mask[m:] = add[b, :lens[b]]
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[b])[:, None], torch.from_numpy(kk), torch.from_numpy(vv),
            attn_mask=torch.from_numpy(mask)[None], scale=0.3)[:, 0]
        np.testing.assert_allclose(got[b][0], want.numpy(), atol=1e-12)
        s = np.einsum("hd,htd->ht", q[b], kk) * 0.3 + mask
        np.testing.assert_allclose(got[b][1], np.log(np.exp(s).sum(1)))
        w = np.exp(s - got[b][1][:, None])
        np.testing.assert_allclose(got[b][2], w.reshape(Hkv, 2, -1).sum(1)[:, m:], atol=1e-13)


def test_a_row_without_tokens_and_one_masked_whole():
    kc = np.ones((1, 1, 16, 4))
    got = cache_ops.shared_attention(np.ones((2, 1, 4)), kc, kc, [[-1], [0]], [0, 3], 1.0,
                                     bias=np.full((2, 3), -np.inf))
    for out, lse, w, _, _ in got:
        assert (out == 0).all() and (lse == -np.inf).all() and (w == 0).all()


@pytest.mark.parametrize("mass,keep,sink,recent,want", [
    ([5, 1, 4, 2, 3], 3, 0, 0, [0, 2, 4]), ([5, 1, 4, 2, 3], 3, 0, 2, [0, 3, 4]),
    ([1, 9, 9, 9, 1], 2, 1, 0, [0, 1]), ([2, 2, 2, 2], 2, 0, 0, [0, 1]),
    ([0.0, -0.0, 1.0], 2, 0, 0, [0, 2]), ([1, float("nan"), 7], 1, 0, 0, [1]),
    ([1, 2, 3], 5, 4, 4, [0, 1, 2]), ([1, 2, 3, 4], 2, 4, 4, [2, 3]), ([1, 2, 3, 4], 3, 2, 1, [0, 1, 3]),
    ([1, 2], 0, 1, 1, [])])
def test_kept_tokens_worked_by_hand(mass, keep, sink, recent, want):
    assert cache_ops.kept_tokens(np.array(mass, float), keep, sink, recent).tolist() == want


def test_eviction_moves_rows_of_both_caches_and_the_weights():
    k = np.arange(3 * 1 * 16.0).reshape(3, 1, 16, 1)
    m = np.zeros((3, 1, 16))
    tab = [[2, 0]]                       # token t: block 2 row t, then block 0 row t - 16
    m[2, 0, 3], m[0, 0, 1] = 4.0, 9.0    # tokens 3 and 17
    (nk, nv, nm), kept = cache_ops.evict((k, -k, m), tab, [18], [2])
    assert kept[0][0].tolist() == [3, 17]
    assert nk[2, 0, :3, 0].tolist() == [32 + 3, 1, 32 + 2] and (nv == -nk).all()
    assert nm[2, 0, :3].tolist() == [4.0, 9.0, 0.0] and nm[0, 0, 1] == 9.0
