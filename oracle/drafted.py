"""Attention of drafted tokens, accepted paths and rotary positions with several axes, in
float64.

Test infrastructure only (see the package docstring).
"""
import numpy as np

from .attention import gather_sequence


def tree_visible(mask, first, n, base):
    """Boolean [n, base + n]: what the n nodes of a row see, from their mask words (None: a
    node sees the nodes up to itself)."""
    sees = np.ones((n, base + n), bool)
    for i in range(n):
        for j in range(n):
            sees[i, base + j] = j <= i if mask is None else int(mask[first + i, j // 32]) >> j % 32 & 1
    return sees


def tree_attention(q, k_cache, v_cache, tables, lens, starts, scale, mask=None):
    """``(out [T,Hq,d], lse [T,Hq], sum p|v| [T,Hq,d], swing [T,Hq])``: the output, the natural
    log-sum-exp and the error scales (swing: scale * the largest sum |q||k|) of every query
    row; rows of no batch row are NaN."""
    T, Hq, d = q.shape
    G = Hq // k_cache.shape[1]
    out, absv = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse, swing = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)
    for b in range(len(lens)):
        a, n = int(starts[b]), int(starts[b + 1]) - int(starts[b])
        if n == 0:
            continue
        sees = tree_visible(mask, a, n, int(lens[b]) - n)
        for h in range(Hq):
            k = gather_sequence(k_cache, tables[b], int(lens[b]), h // G)
            v = gather_sequence(v_cache, tables[b], int(lens[b]), h // G)
            for i in range(n):
                ks, vs, x = k[sees[i]], v[sees[i]], q[a + i, h]
                if not len(ks):
                    out[a + i, h], absv[a + i, h] = 0.0, 0.0
                    lse[a + i, h], swing[a + i, h] = -np.inf, 0.0
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    s = ks @ x * scale
                    m = s.max()
                    w = np.exp(s - m)
                    total = w.sum()
                    out[a + i, h] = w @ vs / total
                    absv[a + i, h] = w @ np.abs(vs) / total
                    lse[a + i, h] = m + np.log(total)
                    swing[a + i, h] = abs(scale) * (np.abs(ks) @ np.abs(x)).max()
    return out, lse, absv, swing


def accept(cache, tables, lens, starts, path, counts):
    """The cache ``[blocks,Hkv,16,d]`` after every row's accepted tokens have moved."""
    cache = np.array(cache)
    for b in range(len(lens)):
        base = int(lens[b]) - (int(starts[b + 1]) - int(starts[b]))
        rows = [cache[tables[b][(base + i) // 16], :, (base + i) % 16].copy() for i in path[b][:counts[b]]]
        for j, x in enumerate(rows):
            cache[tables[b][(base + j) // 16], :, (base + j) % 16] = x
    return cache


def axes_of(sections, order="blocked"):
    """Axis of every pair, and its number among its axis' pairs."""
    left, axis = list(sections), []
    while any(left):
        for a in range(len(left)):
            take = left[a] if order == "blocked" else min(left[a], 1)
            axis += [a] * take
            left[a] -= take
    return axis, [axis[:i].count(a) for i, a in enumerate(axis)]


def rotary_axes(x, positions, freq, axis, layout="half", amplitude=1.0):
    """``x [T,H,d]`` rotated at ``positions [axes,T]``: pair i as the complex number x1 + i x2
    times amplitude * exp(i p f_i), p the token's position on the pair's axis."""
    x = np.array(x, np.float64)
    n = len(freq)
    first = np.arange(n) if layout == "half" else 2 * np.arange(n)
    second = first + n if layout == "half" else first + 1
    p = np.asarray(positions, np.float64)[np.asarray(axis)].T      # [T, pairs]
    z = (x[..., first] + 1j * x[..., second]) * (amplitude * np.exp(1j * p * freq))[:, None]
    x[..., first], x[..., second] = z.real, z.imag
    return x
