"""Rotary layouts and scalings, attention over a shared prefix and own tokens, and
eviction by accumulated weight, in float64.

Test infrastructure only (see the package docstring).
"""
import math

import numpy as np

from .attention import gather_sequence


# --------------------------------------------------------------------------- rotary
def rotary_frequencies(rot_dim, scaling="plain", base=10000.0, factor=1.0, low=1.0, high=32.0,
                       original_len=0):
    """Radians per position of pairs ``i < rot_dim/2``, one pair at a time from the
    definitions."""
    out = []
    for i in range(rot_dim // 2):
        b = base * factor ** (rot_dim / (rot_dim - 2.0)) if scaling == "ntk" else base
        g = b ** (-2.0 * i / rot_dim)
        turns = original_len * g / (2 * math.pi)
        if scaling in ("plain", "ntk"):
            f = g
        elif scaling == "linear":
            f = g / factor
        elif scaling == "bands":
            # pairs that turn often keep their speed, slow ones are stretched
            if turns >= high:
                f = g
            elif turns <= low:
                f = g / factor
            else:
                s = (turns - low) / (high - low)
                f = s * g + (1 - s) * g / factor
        elif scaling == "ramp":
            def pair(t):   # the (real-valued) pair that makes t turns over original_len
                return rot_dim / 2 * math.log(original_len / (2 * math.pi * t)) / math.log(base)
            lo, hi = max(0, math.floor(pair(high))), min(rot_dim - 1, math.ceil(pair(low)))
            w = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = (1 - w) * g + w * g / factor
        else:
            raise ValueError(scaling)
        out.append(f)
    return np.array(out)


def rotary(x, positions, freq, layout="half", amplitude=1.0):
    """``x [T,H,d]`` rotated at ``positions [T]``: pair i as the complex number
    x1 + i x2 times amplitude * exp(i p f_i); elements behind the pairs unchanged."""
    x = np.array(x, np.float64)
    n = len(freq)
    first = np.arange(n) if layout == "half" else 2 * np.arange(n)
    second = first + n if layout == "half" else first + 1
    turn = amplitude * np.exp(1j * np.asarray(positions, np.float64)[:, None, None] * freq)
    z = (x[..., first] + 1j * x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x


# --------------------------------------------------------------------------- attention
def shared_attention(q, k_cache, v_cache, tables, lens, scale, prefix_tables=(), prefix_lens=(),
                     row_prefix=None, bias=None):
    """Per row: output ``[Hq,d]``, natural log-sum-exp ``[Hq]``, the own tokens' weights
    ``[Hkv, lens[b]]`` summed over the group, and the error scales ``(sum p|v| [Hq,d],
    max score error per unit of rounding [Hq])``."""
    q = np.asarray(q, np.float64)
    B, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    rows = []
    for b in range(B):
        n = int(lens[b])
        p = -1 if row_prefix is None else int(row_prefix[b])
        out, absv = np.zeros((Hq, d)), np.zeros((Hq, d))
        lse, weight = np.full(Hq, -np.inf), np.zeros((Hkv, n))
        swing = np.zeros(Hq)
        for h in range(Hq):
            g = h // G
            k = gather_sequence(k_cache, tables[b], n, g)
            v = gather_sequence(v_cache, tables[b], n, g)
            add = np.zeros(n) if bias is None else np.asarray(bias[b][:n], np.float64)
            if p >= 0:
                m = int(prefix_lens[p])
                k = np.concatenate([gather_sequence(k_cache, prefix_tables[p], m, g), k])
                v = np.concatenate([gather_sequence(v_cache, prefix_tables[p], m, g), v])
                add = np.concatenate([np.zeros(m), add])
            if not len(k):
                continue
            s = (k @ q[b, h]) * scale + add
            top = s.max()
            if top == -np.inf:
                continue
            e = np.exp(s - top)
            w = e / e.sum()
            out[h], absv[h] = w @ v, w @ np.abs(v)
            lse[h] = top + np.log(e.sum())
            weight[g] += w[len(w) - n:]
            swing[h] = (np.abs(k) @ np.abs(q[b, h])).max() * abs(scale)
        rows.append((out, lse, weight, absv, swing))
    return rows


# --------------------------------------------------------------------------- eviction
def kept_tokens(mass, keep, sink=0, recent=0):
    """Ascending indices kept of a row whose tokens have accumulated ``mass [L]``."""
    L = len(mass)
    if L <= keep:
        return np.arange(L)
    r = min(recent, keep)
    s = min(sink, keep - r)
    between = range(s, L - r)
    # larger weight first, NaN above everything, then the lower index
    def rank(t):
        x = float(mass[t])
        return (0, 0.0, t) if math.isnan(x) else (1, -x, t)
    best = sorted(between, key=rank)[:keep - r - s]
    return np.array(sorted(list(range(s)) + best + list(range(L - r, L))), np.int64)


def evict(caches, tables, lens, keeps, sink=0, recent=0):
    """``caches = (k, v, mass)`` as ``[blocks,Hkv,16,...]``; returns copies after the
    compaction and, per row and KV head, the kept indices."""
    new = [np.array(c, copy=True) for c in caches]
    kept = []
    for b, (L, K) in enumerate(zip(lens, keeps)):
        t = np.arange(L)
        blk, row = np.asarray(tables[b])[t // 16], t % 16
        heads = []
        for g in range(caches[0].shape[1]):
            src = kept_tokens(caches[2][blk, g, row], int(K), sink, recent)
            for c, o in zip(new, caches):
                c[blk[:len(src)], g, row[:len(src)]] = o[blk[src], g, row[src]]
            heads.append(src)
        kept.append(heads)
    return new, kept
