"""Rotary positions, a paged key/value cache and attention over it (test
infrastructure), everything in float64 from the formulas.

Readings:
 28. angles pos * inv_freq with inv_freq as the fp32 it is stored as, pairs
     (i, i + rot/2) or (2i, 2i + 1) of a head's first rot values; the scale
     multiplies the rotated values only; a cached FP8 key or value is the
     activation quantizer over its head, of the unrounded rotated key;
 29. a token sees the shared prefix's keys, then its sequence's own, up to
     its own position and from `window` before it on; a page id outside the
     cache hides its keys; no key: 0.
"""

import numpy as np

from .formats import e4m3_decode


def inv_freq(rot, base, scaling=0, factor=1.0, low=1.0, high=32.0, orig_len=0.0):
    theta = float(base) ** (-2.0 * np.arange(rot // 2) / rot) if rot else np.zeros(0)
    if scaling == 1:
        theta = theta / factor
    elif scaling == 2:
        g = np.clip((orig_len * theta / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        theta = theta * g + theta / factor * (1.0 - g)
    return theta.astype(np.float32)


def rotate(x, positions, freq, interleaved=False, mscale=1.0):
    """x (T, H, D) float64."""
    y = np.array(x, dtype=np.float64)
    half = len(freq)
    t = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(freq, dtype=np.float64)
    c, s = np.cos(t) * mscale, np.sin(t) * mscale
    ia = 2 * np.arange(half) if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def cache_values(codes, scales, fmt):
    """float64 values of a cache in the pages' own shape; fmt 0, 1 (E4M3 bytes
    with fp32 or E8M0 scales) or 2 (values already)."""
    if fmt == 2:
        return np.asarray(codes, dtype=np.float64)
    s = np.asarray(scales, dtype=np.float64)
    s = s if fmt == 0 else 2.0 ** (s - 127.0)
    return e4m3_decode(codes).astype(np.float64) * s[..., None]


def _keys(pages, table, count, h):
    """(values (count, D), there (count,)) of head h."""
    P, _, ps, D = pages.shape
    x, ok = np.zeros((count, D)), np.zeros(count, bool)
    for j0 in range(0, count, ps):
        m, p = min(ps, count - j0), int(table[j0 // ps])
        if 0 <= p < P:
            x[j0:j0 + m], ok[j0:j0 + m] = pages[p, h, :m], True
    return x, ok


def attention(q, kpages, vpages, kv_len, table, scale, q_start=None, prefix_table=None, prefix_len=0,
              window=0):
    """(y, spread, reach, keys): y (T, Hq, D) with NaN rows for tokens of no
    sequence; for error bounds, per element, spread = sum p |v| / sum p; per
    row, reach = max over seen keys of scale sum |q k| and the number of keys."""
    T, Hq, D = q.shape
    P, Hkv, ps, _ = kpages.shape
    G, B = Hq // Hkv, len(kv_len)
    y, spread = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D))
    reach, seen = np.zeros((T, Hq)), np.zeros((T, Hq))
    start = np.arange(B + 1) if q_start is None else np.asarray(q_start)
    for b in range(B):
        n = start[b + 1] - start[b]
        length = int(min(max(kv_len[b], 0), table.shape[1] * ps))
        if n == 0:
            continue
        pos = prefix_len + length - n + np.arange(n)
        at = np.arange(prefix_len + length)
        for h in range(Hkv):
            k, ok = _keys(kpages, table[b], length, h)
            v, _ = _keys(vpages, table[b], length, h)
            if prefix_len:
                pk, pok = _keys(kpages, prefix_table, prefix_len, h)
                pv, _ = _keys(vpages, prefix_table, prefix_len, h)
                k, v, ok = np.concatenate([pk, k]), np.concatenate([pv, v]), np.concatenate([pok, ok])
            for i in range(n):
                see = ok & (at <= pos[i])
                if window:
                    see &= at > pos[i] - window
                t = start[b] + i
                for r in range(h * G, (h + 1) * G):
                    if not see.any():
                        y[t, r] = 0.0
                        continue
                    s = k[see] @ q[t, r] * scale
                    p = np.exp(s - s.max()) if np.isfinite(s.max()) else np.exp(s)
                    y[t, r] = p @ v[see] / p.sum()
                    spread[t, r] = p @ np.abs(v[see]) / p.sum()
                    reach[t, r] = (np.abs(k[see]) @ np.abs(q[t, r])).max() * scale
                    seen[t, r] = see.sum()
    return y, spread, reach, seen
