"""Incremental scoring over a paged cache, step by step (TEST INFRASTRUCTURE
ONLY): slot maps, the norm and rotation of queries and keys, and attention
over the keys a token sees.

"Learning to summarize from human feedback" (summary page, method section)
scores a text with a causal decoder; with its keys and values kept, a longer
text is scored from its new tokens alone.  Everything here is fp64 and one
sequence or request at a time.
"""
import numpy as np


def kv_slots(len_before, n_new, page, free, used, table, T):
    """The step's packing, request by request.  Returns (offsets, positions,
    slots, len_after, used_after, unserved, table after)."""
    n, width = table.shape
    table = table.copy()
    offsets, after = [0], []
    positions, slots = np.zeros(T, dtype=np.int64), np.full(T, -1, dtype=np.int64)
    open_, served = True, 0
    for i in range(n):
        b, m = int(len_before[i]), int(n_new[i])
        t = offsets[-1]
        if open_:
            have, need = -(-b // page), -(-(b + m) // page)
            open_ = (b >= 0 and m >= 0 and need <= width and t + m <= T
                     and 0 <= used and used + need - have <= len(free))
        if not open_:
            offsets.append(t)
            after.append(b)
            continue
        served += 1
        for k in range(have, need):
            table[i, k] = free[used]
            used += 1
        for j in range(m):
            pos = b + j
            positions[t + j] = pos
            slots[t + j] = int(table[i, pos // page]) * page + pos % page
        offsets.append(t + m)
        after.append(b + m)
    return np.array(offsets), positions, slots, np.array(after), used, n - served, table


def rope_freqs(rot, base, scaling="plain", factor=1.0, trained=0.0, fast=32.0, slow=1.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        turns = trained * f / (2 * np.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0, 1)
        f = keep * f + (1 - keep) * f / factor
    return f


def norm_rope(x, gain, eps, positions, freqs, layout, mscale=1.0):
    """x [T][heads][d] -> normed (gain not None) and rotated heads, and per
    element the sum of the magnitudes that the last addition adds up."""
    x = np.asarray(x, dtype=np.float64)
    if gain is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(gain, dtype=np.float64)
    y, mag = x.copy(), np.abs(x)
    if freqs is not None and len(freqs):
        h = len(freqs)
        a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freqs)[None]
        c, s = mscale * np.cos(a)[:, None], mscale * np.sin(a)[:, None]
        i0 = np.arange(h) if layout == 0 else 2 * np.arange(h)
        i1 = i0 + (h if layout == 0 else 1)
        p, q = x[..., i0], x[..., i1]
        y[..., i0], y[..., i1] = p * c - q * s, q * c + p * s
        mag[..., i0] = mag[..., i1] = mscale * (np.abs(p) + np.abs(q))
    return y, mag


def seen_keys(pos, window, sinks):
    """The keys 0..pos that the token at position pos of its sequence sees."""
    j = np.arange(pos + 1)
    return j if window <= 0 else j[(j > pos - window) | (j < sinks)]


def attend(q, k, v, seen):
    """One token's heads q [hq][d] over k, v [len][hkv][d]: the output, and per
    element sum p|v| and per head the largest sum |q k| / sqrt(d) (what the
    rounding of P and of the scores scale with).  Nothing seen gives zeros."""
    hq, d = q.shape
    out, mag, top = np.zeros((hq, d)), np.zeros((hq, d)), np.zeros(hq)
    if len(seen) == 0:
        return out, mag, top
    hkv = k.shape[1]
    for h in range(hq):
        kk, vv = k[seen, h // (hq // hkv)], v[seen, h // (hq // hkv)]
        s = kk @ q[h] / np.sqrt(d)
        p = np.exp(s - s.max())
        p /= p.sum()
        out[h], mag[h] = p @ vv, p @ np.abs(vv)
        top[h] = (np.abs(kk) @ np.abs(q[h])).max() / np.sqrt(d)
    return out, mag, top


def attend_window(q, k, v, offsets, window, sinks):
    """Packed q [T][hq][d], k, v [T][hkv][d] -> (out, mag, top) for every row."""
    out, mag, top = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    for a, b in zip(offsets[:-1], offsets[1:]):
        for t in range(a, b):
            out[t], mag[t], top[t] = attend(q[t], k[a:b], v[a:b], seen_keys(t - a, window, sinks))
    return out, mag, top
