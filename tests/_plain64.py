"""Plain 64-bit forms of the head transform and of attention with modified scores (not
collected as tests): numpy, one head vector and one query row at a time."""
import numpy as np


def transform(x, weight, positions, inv_freq, *, eps, offset, interleaved):
    """x [n, heads, d] float64; weight [d] or None; inv_freq float32 [rot / 2]."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)
    half = len(inv_freq)
    out = y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = (np.asarray(positions, np.float64) * float(inv_freq[i]))[:, None]
        out[:, :, a] = y[:, :, a] * np.cos(t) - y[:, :, b] * np.sin(t)
        out[:, :, b] = y[:, :, b] * np.cos(t) + y[:, :, a] * np.sin(t)
    return out


def visible(c, i, total, where_q, where_k, tree_bits, window):
    """Which of the `total` keys row i of a sequence with c committed tokens sees."""
    t = np.arange(total)
    j = t - c
    see = t < c
    if tree_bits is None:
        see = see | (j <= i)
    else:
        see = see | np.array([x >= 0 and bool((int(tree_bits) >> int(x)) & 1) for x in j], bool)
    return see & (where_q - where_k < window) if window else see


def attention(k, v, q, c, *, scale, softcap=0.0, slopes=None, window=0, positions=None, tree_mask=None):
    """One sequence: k, v [total, hkv, d] (committed rows, then the new ones), q [n, hq, d]."""
    total, hkv, d = k.shape
    n, hq, _ = q.shape
    where = np.arange(total)
    if positions is not None:
        where[c:] = positions
    out = np.zeros((n, hq, d))
    for i in range(n):
        at = c + i if positions is None else int(positions[i])
        see = visible(c, i, total, at, where, None if tree_mask is None else tree_mask[i], window)
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // (hq // hkv)], v[see, h // (hq // hkv)]
            s = kk @ q[i, h] * scale
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s - float(slopes[h]) * (at - where[see])
            p = np.exp(s - s.max())
            out[i, h] = (p / p.sum()) @ vv
    return out
