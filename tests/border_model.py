"""Definitions in numpy, 64 bits, of the operators at the borders of the decode path: rotary positions,
attention to an encoder's states, log probabilities. They share no code with the library."""
import math

import numpy as np

D = 128


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Radians per position of each pair and the amplitude."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ramp":
        dim = lambda t: rot * math.log(original_len / (2 * math.pi * t)) / (2 * math.log(base))
        first, last = max(0, math.floor(dim(high))), min(rot - 1, math.ceil(dim(low)))
        g = np.clip((np.arange(rot // 2) - first) / max(last - first, 0.001), 0, 1)
        return f * (1 - g) + f / factor * g, 0.1 * math.log(factor) + 1
    if scaling == "smooth":
        g = np.clip((original_len * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return f * g + f / factor * (1 - g), 1.0
    return f, 1.0


def angles(pos, turns):
    """Radians in [0, 2 pi) of every position and pair, from the fixed-point turns, exactly."""
    return np.array([[(int(p) * int(t) % 2 ** 64) / 2 ** 64 * 2 * math.pi for t in turns] for p in pos])


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turned(x, angle, rot, interleaved, amplitude=1.0, weight=None, eps=0.0):
    """x [layers][rows][heads][128] turned by angle [rows][rot / 2]; returns it with the sum of
    the magnitudes that went into each value."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    a, b = pairs(rot, interleaved)
    c, s = amplitude * np.cos(angle)[None, :, None], amplitude * np.sin(angle)[None, :, None]
    y, mag = x.copy(), np.abs(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, mag


def cross_attention(q, k, v):
    """q [rows][hq][128] over k, v [hkv][n][128]; returns the outputs and sum_j w_j |v_j|."""
    rows, hq, _ = q.shape
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    if k.shape[1] == 0:
        return out, mag
    for h in range(hq):
        g = h // (hq // k.shape[0])
        z = q[:, h] @ k[g].T / math.sqrt(D)
        w = np.exp(z - z.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        out[:, h], mag[:, h] = w @ v[g], w @ np.abs(v[g])
    return out, mag


def score(x, token, n_top):
    """x [rows][vocab] float64, token [rows]: log probabilities, ranks, entropies, best tokens and
    theirs."""
    rows, vocab = x.shape
    lp, rank, ent = np.full(rows, np.nan), np.full(rows, -1), np.full(rows, np.nan)
    top, top_lp = np.full((rows, n_top), -1), np.full((rows, n_top), np.nan)
    for r in range(rows):
        t = int(token[r])
        if t < 0:
            lp[r] = 0.0
        m = x[r].max()
        if not np.isfinite(m):          # (NaN, +inf, or -inf alone)
            continue
        w = np.exp(x[r] - m)
        ls = math.log(w.sum())          # (beside m: added to it, it would round at the size of m)
        p = w / w.sum()
        ent[r] = -(p[p > 0] * np.log(p[p > 0])).sum()
        order = np.lexsort((np.arange(vocab), -x[r]))[:n_top]
        top[r], top_lp[r] = order, x[r][order] - m - ls
        if 0 <= t < vocab:
            lp[r] = x[r, t] - m - ls
            rank[r] = (x[r] > x[r, t]).sum() + (x[r, :t] == x[r, t]).sum()
    return lp, rank, ent, top, top_lp
