"""Plain 64-bit forms of rotary positions and of attention over a paged cache, on the CPU.

Written from the operators' definitions, row by row; numpy only.
"""
import math

import numpy as np


def radians(rd, kind="none", base=10000.0, factor=1.0, length=4096.0, fast=32.0, slow=1.0):
    """Angle per position of each pair."""
    if kind == "base":
        base = base * factor ** (rd / (rd - 2))
    f = np.array([base ** (-2 * i / rd) for i in range(rd // 2)])
    if kind == "linear":
        return f / factor
    if kind == "ramp":
        pair = lambda turns: rd / 2 * math.log(length / (turns * 2 * math.pi)) / math.log(base)  # noqa: E731
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rd - 1)
        r = np.clip((np.arange(rd // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - r) + f / factor * r
    if kind == "smooth":
        k = np.clip((length * f / (2 * math.pi) - slow) / (fast - slow), 0, 1)
        return f * k + f / factor * (1 - k)
    return f


def rope(x, pos, f, layout="half", amplitude=1.0, transpose=False):
    """x [rows][H][D] turned to the rows' positions, and the largest |x1| + |x2| behind each value."""
    rd = 2 * len(f)
    angle = pos[:, None].astype(np.float64) * f * (-1 if transpose else 1)
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
    i = np.arange(rd // 2)
    a, b = (i, i + rd // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y, size = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(amplitude)
    return y, size


def attn(lens, kv, q, tokens, scale, causal=True, window=0):
    """Attention of rows over their sequences' tokens.

    q: [T][Hq][D]; tokens(s) -> (keys, values [Hkv][kv][D], visible [kv]) of sequence s.
    Returns out and lse (NaN where no row is written), the weighted mean of |v| beside each output, and
    the largest scaled sum of |q_i k_i| of each row and head (what a score's rounding is relative to)."""
    T, Hq, D = q.shape
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    mean, size = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    t = 0
    for s, (n, L) in enumerate(zip(lens, kv)):
        if L >= 0 and n:
            k, v, visible = tokens(s)
            G = Hq // k.shape[0]
            j = np.arange(L)
            for r in range(n):
                p = L - n + r
                seen = visible.copy()
                if causal:
                    seen &= j <= p
                    if window:
                        seen &= j > p - window
                for h in range(Hq):
                    kk, vv, qq = k[h // G][seen], v[h // G][seen], q[t + r, h]
                    if not len(kk):
                        out[t + r, h], lse[t + r, h] = 0, -np.inf
                        continue
                    x = kk @ qq * scale
                    m = x.max()
                    w = np.exp(x - m)
                    out[t + r, h] = w @ vv / w.sum()
                    mean[t + r, h] = w @ np.abs(vv) / w.sum()
                    lse[t + r, h] = m + math.log(w.sum())
                    size[t + r, h] = (np.abs(kk) @ np.abs(qq)).max() * scale
        t += n
    return out, lse, mean, size
