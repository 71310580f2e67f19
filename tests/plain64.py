"""Plain 64-bit forms of the operators around one-decay heads, on the CPU.

Written from the operators' definitions, row by row; numpy only.
"""
import numpy as np


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def gdn(lens, q, k, v, a, b, A_log, dt_bias, state, slots, scale, l2=True, eps=1e-6):
    """Outputs (NaN where no row is written) and states after the rule over
    consecutive sequences.  q, k: [T][Hk][dk]; v: [T][Hv][dv]; state: [slots][Hv][dk][dv]."""
    T, Hv, dv = v.shape
    rep = Hv // q.shape[1]
    state = state.copy()
    out = np.full((T, Hv, dv), np.nan)
    if l2:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + eps)
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    alpha, beta = np.exp(-np.exp(A_log) * softplus(a + dt_bias)), sigmoid(b)
    t = 0
    for n, ln in enumerate(lens):
        s = int(slots[n])
        if s < 0:
            t += ln
            continue
        S = state[s]
        for _ in range(ln):
            S = S * alpha[t][:, None, None]
            u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            out[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
            t += 1
        state[s] = S
    return out, state


def conv(lens, x, w, state, slots):
    """y (NaN where no row is written) and states.  x: [T][C]; w: [C][K]; state: [slots][K-1][C]."""
    K = w.shape[1]
    y, state = np.full(x.shape, np.nan), state.copy()
    t = 0
    for n, ln in enumerate(lens):
        s = int(slots[n])
        if s >= 0 and ln:
            full = np.concatenate([state[s], x[t:t + ln]])
            acc = sum(full[j:j + ln] * w[:, j] for j in range(K))
            y[t:t + ln] = acc * sigmoid(acc)
            state[s] = full[ln:]
        t += ln
    return y, state


def block_norm(y, gate, act, residual, alpha, post, post_w, pre_w, eps):
    t = y
    if post:
        t = t / np.sqrt((t * t).mean(-1, keepdims=True) + eps) * post_w
    if act == 1:
        t = t * sigmoid(gate)
    elif act == 2:
        t = t * gate * sigmoid(gate)
    h = alpha * t + (0 if residual is None else residual)
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * pre_w


def compact_plan(live):
    """(moves, remap) that close the holes of a pool."""
    L = int(np.count_nonzero(live))
    holes = [i for i in range(L) if not live[i]]
    movers = [i for i in range(L, len(live)) if live[i]]
    remap = [i if live[i] and i < L else -1 for i in range(len(live))]
    for s, d in zip(movers, holes):
        remap[s] = d
    return list(zip(movers, holes)), remap


def rel(x, ref):
    """Relative 2-norm of the difference, over the values that the reference has."""
    x, ref = np.asarray(x, np.float64), np.asarray(ref, np.float64)
    m = ~np.isnan(ref)
    d, n = np.linalg.norm(x[m] - ref[m]), np.linalg.norm(ref[m])
    return d / n if n else d
