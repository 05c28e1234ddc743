"""The operators between the q/k/v projection and the output projection, from their definitions, in numpy and fp64:
norms and rotation of heads, the paged cache, and attention over a shared prefix.  Test infrastructure only."""
from __future__ import annotations

import math

import numpy as np


def head_norm(x, weight, bias, kind, eps):
    """x (tokens, heads, D) normed over D."""
    x = np.asarray(x, dtype=np.float64)
    if kind is None:
        return x
    if kind == "layer":
        x = x - x.mean(axis=-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    return y if bias is None else y + bias


def rotate(x, positions, inv_freq, axis, pairs):
    """The first 2 len(inv_freq) values of each head turned: pair i of token t by positions[axis[i], t] *
    inv_freq[i].  The angle is reduced in Python's integers and fractions of a turn would not be exact, so positions
    stay below 2^31 and frequencies are doubles: pos * freq is off by 2^-53 of itself."""
    y = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (i, i + n) if pairs == "halves" else (2 * i, 2 * i + 1)
        for t in range(x.shape[0]):
            angle = math.fmod(float(positions[axis[i]][t]) * f, 2.0 * math.pi)
            c, s = math.cos(angle), math.sin(angle)
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def attention(q, k, v, tables, seq_lens, prefix_pages, prefix_len, q_start, scale):
    """(out, lse, spread, reach) of tokens q (T, Hq, D) over a paged cache k, v (pages, page, Hkv, D): spread =
    sum_j p_j |v_j|, reach = max_j scale sum_d |q_d k_jd| (for tolerances).  Tokens behind q_start's last entry get
    NaN."""
    T, heads, D = q.shape
    pages, page, kv, _ = k.shape
    group = heads // kv
    out = np.full((T, heads, D), np.nan)
    spread = np.full((T, heads, D), np.nan)
    lse = np.full((T, heads), np.nan)
    reach = np.zeros((T, heads))

    def rows(table, n):
        if n == 0:
            return np.zeros((0, kv, D)), np.zeros((0, kv, D))
        at = np.arange(n)
        p = np.asarray(table, dtype=np.int64)[at // page]
        ok = (p >= 0) & (p < pages)
        p = np.where(ok, p, 0)
        return tuple(np.where(ok[:, None, None], c[p, at % page], 0.0) for c in (k, v))

    kp, vp = rows(prefix_pages, prefix_len)
    for b, m in enumerate(seq_lens):
        t0, t1 = q_start[b], q_start[b + 1]
        ks, vs = rows(tables[b], m)
        for t in range(t0, t1):
            seen = max(0, m - (t1 - t0) + (t - t0) + 1)
            K, V = np.concatenate((kp, ks[:seen])), np.concatenate((vp, vs[:seen]))
            for h in range(heads):
                Kh, Vh = K[:, h // group], V[:, h // group]
                if len(Kh) == 0:
                    out[t, h], spread[t, h], lse[t, h] = 0.0, 0.0, -np.inf
                    continue
                s = scale * (Kh @ q[t, h])
                top = s.max()
                e = np.exp(s - top)
                w = e / e.sum()
                out[t, h] = w @ Vh
                spread[t, h] = w @ np.abs(Vh)
                lse[t, h] = top + math.log(e.sum())
                reach[t, h] = scale * (np.abs(Kh) @ np.abs(q[t, h])).max()
    return out, lse, spread, reach
