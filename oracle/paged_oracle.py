"""Plain float64 definitions of the paged key/value cache operators: RoPE
tables, head norms with rotation, publication into 128-row pages, and attention
over such a cache.  Test infrastructure; shares no code with the CUDA library."""

from __future__ import annotations

import math

import numpy as np

PAGE = 128


def rope_frequencies(rope_dim, theta=10000.0, scaling="none", factor=1.0, orig_len=0,
                     beta_fast=32.0, beta_slow=1.0):
    """Rotation per position of each channel pair, [rope_dim / 2]."""
    d = rope_dim
    base = theta * factor ** (d / (d - 2)) if scaling == "ntk" else theta
    f = np.array([base ** (-2.0 * i / d) for i in range(d // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        def pair(turns):
            return d * math.log(orig_len / (2 * math.pi * turns)) / (2 * math.log(theta))

        lo = max(math.floor(pair(beta_fast)), 0)
        hi = min(math.ceil(pair(beta_slow)), d - 1)
        r = np.clip((np.arange(d // 2) - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f * (1 - r) + f / factor * r
    return f


def rope_table(n_pos, rope_dim, pos0=0, attn_factor=1.0, **kw):
    a = (pos0 + np.arange(n_pos, dtype=np.float64))[:, None] * rope_frequencies(rope_dim, **kw)
    return attn_factor * np.cos(a), attn_factor * np.sin(a)


def norm_rotate(x, pos, *, norm=True, gamma=None, eps=1e-6, cos=None, sin=None,
                layout="adjacent", start=None):
    """x [rows, heads, dim] normed over each head and turned at pos [rows]."""
    y = np.array(x, dtype=np.float64)
    if norm:
        y = y / np.sqrt(np.mean(y * y, -1, keepdims=True) + eps)
        if gamma is not None:
            y = y * np.asarray(gamma, dtype=np.float64)
    if cos is None:
        return y
    half = cos.shape[1]
    start = y.shape[-1] - 2 * half if start is None else start
    for t, p in enumerate(pos):
        if p < 0 or p >= cos.shape[0]:
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if layout == "adjacent" else (i, i + half)
            u, v = y[t, :, start + a].copy(), y[t, :, start + b].copy()
            c, s = float(cos[p, i]), float(sin[p, i])
            y[t, :, start + a] = u * c - v * s
            y[t, :, start + b] = u * s + v * c
    return y


def mxfp8_exponent(group):
    """The smallest e with 448 * 2^e >= amax (amax 0: -127)."""
    amax = float(np.max(np.abs(group)))
    if amax == 0:
        return -127
    e = math.ceil(math.log2(amax / 448.0))
    while 448.0 * 2.0 ** e < amax:
        e += 1
    while 448.0 * 2.0 ** (e - 1) >= amax:
        e -= 1
    return max(-127, min(127, e))


def visible(p, kv_len, causal=True, window=0):
    """Half-open range of the positions that a row at p sees."""
    hi = min(kv_len, p + 1) if causal else kv_len
    lo = max(0, p - window + 1) if window > 0 else 0
    return lo, max(lo, hi)


def paged_attention(q, row_req, row_pos, k_pool, v_pool, table, kv_len, scale, *, causal=True,
                    window=0, sink=None):
    """out [rows, heads, dim], lse [rows, heads], and spread, the sum of
    p_j |v_j| (what a relative error of the probabilities can move out by).
    Positions on unmapped pages are not seen."""
    T, H, D = q.shape
    nb, _, KH, _ = k_pool.shape
    G = H // KH
    out, spread = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    for t in range(T):
        b = int(row_req[t])
        if b < 0 or b >= len(kv_len):
            continue
        lo, hi = visible(int(row_pos[t]), min(int(kv_len[b]), table.shape[1] * PAGE), causal, window)
        j = np.arange(lo, hi)
        phys = np.asarray(table[b])[j // PAGE] if len(j) else np.zeros(0, dtype=np.int64)
        keep = (phys >= 0) & (phys < nb)
        j, phys = j[keep], phys[keep].astype(np.int64)
        k, v = k_pool[phys, j % PAGE], v_pool[phys, j % PAGE]  # [n, KH, D]
        for h in range(H):
            x = scale * (k[:, h // G] @ q[t, h])
            s = -np.inf if sink is None else float(sink[h])
            m = max([s] + [float(x.max())] if len(x) else [s])
            if m == -np.inf:
                continue
            w = np.exp(x - m)
            L = w.sum() + math.exp(s - m)
            out[t, h] = w @ v[:, h // G] / L
            spread[t, h] = w @ np.abs(v[:, h // G]) / L
            lse[t, h] = m + math.log(L)
    return out, lse, spread
