"""fp64 oracle of the prompt and attention calls (include/ssm_prompt.h, include/ssm_attention.h):
the definitions, token by token and row by row, in numpy."""
from __future__ import annotations

import numpy as np

from .ssm_oracle import silu, softplus


def prompt_conv(conv_w, conv_b, rows, window):
    """rows [T, c], window [3, c] (the rows before the first, oldest first): (post [T, c], the last
    three rows, sum of |products| + |bias| for error bounds)."""
    r = np.concatenate([window, rows])
    T = len(rows)
    z = np.zeros(rows.shape) + conv_b
    mag = np.zeros(rows.shape) + np.abs(conv_b)
    for t in range(T):
        for k in range(4):
            z[t] += conv_w[:, k] * r[t + k]
            mag[t] += np.abs(conv_w[:, k] * r[t + k])
    return silu(z), r[len(r) - 3:], mag


def prompt_scan(x, B, C, dt, dt_bias, A_log, D, h0, magnitude=False):
    """x [T, H, P], B, C [T, G, N], dt [T, H], h0 [H, P, N]: (y [T, H, P], h after the last token).
    magnitude: the same sums over absolute values (decays and step sizes are positive), which bound
    what a relative error of the summands can do."""
    T, H, P = x.shape
    G = B.shape[1]
    a = np.abs if magnitude else (lambda v: v)
    x, B, C, D, h = a(x), a(B), a(C), a(D), a(np.array(h0, np.float64))
    of = np.arange(H) // (H // G)
    y = np.zeros((T, H, P))
    for t in range(T):
        delta = softplus(dt[t] + dt_bias)
        h = np.exp(-delta * np.exp(A_log))[:, None, None] * h + delta[:, None, None] * x[t][:, :, None] * B[t, of][:, None]
        y[t] = np.einsum("hpn,hn->hp", h, C[t, of]) + D[:, None] * x[t]
    return y, h


def tree_attention(q, k, v, parent, k_cache, v_cache, scale):
    """q [n, Hq, D], k, v [n, Hkv, D], caches [len, Hkv, D]: (o [n, Hq, D], sum of weight |v|).
    Node u sees the cache's rows, its ancestors and itself; nothing of any other row is read."""
    n, Hq, D = q.shape
    g = Hq // k.shape[1]
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    for u in range(n):
        chain, w = [], u
        while w >= 0:
            chain.append(w)
            w = int(parent[w])
        for j in range(Hq):
            K = np.concatenate([k_cache[:, j // g], k[chain, j // g]])
            V = np.concatenate([v_cache[:, j // g], v[chain, j // g]])
            s = (K @ q[u, j]) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            o[u, j], mag[u, j] = p @ V, p @ np.abs(V)
    return o, mag


def kv_commit(pages, rows, path, table, length):
    """pages [n_pages, Hkv, page, D] (changed in place), rows [n, Hkv, D], path: node indices.  Returns the new length."""
    page = pages.shape[2]
    for i, u in enumerate(path):
        at = length + i
        pages[table[at // page], :, at % page] = rows[u]
    return length + len(path)
