"""fp64 oracle of the calls of an 8-bit cache, rotary positions and token scores (include/ssm_attention.h,
include/ssm_logits.h): the definitions, row by row, in numpy."""
from __future__ import annotations

import numpy as np


def e4m3(x):
    """The nearest value of 4 exponent and 3 mantissa bits (ties to the even mantissa, at most 448); not finite: NaN."""
    x = np.asarray(x, np.float64)
    ok = np.isfinite(x)
    a = np.abs(np.where(ok, x, 0.0))
    _, e = np.frexp(a)  # a = f * 2^e, f in [1/2, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    r = np.minimum(np.rint(a / step) * step, 448.0)
    return np.where(ok, np.copysign(r, x), np.nan)


def least_scale(rows):
    """The least power of two, from 2^-100 on, under which the largest finite magnitude is at most 448 of it."""
    a = np.abs(np.asarray(rows, np.float64))
    most = np.max(np.where(np.isfinite(a), a, 0.0), initial=0.0)
    e = -100
    while most > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def kv_commit_fp8(pages, scales, rows, path, table, length):
    """pages [n_pages, Hkv, page, D] (what the 8 bits hold, without the scale) and scales [n_pages, Hkv, page / block], both
    changed in place; rows [n, Hkv, D], path: node indices.  Returns the new length."""
    page, block = pages.shape[2], pages.shape[2] // scales.shape[2]
    end = length + len(path)
    if end == length:
        return end
    for first in range(length // block * block, end, block):
        pg, at = table[first // page], first % page
        lo, hi = max(first, length), min(first + block, end)
        for j in range(pages.shape[1]):
            new = np.stack([rows[path[r - length], j] for r in range(lo, hi)])
            scale, k = least_scale(new), lo - first
            old = scales[pg, j, at // block]
            if k and 2.0 ** -100 <= old <= 2.0 ** 120:
                if old < scale:
                    pages[pg, j, at:at + k] = e4m3(pages[pg, j, at:at + k] * (old / scale))
                scale = max(scale, old)
            pages[pg, j, at + k:at + k + hi - lo] = e4m3(new / scale)
            scales[pg, j, at // block] = scale
    return end


def rope_frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "base":
        return np.array([(base * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "by_parts":
        turns = original_len * f / (2 * np.pi)
        keep = np.clip((turns - low) / (high - low), 0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor)
    return f


def rope(x, pos, freq, interleaved=False, amplitude=1.0):
    """x [T, heads, D], pos [T], freq [rot / 2]: (the turned rows, |a| + |b| of each column's pair for error bounds)."""
    y, mag = np.array(x, np.float64), np.abs(np.array(x, np.float64))
    half = len(freq)
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(pos * f)[:, None] * amplitude, np.sin(pos * f)[:, None] * amplitude
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, b] * c + x[:, :, a] * s
        mag[:, :, a] = mag[:, :, b] = abs(amplitude) * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
    return y, mag


def token_scores(x, tokens, k, scale=1.0):
    """x [T, V] fp64, tokens [T, m]: (logprob [T, m], entropy [T], top [T, k], top_logprob [T, k]).  Token -1: 0."""
    T, V = x.shape
    logprob, entropy = np.zeros(tokens.shape), np.zeros(T)
    top, top_logprob = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            m = np.max(x[t])
            lp = (x[t] - m) * scale
            lp = lp - np.log(np.sum(np.exp(lp)))
            p = np.exp(lp)
            entropy[t] = -np.sum(np.where(p == 0, 0.0, p * lp))
        key = np.where(np.isnan(x[t]), -np.inf, x[t])  # a NaN behind all others
        order = np.lexsort((np.arange(V), -key, np.isnan(x[t])))
        top[t] = order[:k]
        top_logprob[t] = lp[top[t]]
        logprob[t] = [0.0 if i == -1 else lp[i] if 0 <= i < V else np.nan for i in tokens[t]]
    return logprob, entropy, top, top_logprob
