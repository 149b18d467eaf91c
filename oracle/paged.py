"""CPU oracle of the paged cache's operators (test infrastructure only): plain float64 numpy
statements, sharing nothing with the CUDA path. Pages of e4m3 codes are held as the codes' values."""
from __future__ import annotations

import math

import numpy as np

from . import decode_ref as O

MIN_EXP = -64


def _e4m3_values():
    """The finite values of e4m3 that are not negative, in order: sign, 4 exponent bits (bias 7), 3
    fraction bits; all ones is NaN."""
    out = []
    for code in range(0x7f):
        e, f = code >> 3, code & 7
        out.append(f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return np.array(out)


E4M3 = _e4m3_values()


def to_e4m3(x):
    """The nearest value, ties to the even code; beyond the largest the largest, NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 0, E4M3.size - 1)
    lo = np.maximum(hi - 1, 0)
    with np.errstate(invalid="ignore"):
        up, down = E4M3[hi] - a, a - E4M3[lo]
        take_hi = (up < down) | ((up == down) & (hi % 2 == 0)) | (a >= E4M3[-1])
    r = np.where(take_hi, E4M3[hi], E4M3[lo])
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def scale_for(x):
    """The smallest power of two s >= 2^-64 with |x| <= 448 s for the finite x."""
    a = np.abs(x[np.isfinite(x)])
    top = a.max(initial=0.0)
    e = MIN_EXP
    while top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotated(x, w, pos, theta, layout, rot, eps, inv_freq=None):
    """x [heads, D] at position pos: RMSNorm over D, then RoPE of the first `rot` elements."""
    x = np.asarray(x, dtype=np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y = x.copy()
    half = rot // 2
    for i in range(half):
        f = theta ** (-2.0 * i / rot) if inv_freq is None else inv_freq[i]
        c, s = math.cos(pos * f), math.sin(pos * f)
        p, q = (i, i + half) if layout == "neox" else (2 * i, 2 * i + 1)
        y[:, p] = x[:, p] * c - x[:, q] * s
        y[:, q] = x[:, p] * s + x[:, q] * c
    return y


def append(q, k_new, v_new, cache, table, start, cu, theta, layout, rot, qw=None, kw=None,
           eps=1e-6, inv_freq=None):
    """Rotated q, and the cache after the append: cache = dict(k, v [P, Hkv, page, D], ks, vs
    [P, Hkv] or None)."""
    c = {n: None if a is None else np.array(a, dtype=np.float64) for n, a in cache.items()}
    P, Hkv, page, D = c["k"].shape
    q = np.array(q, dtype=np.float64)
    for b in range(len(start)):
        lo, hi = (b, b + 1) if cu is None else (int(cu[b]), int(cu[b + 1]))
        runs = {}  # slot -> tokens
        for i in range(lo, hi):
            p = int(start[b]) + i - lo
            if start[b] < 0:
                continue
            q[i] = rotated(q[i], qw, p, theta, layout, rot, eps, inv_freq)
            if p // page < table.shape[1] and 0 <= table[b, p // page] < P:
                runs.setdefault(p // page, []).append((i, p))
        for slot, tokens in runs.items():
            at, r0 = int(table[b, slot]), tokens[0][1] % page
            n = len(tokens)
            k = np.stack([rotated(k_new[i], kw, p, theta, layout, rot, eps, inv_freq)
                          for i, p in tokens], 1)
            v = np.stack([np.asarray(v_new[i], dtype=np.float64) for i, _ in tokens], 1)
            for x, pages, scales in ((k, c["k"], c["ks"]), (v, c["v"], c["vs"])):
                if scales is None:
                    pages[at, :, r0:r0 + n] = x
                    continue
                for g in range(Hkv):
                    s = scale_for(x[g])
                    if r0 > 0:
                        s = max(s, scales[at, g])
                        if s > scales[at, g]:
                            pages[at, g, :r0] = to_e4m3(pages[at, g, :r0] * (scales[at, g] / s))
                    scales[at, g] = s
                    pages[at, g, r0:r0 + n] = to_e4m3(x[g] / s)
    return q, c


def tokens(cache, table, b, lo, hi):
    """(K, V) [Hkv, hi - lo, D] of sequence b's tokens, and which of them have a page."""
    P, Hkv, page, D = cache["k"].shape
    K, V = np.zeros((Hkv, hi - lo, D)), np.zeros((Hkv, hi - lo, D))
    has = np.zeros(hi - lo, dtype=bool)
    for t in range(lo, hi):
        at = int(table[b, t // page])
        if not 0 <= at < P:
            continue
        has[t - lo] = True
        for pages, scales, out in ((cache["k"], cache["ks"], K), (cache["v"], cache["vs"], V)):
            out[:, t - lo] = pages[at, :, t % page] * (1 if scales is None else scales[at][:, None])
    return K, V, has


def attention(q, cache, table, lens, scale=None, window=0):
    """(out, size, floor): single-query attention, sum_t p_t |v_t|, and with codes c_t under scales s_t
    max_t p_t s_t sum_t |c_t| (0 without scales)."""
    B, Hq, D = q.shape
    Hkv = cache["k"].shape[1]
    G = Hq // Hkv
    scale = scale if scale else 1.0 / math.sqrt(D)
    out, size, floor = (np.zeros(q.shape) for _ in range(3))
    for b in range(B):
        n = int(lens[b])
        lo = max(0, n - window) if window else 0
        K, V, has = tokens(cache, table, b, lo, n)
        if not has.any():
            continue
        for g in range(Hkv):
            heads = slice(g * G, (g + 1) * G)
            w = O.softmax(scale * (q[b, heads] @ K[g, has].T))
            out[b, heads] = w @ V[g, has]
            size[b, heads] = w @ np.abs(V[g, has])
            if cache["vs"] is not None:
                page = cache["k"].shape[2]
                s = np.array([cache["vs"][int(table[b, t // page]), g] for t in np.arange(lo, n)[has]])
                floor[b, heads] = (w * s).max(1)[:, None] * np.abs(V[g, has] / s[:, None]).sum(0)
    return out, size, floor
