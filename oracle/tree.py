"""CPU oracle of the draft-tree operators (test infrastructure only): plain float64 numpy
statements, one query row at a time, sharing nothing with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

from . import decode_ref as O


def rope_tree(q, k_new, v_new, q_norm_w, k_norm_w, k_tree, v_tree, pos, n_nodes, theta, layout,
              eps, inv_freq=None):
    """Rotated q, and the tree buffers with the nodes' rows written (copies)."""
    q, k_tree, v_tree = q.copy(), k_tree.copy(), v_tree.copy()
    B, N = pos.shape
    for b in range(B):
        for n in range(int(n_nodes[b])):
            p = int(pos[b, n])
            if p < 0:
                continue
            at = np.array([p])
            q[b, n] = O.qknorm_rope(q[b, n][None], q_norm_w, at, theta, layout, eps, inv_freq)[0]
            k_tree[b, :, n] = O.qknorm_rope(k_new[b, n][None], k_norm_w, at, theta, layout, eps,
                                            inv_freq)[0]
            v_tree[b, :, n] = v_new[b, n]
    return q, k_tree, v_tree


def seen_keys(L, live, n, word, pos, window):
    """Indices of the keys node n sees: cache slots t < L, then nodes as L + j."""
    keys = list(range(L)) + [L + j for j in range(live) if (word >> j) & 1]
    if window:
        p = max(int(pos[n]), L)
        at = [t if t < L else max(int(pos[t - L]), L) for t in keys]
        keys = [t for t, x in zip(keys, at) if p - x < window]
    return keys


def tree_attention(q, k_cache, v_cache, lens, k_tree, v_tree, mask, n_nodes, pos=None, slopes=None,
                   scale=None, softcap=0.0, window=0):
    """(out, absolute): attention of every live node, and sum_t p_t |v_t| beside it (the size
    the error of a weighted sum goes by). Rows of dead nodes are NaN."""
    B, N, Hq, D = q.shape
    Hkv, T_cap = k_cache.shape[1:3]
    G = Hq // Hkv
    scale = scale if scale else 1.0 / math.sqrt(D)
    out = np.full(q.shape, np.nan)
    size = np.full(q.shape, np.nan)
    for b in range(B):
        L = min(max(int(lens[b]), 0), T_cap)
        live = min(max(int(n_nodes[b]), 0), N)
        for n in range(live):
            p = None if pos is None else pos[b]
            keys = np.array(seen_keys(L, live, n, int(mask[b, n]), p, window), dtype=np.int64)
            for g in range(Hkv):
                heads = slice(g * G, (g + 1) * G)
                if keys.size == 0:
                    out[b, n, heads] = size[b, n, heads] = 0.0
                    continue
                c, t = keys[keys < L], keys[keys >= L] - L
                K = np.concatenate([k_cache[b, g, c], k_tree[b, g, t]])
                V = np.concatenate([v_cache[b, g, c], v_tree[b, g, t]])
                z = scale * (q[b, n, heads] @ K.T)
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                if slopes is not None:
                    own = max(int(p[n]), L)
                    at = np.concatenate([c, np.maximum(p[t], L)])
                    z = z - slopes[heads, None] * (own - at)[None]
                w = O.softmax(z)
                out[b, n, heads] = w @ V
                size[b, n, heads] = w @ np.abs(V)
    return out, size


def commit(k_tree, v_tree, path, n_path, k_cache, v_cache, lens):
    k, v = k_cache.copy(), v_cache.copy()
    B, N = path.shape
    T_cap = k_cache.shape[2]
    for b in range(B):
        for i in range(min(max(int(n_path[b]), 0), N)):
            node, slot = int(path[b, i]), int(lens[b]) + i
            if 0 <= node < N and 0 <= slot < T_cap:
                k[b, :, slot], v[b, :, slot] = k_tree[b, :, node], v_tree[b, :, node]
    return k, v


def logprobs(row, ids, top_k, temperature=1.0):
    """(log probabilities of ids, entropy, top ids, their log probabilities) of one row."""
    z = np.asarray(row, dtype=np.float64) / temperature
    m = z.max()
    e = np.exp(z - m)
    lse = m + math.log(e.sum())
    p = e / e.sum()
    nz = p > 0
    entropy = float(-(p[nz] * (z[nz] - lse)).sum())
    lp = np.array([z[i] - lse if 0 <= i < z.size else -np.inf for i in ids])
    top = np.lexsort((np.arange(z.size), -np.asarray(row, dtype=np.float64)))[:top_k]
    return lp, entropy, top, z[top] - lse
