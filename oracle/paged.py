"""fp64 CPU oracle of the paged-cache operators: attention of new tokens over a cache in pages, append, the weight
each cached key receives, and eviction by it. Test infrastructure, like ``oracle.attention``.

The definitions are those of ``oracle.attention`` on the keys that a sequence's page table names, in order: key j of
sequence b is row j % P of page table[b][j // P]. The new tokens of a sequence are its last keys, so a causal row i of
n sees the keys j <= i + L - n. The cached rows are read by plain indexing and the softmax is written out here again,
one K/V head at a time; ``tests/test_oracle_paged.py`` pins it against ``oracle.attention``.
"""

from __future__ import annotations

import numpy as np


def keys_of(cache, table, length, b, h):
    """fp64 [length, d]: the cached rows of sequence b and K/V head h."""
    P = cache.shape[1]
    j = np.arange(length)
    return np.asarray(cache, dtype=np.float64)[np.asarray(table)[b, j // P], j % P, h]


def new_rows(x, b, cu):
    """The new tokens' rows of sequence b, [n, heads, d]."""
    return x[b] if cu is None else x[cu[b]:cu[b + 1]]


def head_scores(q, k, scale, causal):
    """Masked scaled scores [n, L] of one query head's new rows against its keys."""
    n, L = q.shape[0], k.shape[0]
    s = scale * (np.asarray(q, dtype=np.float64) @ k.T)
    if causal:
        s[np.arange(L)[None, :] > np.arange(n)[:, None] + (L - n)] = -np.inf
    return s


def row_lse(s):
    if s.shape[1] == 0:
        return np.full(s.shape[0], -np.inf)
    m = s.max(axis=1)
    safe = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        return np.where(np.isneginf(m), -np.inf, safe + np.log(np.exp(s - safe[:, None]).sum(axis=1)))


def row_probs(s, lse):
    """exp(s - lse); rows without a visible key are 0."""
    return np.exp(s - np.where(np.isneginf(lse), np.inf, lse)[:, None])


def attention(q, k_cache, v_cache, table, lengths, scale, causal=False, cu=None):
    """Per sequence (o [n, H, d], lse [H, n], a [n, H, d]) with a = sum_j P_ij |v_j|, the scale of rounding errors."""
    out = []
    Hkv = k_cache.shape[2]
    for b, L in enumerate(lengths):
        x = new_rows(q, b, cu)
        n, H, d = x.shape
        o, a, lse = np.zeros((n, H, d)), np.zeros((n, H, d)), np.full((H, n), -np.inf)
        for h in range(H):
            k = keys_of(k_cache, table, L, b, h // (H // Hkv))
            v = keys_of(v_cache, table, L, b, h // (H // Hkv))
            s = head_scores(x[:, h], k, scale, causal)
            lse[h] = row_lse(s)
            p = row_probs(s, lse[h])
            o[:, h], a[:, h] = p @ v, p @ np.abs(v)
        out.append((o, lse, a))
    return out


def key_weights(q, k_cache, table, lengths, lses, scale, causal=False, cu=None):
    """Per sequence [Hkv, L]: the weight its rows (LSE [H, n] each) pay every key."""
    out = []
    Hkv = k_cache.shape[2]
    for b, L in enumerate(lengths):
        x = new_rows(q, b, cu)
        H = x.shape[1]
        w = np.zeros((Hkv, L))
        for h in range(H):
            k = keys_of(k_cache, table, L, b, h // (H // Hkv))
            w[h // (H // Hkv)] += row_probs(head_scores(x[:, h], k, scale, causal), np.asarray(lses[b][h], float)).sum(0)
        out.append(w)
    return out


def append(k, v, k_cache, v_cache, table, lengths, cu=None, weights=None):
    """The caches (and weights) after the new rows took the last places of their sequences, in place."""
    P = k_cache.shape[1]
    for b, L in enumerate(lengths):
        kb, vb = new_rows(k, b, cu), new_rows(v, b, cu)
        for i in range(kb.shape[0]):
            j = L - kb.shape[0] + i
            if 0 <= j < table.shape[1] * P:
                page = table[b][j // P]
                k_cache[page, j % P], v_cache[page, j % P] = kb[i], vb[i]
                if weights is not None:
                    weights[page, :, j % P] = 0.0


def evict(k_cache, v_cache, weights, table, lengths, keep, recent):
    """(kept [B, Hkv, keep], new lengths) and the caches and weights moved in place. Keys are ordered by weight, NaN
    below every number, and by index among equal weights."""
    P, Hkv = k_cache.shape[1], k_cache.shape[2]
    kept = np.full((len(lengths), Hkv, keep), -1, dtype=np.int32)
    for b, L in enumerate(lengths):
        for h in range(Hkv):
            if L <= keep:
                kept[b, h, :L] = np.arange(L)
                continue
            old = L - recent
            w = [float(weights[table[b][j // P], h, j % P]) for j in range(old)]
            order = sorted(range(old), key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0.0, j))
            stay = sorted(order[:keep - recent]) + list(range(old, L))
            kept[b, h] = stay
            src = [(table[b][j // P], j % P) for j in stay]
            rows = [(k_cache[p, s, h].copy(), v_cache[p, s, h].copy(), weights[p, h, s]) for p, s in src]
            for t, (kr, vr, wr) in enumerate(rows):
                page = table[b][t // P]
                k_cache[page, t % P, h], v_cache[page, t % P, h], weights[page, h, t % P] = kr, vr, wr
    return kept, np.minimum(np.asarray(lengths), keep)
