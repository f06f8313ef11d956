"""CPU float64 oracle of the paged-cache operators.

TEST INFRASTRUCTURE ONLY, like the rest of this package: the plain statement of
a chunk's append to pages, its attention over them, the weights that cached
tokens receive from it, and their eviction.

A sequence is its tokens' keys and values in order, [tokens][kv_heads][d];
where they lie in a pool is the test's business.  Token a sees token j <= a when
j < m (the prefix, or a few tokens that stay visible) or j > a - n (the window;
N(t) = P U D_n(t), "Unlimited-OCR deep dive", R-SWA pseudo-code block).
"""

from __future__ import annotations

import numpy as np

__all__ = ["sees", "attend", "weigh", "evict"]


def sees(a, m, n):
    """The tokens that token a sees, in order."""
    return [j for j in range(a + 1) if j < m or j > a - n]


def attend(q, K, V, m, n):
    """Rows q [T][H][d], the last T tokens of K, V [L][kv_heads][d].  Returns o
    [T][H][d], lse [T][H], the sums of p |v| [T][H][d], and the largest
    sum |q k| / sqrt(d) of each row and head [T][H]."""
    q, K, V = (np.asarray(x, np.float64) for x in (q, K, V))
    T, H, d = q.shape
    L, Hkv = K.shape[:2]
    o, mass = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse, size = np.zeros((T, H)), np.zeros((T, H))
    for i in range(T):
        at = sees(L - T + i, m, n)
        for h in range(H):
            k, v = K[at, h // (H // Hkv)], V[at, h // (H // Hkv)]
            x = k @ q[i, h] / np.sqrt(d)
            top = x.max()
            w = np.exp(x - top)
            o[i, h], mass[i, h] = w @ v / w.sum(), w @ np.abs(v) / w.sum()
            lse[i, h] = top + np.log(w.sum())
            size[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() / np.sqrt(d)
    return o, lse, mass, size


def weigh(q, K, lse, m, n):
    """What each of the L tokens receives: [kv_heads][L], the sum of
    exp(q k / sqrt(d) - lse) over the rows that see it and the heads of its group."""
    q, K, lse = (np.asarray(x, np.float64) for x in (q, K, lse))
    T, H, d = q.shape
    L, Hkv = K.shape[:2]
    w = np.zeros((Hkv, L))
    for i in range(T):
        at = sees(L - T + i, m, n)
        for h in range(H):
            g = h // (H // Hkv)
            w[g, at] += np.exp(K[at, g] @ q[i, h] / np.sqrt(d) - lse[i, h])
    return w


def evict(weights, budget, first, last):
    """The tokens that stay of one head's L weights, in order."""
    L = len(weights)
    if L <= budget:
        return list(range(L))
    middle = range(first, L - last)
    weight = [-np.inf if np.isnan(w) else w for w in weights]
    # a NaN weighs less than anything, the least number too
    heavy = sorted(middle, key=lambda j: (np.isnan(weights[j]), -weight[j], j))
    return list(range(first)) + sorted(heavy[:budget - first - last]) + list(range(L - last, L))
