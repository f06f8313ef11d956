"""CPU float64 oracle of the draft-and-verify operators.

TEST INFRASTRUCTURE ONLY, like the rest of this package: the plain statement of
the norm and rotation of query and key heads, of a tree of drafted tokens over
an R-SWA cache, and of the append of its accepted path.

A cache state is the dict of ``prefill_cache`` (Kp, Vp, Kr, Vr, t).  Node i of
a tree stands for output t + depth(i) and sees what that output would see if
the chain from its root to it were the outputs t, t + 1, ... (N(t) = P U D_n(t),
"Unlimited-OCR deep dive", R-SWA pseudo-code block).
"""

from __future__ import annotations

import numpy as np

from .rswa_oracle import append_kv, ring_outputs

__all__ = ["norm_rope", "chain", "tree_attention", "commit_tree"]


def norm_rope(x, weight, positions, inv_freq, eps, interleaved):
    """x [rows][heads][d] -> y: each head y = x w / sqrt(mean(x^2) + eps) (no
    norm where weight is None), its first 2 len(inv_freq) elements turned in
    pairs by positions[row] * inv_freq[pair]."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    out = y.copy()
    for r, pos in enumerate(positions):
        for i in range(len(f)):
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + len(f))
            c, s = np.cos(float(pos) * f[i]), np.sin(float(pos) * f[i])
            a, b = y[r, :, ia], y[r, :, ib]
            out[r, :, ia], out[r, :, ib] = a * c - b * s, b * c + a * s
    return out


def chain(parents, i):
    """Node i, its parent, ... up to its root."""
    out = [i]
    while parents[out[-1]] >= 0:
        out.append(parents[out[-1]])
    return out


def tree_attention(state, q, k, v, parents, n):
    """Attention of every node of one sequence's tree.

    q [N][H][d]; k, v [N][H_kv][d]; parents [N].  Returns (o [N][H][d], lse
    [N][H], seen): seen[i] is the matrix of keys node i sees, rows of
    [prefix | cached outputs | ancestors], with K and V of the same rows, as
    (K, V) of shape [keys][H_kv][d].
    """
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    N, H, d = q.shape
    Hkv = k.shape[1]
    t = state["t"]
    slot = {j: s for s, j in ring_outputs(t, n).items()}
    o, lse, seen = np.empty((N, H, d)), np.empty((N, H)), []
    for i in range(N):
        up = chain(parents, i)
        here = t + len(up) - 1
        ring = [slot[j] for j in range(max(0, here - n + 1), t)]
        K = np.concatenate([state["Kp"], state["Kr"][ring], k[up[:n]]])
        V = np.concatenate([state["Vp"], state["Vr"][ring], v[up[:n]]])
        seen.append((K, V))
        for h in range(H):
            g = h // (H // Hkv)
            x = K[:, g] @ q[i, h] / np.sqrt(d)
            top = x.max()
            w = np.exp(x - top)
            o[i, h] = (w @ V[:, g]) / w.sum()
            lse[i, h] = top + np.log(w.sum())
    return o, lse, seen


def commit_tree(state, k, v, path, n):
    """Append the nodes of `path` in order."""
    for i in path:
        state = append_kv(state, np.asarray(k, np.float64)[i], np.asarray(v, np.float64)[i], n)
    return state
