"""Plain NumPy fp64 model of rotary positions and of trees of drafted tokens beside
the paged cache of cache_ref.py.  Loops over sequences, heads and nodes; shares no
code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

import oracle.cache_ref as cr


# --------------------------------------------------------------- rotation ---

def cos_sin(pos, inv_freq):
    """cos and sin of pos * inv_freq, pos whole numbers [..], inv_freq fp32 [m]: the product
    (31 + 24 bits) is exact in the long type, and a turn is taken off there."""
    x = np.asarray(pos).astype(np.longdouble)[..., None] * np.asarray(inv_freq, np.float32).astype(np.longdouble)
    two_pi = np.longdouble(2) * np.longdouble("3.14159265358979323846264338327950288")
    x = x - np.rint(x / two_pi) * two_pi
    return np.cos(x).astype(np.float64), np.sin(x).astype(np.float64)


def rotate(x, pos, inv_freq, interleaved=False, scale=1.0, transpose=False):
    """x [.., T, d] turned to positions pos [T]."""
    x = np.asarray(x, np.float64).copy()
    h = len(inv_freq)
    c, s = cos_sin(pos, inv_freq)
    if transpose:
        s = -s
    lo, hi = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    a, b = x[..., lo].copy(), x[..., hi].copy()
    x[..., lo] = (a * c - b * s) * np.float64(np.float32(scale))
    x[..., hi] = (a * s + b * c) * np.float64(np.float32(scale))
    return x


# ------------------------------------------------------------------ trees ---

def lines(parent) -> list[list[int]]:
    """Each node's line, from the root to the node itself."""
    out: list[list[int]] = []
    for t, up in enumerate(parent):
        out.append((out[up] if 0 <= up < t else []) + [t])
    return out


def depths(parent) -> np.ndarray:
    return np.array([len(p) - 1 for p in lines(parent)], np.int64)


def accept(token, target, prev, parent, n_new=None):
    """(paths, last): each sequence's accepted path and the choice after it."""
    B, T = token.shape
    paths, last = [], []
    for b in range(B):
        m = T if n_new is None else int(n_new[b])
        best: list[int] = []
        for line in lines(parent[b][:m]):
            after = [prev[b]] + [target[b][t] for t in line[:-1]]
            if all(token[b][t] == a for t, a in zip(line, after)) and len(line) > len(best):
                best = line
        paths.append(best)
        last.append(target[b][best[-1]] if best else prev[b])
    return paths, np.array(last)


def attention(c: dict, Q, K, V, gid, parent, w: int, scale: float, n_new=None) -> dict:
    """Q [B, H, T, d], K, V [B, H_kv, T, d].  Returns O, lse (NaN where t >= n_new) and for error
    bounds what cache_ref.attention returns (page: the largest value of the page of the kept
    slot, or of the drafted row, with the most weight * scale)."""
    Q, K, V = (np.asarray(x, np.float64) for x in (Q, K, V))
    B, H, T, d = Q.shape
    H_kv, A = c["k"].shape[1], gid.shape[1]
    G = H // H_kv
    O, pv = np.full((B, H, T, d), np.nan), np.full((B, H, T, d), np.nan)
    lse, dot = np.full((B, H, T), np.nan), np.zeros((B, H, T))
    kept, big = np.zeros((B, H, T), np.int64), np.zeros((B, H, T))
    for b in range(B):
        m = T if n_new is None else int(n_new[b])
        line = lines(parent[b][:m])
        for h in range(H):
            kv = h // G
            page, row = cr.slots(c, b, kv)
            k, v = cr.values(c, "k", page, kv, row), cr.values(c, "v", page, kv, row)
            pos, ids = c["pos"][page, kv, row].astype(np.int64), c["gid"][page, kv, row]
            mine = gid[b, 0 if A == 1 else kv]
            for t in range(m):
                i = int(c["next"][b]) + len(line[t]) - 1
                keep = (pos <= i) & ((i - pos < max(w, 1)) | (ids == mine[t]))
                own = [j for x, j in enumerate(line[t]) if len(line[t]) - 1 - x < max(w, 1) or mine[j] == mine[t]]
                ks, vs = np.concatenate([k[keep], K[b, kv, own]]), np.concatenate([v[keep], V[b, kv, own]])
                step = np.concatenate([c["v_scale"][page[keep], kv].astype(np.float64),
                                       [2.0 ** cr.need_exp(V[b, kv, j]) for j in own]])
                with np.errstate(invalid="ignore", over="ignore"):
                    s = ks @ Q[b, h, t] * scale
                    top = s.max()
                    p = np.exp(s - top)
                    lse[b, h, t] = top + np.log(p.sum())
                    p /= p.sum()
                    O[b, h, t], pv[b, h, t] = p @ vs, p @ np.abs(vs)
                    kept[b, h, t] = len(s)
                    big[b, h, t] = 448.0 * step[np.argmax(s / np.log(2.0) + np.log2(step))]
                    dot[b, h, t] = scale * (np.abs(ks) @ np.abs(Q[b, h, t])).max()
    return dict(O=O, lse=lse, pv=pv, dot=dot, kept=kept, page=big)
