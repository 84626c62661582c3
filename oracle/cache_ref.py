"""Plain NumPy fp64 model of the paged 8-bit key/value cache: append, attention
over it, eviction.  One loop per sequence, head and page; shares no code with
the CUDA path.

A cache is a dict of arrays: k, v [n_pages, H_kv, 64, d] uint8 codes, k_scale,
v_scale [n_pages, H_kv], pos, gid, mass [n_pages, H_kv, 64], table [B, max_pages],
len [B, H_kv], next [B].
"""
from __future__ import annotations

import numpy as np

PAGE = 64
MIN_EXP = -64


def _table() -> np.ndarray:
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        if c & 127 == 127:
            x = np.nan
        v[c] = -x if c & 128 else x
    return v


VALUES = _table()              # the number each e4m3 code stands for
_POSITIVE = VALUES[:127]       # ascending


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code, ties to the even code, saturating; NaN -> NaN code."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def need_exp(rows: np.ndarray) -> int:
    """Least e >= MIN_EXP with every finite |value| <= 448 * 2^e."""
    a = np.abs(rows[np.isfinite(rows)])
    top = float(a.max()) if a.size else 0.0
    e = MIN_EXP
    while 448.0 * 2.0 ** e < top:
        e += 1
    return e


def copy(c: dict) -> dict:
    return {k: v.copy() for k, v in c.items()}


def slots(c: dict, b: int, h: int):
    """(page, row) arrays of the slots in use of one head, in order."""
    s = np.arange(c["len"][b, h])
    return c["table"][b][s // PAGE], s % PAGE


def values(c: dict, name: str, page, h: int, row) -> np.ndarray:
    return VALUES[c[name][page, h, row]] * c[name + "_scale"][page, h].astype(np.float64)[..., None]


def append(c: dict, K, V, gid, n_new=None) -> dict:
    """K, V [B, H_kv, T, d]; gid [B, A, T].  Returns the cache after the append."""
    c = copy(c)
    B, H_kv, T, _ = K.shape
    A = gid.shape[1]
    for b in range(B):
        m = T if n_new is None else int(n_new[b])
        if (c["len"][b] + m).max() > c["table"].shape[1] * PAGE:
            continue
        for h in range(H_kv):
            n = int(c["len"][b, h])
            for s0 in range(n // PAGE * PAGE, n + m, PAGE):
                lo, hi = max(n, s0), min(n + m, s0 + PAGE)
                if lo >= hi:
                    continue
                g, r = int(c["table"][b, s0 // PAGE]), lo - s0
                for name, x in (("k", K), ("v", V)):
                    rows = np.asarray(x[b, h, lo - n:hi - n], np.float64)
                    e = need_exp(rows)
                    if r:
                        was = float(c[name + "_scale"][g, h])
                        e = max(e, int(np.log2(was)))
                        c[name][g, h, :r] = encode(VALUES[c[name][g, h, :r]] * was / 2.0 ** e)
                    c[name][g, h, r:r + hi - lo] = encode(rows / 2.0 ** e)
                    c[name + "_scale"][g, h] = 2.0 ** e
                c["pos"][g, h, r:r + hi - lo] = c["next"][b] + np.arange(lo - n, hi - n)
                c["gid"][g, h, r:r + hi - lo] = gid[b, 0 if A == 1 else h, lo - n:hi - n]
                if "mass" in c:
                    c["mass"][g, h, r:r + hi - lo] = 0.0
        c["len"][b] += m
        c["next"][b] += m
    return c


def attention(c: dict, Q, gid, w: int, scale: float, n_new=None) -> dict:
    """Q [B, H, T, d].  Returns O, lse (NaN where t >= n_new), the weight every
    slot received (got, like mass), and for error bounds: pv = sum P |v|, dot = the
    largest scale * sum |q| |k| of a row, kept = slots kept by a row, page = the
    largest value that the page of the slot with the most weight * page scale holds."""
    Q = np.asarray(Q, np.float64)
    B, H, T, d = Q.shape
    H_kv, A = c["k"].shape[1], gid.shape[1]
    G = H // H_kv
    O, pv = np.full((B, H, T, d), np.nan), np.full((B, H, T, d), np.nan)
    lse, dot = np.full((B, H, T), np.nan), np.zeros((B, H, T))
    kept, big = np.zeros((B, H, T), np.int64), np.zeros((B, H, T))
    got = np.zeros(c["pos"].shape)
    for b in range(B):
        m = T if n_new is None else int(n_new[b])
        for h in range(H):
            kv = h // G
            page, row = slots(c, b, kv)
            k, v = values(c, "k", page, kv, row), values(c, "v", page, kv, row)
            pos, ids = c["pos"][page, kv, row].astype(np.int64), c["gid"][page, kv, row]
            for t in range(m):
                i = int(c["next"][b]) - m + t
                keep = (pos <= i) & ((i - pos < max(w, 1)) | (ids == gid[b, 0 if A == 1 else kv, t]))
                kept[b, h, t] = keep.sum()
                if not keep.any():
                    O[b, h, t], pv[b, h, t], lse[b, h, t] = 0.0, 0.0, -np.inf
                    continue
                s = k[keep] @ Q[b, h, t] * scale
                top = s.max()
                vs = c["v_scale"][page[keep], kv].astype(np.float64)
                big[b, h, t] = 448.0 * vs[np.argmax(s / np.log(2.0) + np.log2(vs))]
                p = np.exp(s - top)
                lse[b, h, t] = top + np.log(p.sum())
                p /= p.sum()
                O[b, h, t], pv[b, h, t] = p @ v[keep], p @ np.abs(v[keep])
                dot[b, h, t] = scale * (np.abs(k[keep]) @ np.abs(Q[b, h, t])).max()
                np.add.at(got, (page[keep], kv, row[keep]), p)
    return dict(O=O, lse=lse, got=got, pv=pv, dot=dot, kept=kept, page=big)


def stays(mass, pos, nxt: int, budget: int, recent: int) -> np.ndarray:
    """Indices, ascending, of the slots of one head that an eviction keeps."""
    n = len(mass)
    if n <= budget:
        return np.arange(n)
    late = [s for s in range(n) if pos[s] >= nxt - recent]

    def rank(s):
        x = float(mass[s])
        return (0, 0.0, s) if np.isnan(x) else (1, -x, s)

    rest = sorted((s for s in range(n) if pos[s] < nxt - recent), key=rank)
    return np.array(sorted((late + rest)[:budget]), np.int64)


def evict(src: dict, dst: dict, budget: int, recent: int) -> dict:
    """dst after the eviction's copy of what stays of src."""
    out = copy(dst)
    B, H_kv = src["len"].shape
    for b in range(B):
        for h in range(H_kv):
            page, row = slots(src, b, h)
            at = stays(src["mass"][page, h, row], src["pos"][page, h, row], int(src["next"][b]), budget, recent)
            page, row = page[at], row[at]
            for j in range(0, len(at), PAGE):
                g, pg, rw = int(dst["table"][b, j // PAGE]), page[j:j + PAGE], row[j:j + PAGE]
                for name in ("k", "v"):
                    x = values(src, name, pg, h, rw)
                    e = need_exp(x)
                    out[name][g, h, :len(pg)] = encode(x / 2.0 ** e)
                    out[name + "_scale"][g, h] = 2.0 ** e
                for name in ("pos", "gid", "mass"):
                    out[name][g, h, :len(pg)] = src[name][pg, h, rw]
            out["len"][b, h] = len(at)
        out["next"][b] = src["next"][b]
    return out


def empty(B: int, H_kv: int, d: int, n_pages: int, max_pages: int, seed: int) -> dict:
    """An empty cache whose pages lie anywhere in the pool, with junk in the unused rows."""
    rng = np.random.default_rng(seed)
    shape = (n_pages, H_kv, PAGE)
    table = np.full((B, max_pages), -1, np.int32)              # entries past the last page are not read
    pages = rng.permutation(n_pages)[:B * max_pages].reshape(B, -1)
    table[:, :pages.shape[1]] = pages
    return dict(k=rng.integers(0, 256, shape + (d,)).astype(np.uint8), v=rng.integers(0, 256, shape + (d,)).astype(np.uint8),
                k_scale=np.full(shape[:2], np.float32(np.nan)), v_scale=np.full(shape[:2], np.float32(np.nan)),
                pos=rng.integers(0, 1 << 20, shape).astype(np.int32), gid=np.zeros(shape, np.int16),
                mass=np.full(shape, np.float32(np.nan)), table=table, len=np.zeros((B, H_kv), np.int32),
                next=np.zeros(B, np.int32))
