"""Rotary positions, appends with the rotation on the way and the accepted paths of
drafted trees on the GPU against their fp64 oracle.

Turned rows, per output of a pair (a, b), S = (|a| + |b|) scale, u = 2^-24: sine and cosine
are off by at most u/2 (the phase's rounding, an eighth of a turn held to 2^-25 of itself)
and 2 u (two units in the last place, below 1), and u more times scale; two products and a
sum round by u S each: 5.5 u S in all, bounded by 2^-21 S.  bf16: and half a step, 2^-8 of
the value.

What an append stores is compared exactly: codes as the numbers they stand for, scales,
positions, group ids, mass and counts.
"""
import numpy as np
import pytest

import oracle.cache_ref as cr
import oracle.tree_ref as tr
from learned_group_sparse_focus_gb300 import synth
from test_gpu_cache import NAMES, _cache, _dev, _host, _make, _params, _rows, _same, _type

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fz():
    from learned_group_sparse_focus_gb300 import focus
    return focus


def _freq(dim, theta=10000.0):
    return (theta ** (-2.0 * np.arange(dim // 2) / dim)).astype(np.float32)


def _rot(fz, freq, interleaved=False, scale=1.0):
    return fz.Rotary(_dev(freq), interleaved=interleaved, scale=scale)


def _random_tree(rng, B, T):
    return np.array([[int(rng.integers(-1, t)) if t else -1 for t in range(T)] for _ in range(B)], np.int32)


def _turned(x, at, freq, interleaved, scale, transpose, m):
    """Expected rows of one sequence and their bounds before rounding; NaN behind m."""
    want = np.full(x.shape, np.nan)
    size = np.zeros(x.shape)
    want[:, :m] = tr.rotate(x[:, :m], at[:m], freq, interleaved, scale, transpose)
    h = len(freq)
    lo, hi = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    both = (np.abs(x[..., lo]) + np.abs(x[..., hi])) * scale
    size[..., lo] = size[..., hi] = both
    return want, size * 2.0 ** -21


def _check(got, want, bound, dtype):
    live = ~np.isnan(want)
    err = np.abs(got - want)[live]
    lim = (bound + (np.abs(want) * 2.0 ** -8 if dtype == "bf16" else 0))[live]
    assert (err <= lim).all(), (err - lim).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,H_kv,T,d,dim,interleaved,tree,transpose", [
    (1, 1, 1, 1, 64, 64, False, False, False), (3, 4, 2, 1, 128, 128, True, False, False),
    (2, 12, 3, 33, 64, 32, False, True, False), (2, 8, 8, 64, 128, 64, True, True, True),
    (1, 40, 8, 7, 128, 16, False, True, False), (2, 3, 1, 517, 128, 112, False, False, True),
    (1, 2, 2, 1000, 64, 48, True, False, False), (600, 6, 2, 2, 128, 128, False, True, False)])
def test_rotary_matches_the_oracle(fz, dtype, B, H, H_kv, T, d, dim, interleaved, tree, transpose):
    rng = np.random.default_rng(B * T + dim)
    Q, K = _rows(rng, (B, H, T, d), dtype), _rows(rng, (B, H_kv, T, d), dtype)
    freq, scale = _freq(dim), 1.25
    base = rng.integers(0, [1 << 10, 1 << 30][T % 2], B).astype(np.int32)
    parent = _random_tree(rng, B, T) if tree else None
    n_new = rng.integers(0, T + 1, B).astype(np.int32)
    n_new[0] = T
    p, dt = _params(fz, B, H // H_kv, H_kv, T, d, 4, 1, 8, dtype), _type(fz, dtype)
    ws, rot = fz.alloc_workspace_tree(p), _rot(fz, freq, interleaved, scale)
    if tree:
        for b in range(B):
            parent[b, n_new[b]:] = 99                     # not read
    q, k = _dev(Q, dt), _dev(K, dt)
    qo, ko = q.clone().fill_(7.0), k.clone().fill_(7.0)
    kw = dict(base=_dev(base), parent=None if parent is None else _dev(parent), n_new=_dev(n_new), transpose=transpose)
    fz.focus_rotary(p, rot, ws, Q=q, K=k, Q_out=qo, K_out=ko, **kw)
    assert fz.focus_check_errors(ws) == 0
    for x, out in ((Q, qo), (K, ko)):
        got = out.float().cpu().numpy().astype(np.float64)
        for b in range(B):
            m = int(n_new[b])
            at = base[b] + (tr.depths(parent[b][:m]) if tree else np.arange(m)).astype(np.int64)
            want, bound = _turned(x[b], at, freq, interleaved, scale, transpose, m)
            _check(got[b], want, bound, dtype)
            assert (got[b][:, m:] == 7.0).all()
    # one of the two alone, and in place: the same bits; rows behind n_new stay
    only = q.clone().fill_(7.0)
    fz.focus_rotary(p, rot, ws, Q=q, Q_out=only, **kw)
    assert (only == qo).all()
    fz.focus_rotary(p, rot, ws, K=k, K_out=k, **kw)
    there = (np.arange(T) < n_new[:, None])[:, None, :, None]
    assert (k.float().cpu().numpy() == np.where(there, ko.float().cpu().numpy(), K)).all()


def test_rotary_without_base_at_the_largest_positions_and_frequencies(fz):
    import torch
    rng = np.random.default_rng(4)
    freq = np.float32([1.0, -1.0, 3.1415927, 0.5, 1e-9, 100.0, 0.0, 6.2831855])
    for base in (None, np.int32([2 ** 31 - 3]), np.int32([-5])):
        Q = _rows(rng, (1, 2, 3, 64), "f32")
        p = _params(fz, 1, 2, 1, 3, 64, 4, 1, 8, "f32")
        ws = fz.alloc_workspace_tree(p)
        q = _dev(Q)
        out = torch.empty_like(q)
        fz.focus_rotary(p, _rot(fz, freq), ws, Q=q, Q_out=out, base=None if base is None else _dev(base))
        at = np.arange(3) + (0 if base is None else int(base[0]))
        want, bound = _turned(Q[0], at, freq, False, 1.0, False, 3)
        _check(out[0].cpu().numpy().astype(np.float64), want, bound, "f32")
        assert (out[..., 16:] == q[..., 16:]).all()


def test_rotary_special_values_stay_in_their_pairs(fz):
    import torch
    rng = np.random.default_rng(5)
    for interleaved in (False, True):
        Q = _rows(rng, (1, 1, 4, 64), "f32")
        Q[0, 0, 1, 3], Q[0, 0, 2, 40], Q[0, 0, 3, 60] = np.nan, np.inf, -np.inf    # 60 does not turn
        p = _params(fz, 1, 1, 1, 4, 64, 4, 1, 8, "f32")
        ws, freq, q = fz.alloc_workspace_tree(p), _freq(48), _dev(Q)
        out = torch.empty_like(q)
        fz.focus_rotary(p, _rot(fz, freq, interleaved), ws, Q=q, Q_out=out, base=_dev(np.int32([9])))
        got = out[0, 0].cpu().numpy()
        bad = ~np.isfinite(got)
        pair = lambda e: {e, e ^ 1} if interleaved else {e, e + 24 if e < 24 else e - 24}
        assert set(np.flatnonzero(bad[1])) == pair(3) and set(np.flatnonzero(bad[2])) == pair(40)
        assert set(np.flatnonzero(bad[3])) == {60} and got[3, 60] == -np.inf and not bad[0].any()


def test_rotary_gradient_against_differences(fz):
    """<g, R x> has the gradient R' g: differences of fp32 calls (the map is linear, so a step of
    one has no truncation error)."""
    import torch
    rng = np.random.default_rng(6)
    B, H, T, d = 1, 2, 3, 64
    p = _params(fz, B, 1, H, T, d, 4, 1, 8, "f32")
    ws, rot = fz.alloc_workspace_tree(p), _rot(fz, _freq(32), True, 1.5)
    base, x = _dev(np.int32([41])), _dev(_rows(rng, (B, H, T, d), "f32", 0))
    g = _dev(_rows(rng, (B, H, T, d), "f32", 0))
    grad, y0 = torch.empty_like(x), torch.empty_like(x)
    fz.focus_rotary(p, rot, ws, Q=g, Q_out=grad, base=base, transpose=True)
    fz.focus_rotary(p, rot, ws, Q=x, Q_out=y0, base=base)
    for e in rng.integers(0, x.numel(), 40):
        x1, y1 = x.clone(), torch.empty_like(x)
        x1.view(-1)[e] += 1
        fz.focus_rotary(p, rot, ws, Q=x1, Q_out=y1, base=base)
        diff = ((y1.double() - y0.double()) * g.double()).sum().item()
        # both outputs of the pair, each off by 2^-21 S twice (S of the pair grows by 1.5), times |g|
        size = 1.5 * (x1.abs().max().item() * 2 + 1)
        assert abs(diff - grad.view(-1)[e].item()) <= 8 * 2.0 ** -21 * size * g.abs().max().item()


def test_rotary_flags_bad_parents_and_counts(fz):
    import torch
    rng = np.random.default_rng(7)
    B, T, d = 3, 5, 64
    Q = _rows(rng, (B, 1, T, d), "f32")
    p = _params(fz, B, 1, 1, T, d, 4, 1, 8, "f32")
    ws, rot, q = fz.alloc_workspace_tree(p), _rot(fz, _freq(64)), _dev(Q)
    parent = np.int32([[-1, 0, 2, 1, 7], [-5, 0, 0, 0, 0], [-1, 0, 1, 2, 3]])   # 2 -> 2, 4 -> 7, 0 -> -5
    out = torch.empty_like(q)
    fz.focus_rotary(p, rot, ws, Q=q, Q_out=out, parent=_dev(parent))
    assert fz.focus_check_errors(ws) == 8 and fz.focus_check_errors(ws) == 0
    clean = np.int32([[-1, 0, -1, 1, -1], [-1, 0, 0, 0, 0], [-1, 0, 1, 2, 3]])
    want = torch.empty_like(q)
    fz.focus_rotary(p, rot, ws, Q=q, Q_out=want, parent=_dev(clean))
    assert fz.focus_check_errors(ws) == 0 and (out == want).all()
    fz.focus_rotary(p, rot, ws, Q=q, Q_out=out, n_new=_dev(np.int32([9, 2, 3])))
    assert fz.focus_check_errors(ws) == 7


# ----------------------------------------------------------------- append ---

def _append_case(fz, seed, lens, H, H_kv, T, d, dim, A, dtype, interleaved, pad, first=0, path=False):
    rng = np.random.default_rng(seed)
    B, K = len(lens), 5
    c = _make(seed, B, H_kv, d, lens, K, A, dtype, room=T)
    c["next"] += first
    Q = _rows(rng, (B, H, T, d), dtype)
    Kn, Vn = _rows(rng, (B, H_kv, T, d), dtype), _rows(rng, (B, H_kv, T, d), dtype, 2.5)
    gid = rng.integers(0, K, (B, A, T)).astype(np.int32)
    n_new = rng.integers(0, T + 1, B).astype(np.int32) if pad else None
    rows = None
    if path:
        rows = np.stack([rng.permutation(T) for _ in range(B)]).astype(np.int32)
        if pad:
            for b in range(B):
                rows[b, :n_new[b]].sort()
                rows[b, n_new[b]:] = -9                   # not read
    return rng, c, Q, Kn, Vn, gid, n_new, rows


def _oracle_append(c, Kn, Vn, gid, n_new, rows, freq, interleaved, scale):
    B, _, T, _ = Kn.shape
    K64, V2, g2 = np.zeros(Kn.shape), np.zeros_like(Vn), np.zeros_like(gid)
    for b in range(B):
        m = T if n_new is None else int(n_new[b])
        pick = np.arange(m) if rows is None else rows[b, :m]
        at = int(c["next"][b]) + np.arange(m, dtype=np.int64)
        K64[b, :, :m] = tr.rotate(Kn[b][:, pick], at, freq, interleaved, scale) if freq is not None else Kn[b][:, pick]
        V2[b, :, :m], g2[b, :, :m] = Vn[b][:, pick], gid[b][:, pick]
    return cr.append(c, K64, V2, g2, n_new), K64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,H,H_kv,T,d,dim,A,interleaved,pad,first", [
    ([0], 1, 1, 1, 64, 64, 1, False, False, 0), ([1, 63, 64, 65], 8, 2, 1, 128, 128, 2, False, False, 1 << 20),
    ([0, 5, 130], 4, 4, 64, 128, 64, 1, True, True, 77), ([200, 0], 6, 3, 65, 64, 32, 3, False, False, 0),
    ([7], 2, 2, 300, 64, 16, 1, True, True, 1 << 30), ([64, 1], 4, 2, 129, 128, 128, 1, False, False, 5)])
def test_append_rotary_matches_the_oracle(fz, dtype, lens, H, H_kv, T, d, dim, A, interleaved, pad, first):
    import torch
    rng, c, Q, Kn, Vn, gid, n_new, _ = _append_case(fz, T + d, lens, H, H_kv, T, d, dim, A, dtype, interleaved, pad, first)
    B, freq, scale = len(lens), _freq(dim, 500000.0), 1.0 if T % 2 else 1.1387
    if pad:
        for b in range(B):                                # rows behind n_new are not read
            Kn[b, :, n_new[b]:] = Vn[b, :, n_new[b]:] = Q[b, :, n_new[b]:] = np.nan
            gid[b, :, n_new[b]:] = -7
    want, K64 = _oracle_append(c, Kn, Vn, gid, n_new, None, freq, interleaved, scale)
    p, dt = _params(fz, B, H // H_kv, H_kv, T, d, 5, A, 8, dtype), _type(fz, dtype)
    rot, nn = _rot(fz, freq, interleaved, scale), None if n_new is None else _dev(n_new)
    for in_place in (False, True):
        cache = _cache(fz, c)
        ws = fz.alloc_workspace_cache(p, cache)
        q, k, v, g = _dev(Q, dt), _dev(Kn, dt), _dev(Vn, dt), _dev(gid)
        qo, ko = (q, k) if in_place else (torch.full_like(q, 7.0), torch.full_like(k, 7.0))
        ln, nx = (None, None) if in_place else (torch.full_like(cache.len, -1), torch.full_like(cache.next, -1))
        fz.focus_cache_append_rotary(p, rot, k, v, g, cache, ws, Q=q, Q_out=qo, K_out=ko, n_new=nn, len_out=ln, next_out=nx)
        assert fz.focus_check_errors(ws) == 0
        got = _host(cache)
        if not in_place:
            assert np.array_equal(got["len"], c["len"]) and np.array_equal(got["next"], c["next"])
            got.update(len=ln.cpu().numpy(), next=nx.cpu().numpy())
        _same(got, want)
        for b in range(B):
            m = T if n_new is None else int(n_new[b])
            at = int(c["next"][b]) + np.arange(m, dtype=np.int64)
            for x, out in ((Q, qo), (Kn, ko)):
                y = out[b].float().cpu().numpy().astype(np.float64)
                w, bound = _turned(x[b], at, freq, interleaved, scale, False, m)
                _check(y, w, bound, dtype)
                if not in_place:
                    assert (y[:, m:] == 7.0).all()


@pytest.mark.parametrize("dtype,with_rot", [("bf16", True), ("f32", True), ("bf16", False)])
def test_append_of_picked_rows(fz, dtype, with_rot):
    lens, H_kv, T, d, A = [0, 63, 200, 5], 2, 64, 128, 2
    rng, c, _, Kn, Vn, gid, n_new, rows = _append_case(fz, 9, lens, 4, H_kv, T, d, 128, A, dtype, False, True, 1234, True)
    freq = _freq(128) if with_rot else None
    want, _ = _oracle_append(c, Kn, Vn, gid, n_new, rows, freq, False, 1.0)
    p, dt, cache = _params(fz, 4, 2, H_kv, T, d, 5, A, 8, dtype), _type(fz, dtype), _cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    fz.focus_cache_append_rotary(p, _rot(fz, freq) if with_rot else None, _dev(Kn, dt), _dev(Vn, dt), _dev(gid), cache, ws,
                                 rows=_dev(rows), n_new=_dev(n_new))
    assert fz.focus_check_errors(ws) == 0
    _same(_host(cache), want)


def test_append_without_rotation_is_the_plain_append(fz):
    lens, H_kv, T, d, A = [10, 64], 2, 70, 64, 1
    rng, c, _, Kn, Vn, gid, n_new, _ = _append_case(fz, 10, lens, 4, H_kv, T, d, 64, A, "bf16", False, True)
    p, a, b = _params(fz, 2, 2, H_kv, T, d, 5, A, 8), _cache(fz, c), _cache(fz, c)
    ws, dt = fz.alloc_workspace_cache(p, a), _type(fz, "bf16")
    args = [_dev(Kn, dt), _dev(Vn, dt), _dev(gid)]
    fz.focus_cache_append(p, *args, a, ws, n_new=_dev(n_new))
    fz.focus_cache_append_rotary(p, None, *args, b, ws, n_new=_dev(n_new))
    assert fz.focus_check_errors(ws) == 0
    x, y = _host(a), _host(b)
    assert all(np.array_equal(x[k], y[k], equal_nan=True) for k in NAMES)


def test_append_rotary_is_the_same_token_by_token(fz):
    """Codes do not depend on how tokens come in where no scale grows."""
    rng = np.random.default_rng(11)
    H_kv, d, T = 2, 128, 150
    Kn, Vn = (synth.round_bf16(np.clip(rng.standard_normal((1, H_kv, T, d)), -2.2, 2.2).astype(np.float32)) for _ in range(2))
    Kn[0, :, ::64, 0] = Vn[0, :, ::64, 0] = 3.0            # the first row of each page sets its scale
    Kn[0, :, ::64, 64] = 0.0
    gid = rng.integers(0, 5, (1, 1, T)).astype(np.int32)
    freq = _freq(128)
    out = []
    for step in (T, 1, 7):
        p = _params(fz, 1, 1, H_kv, T, d, 5, 1, 8)
        cache = fz.alloc_cache(p, T)
        ws = fz.alloc_workspace_cache(p, cache)
        for t in range(0, T, step):
            m = min(step, T - t)
            q = _params(fz, 1, 1, H_kv, m, d, 5, 1, 8)
            dt = _type(fz, "bf16")
            fz.focus_cache_append_rotary(q, _rot(fz, freq), _dev(Kn[:, :, t:t + m], dt), _dev(Vn[:, :, t:t + m], dt),
                                         _dev(gid[:, :, t:t + m]), cache, ws)
        assert fz.focus_check_errors(ws) == 0
        out.append(cache)
    for c in out[1:]:
        for name in ("k", "v", "k_scale", "v_scale", "pos", "gid", "len", "next"):
            assert (getattr(c, name) == getattr(out[0], name)).all(), name


def test_append_rotary_near_rounding_borders(fz):
    """Rows built so that many turned values lie within 2^-24 of a border of e4m3 or of a page's
    scale: stored as 64-bit arithmetic has them."""
    rng = np.random.default_rng(12)
    H_kv, d, T = 4, 64, 192
    freq = np.float32([0.0] * 16 + [np.pi / 4, 0.3] + [1e-3] * 14)      # the first pairs never turn
    x = rng.choice([9, 11, 13, 15, 17, 19, 27, 29], (1, H_kv, T, d)).astype(np.float32) / 16   # halves between codes, and codes
    x[..., :16] *= 1 + rng.choice([-1, 0, 1], (1, H_kv, T, 16)).astype(np.float32) * 2.0 ** -22
    for page, top in enumerate((3.5, 3.5 * (1 + 2.0 ** -23), 3.5 * (1 - 2.0 ** -24))):
        x[:, :, page * 64, 0] = top
    # a page whose largest value is turned onto the border: sqrt(2) 3.5 / 2 in both halves at an eighth of a turn
    x[:, 1, 64:128, 16] = x[:, 1, 64:128, 48] = np.float32(3.5 / np.sqrt(2.0))
    gid = np.zeros((1, 1, T), np.int32)
    V = _rows(rng, (1, H_kv, T, d), "f32")
    p = _params(fz, 1, 1, H_kv, T, d, 5, 1, 8, "f32")
    for scale in (1.0, 1.0 + 2.0 ** -20):
        c = cr.empty(1, H_kv, d, 5, 4, 3)
        want, _ = _oracle_append(c, x, V, gid, None, None, freq, False, scale)
        cache = _cache(fz, c)
        ws = fz.alloc_workspace_cache(p, cache)
        fz.focus_cache_append_rotary(p, _rot(fz, freq, False, scale), _dev(x), _dev(V), _dev(gid), cache, ws)
        assert fz.focus_check_errors(ws) == 0
        _same(_host(cache), want)


def test_append_rotary_special_values(fz):
    rng = np.random.default_rng(13)
    H_kv, d, T = 2, 64, 10
    for dtype in ("bf16", "f32"):
        Kn, Vn = _rows(rng, (1, H_kv, T, d), dtype), _rows(rng, (1, H_kv, T, d), dtype)
        Kn[0, 0, 2, 5], Kn[0, 0, 3, 40], Kn[0, 1, 4, 60] = np.nan, np.inf, -np.inf     # 60 does not turn
        Kn[0, 1, 5] = 0.0
        Vn[0, 0, 6, 1], Vn[0, 1, 7, 2] = np.inf, np.nan
        gid = np.zeros((1, 1, T), np.int32)
        freq = _freq(48)
        c = cr.empty(1, H_kv, d, 3, 2, 4)
        with np.errstate(invalid="ignore"):
            want, K64 = _oracle_append(c, Kn, Vn, gid, None, None, freq, False, 1.0)
        cache = _cache(fz, c)
        p = _params(fz, 1, 1, H_kv, T, d, 5, 1, 8, dtype)
        ws = fz.alloc_workspace_cache(p, cache)
        dt = _type(fz, dtype)
        fz.focus_cache_append_rotary(p, _rot(fz, freq), _dev(Kn, dt), _dev(Vn, dt), _dev(gid), cache, ws)
        assert fz.focus_check_errors(ws) == 0
        _same(_host(cache), want)


def test_append_rotary_errors_are_flagged_and_contained(fz):
    import torch
    lens, H_kv, T, d = [60, 100, 3], 2, 10, 64
    rng, c, Q, Kn, Vn, gid, _, _ = _append_case(fz, 14, lens, 4, H_kv, T, d, 64, 1, "bf16", False, False)
    mp = c["table"].shape[1]
    c["len"][1] = mp * 64 - 4                              # does not fit
    c["table"][2, 0] = 1 << 20                             # not a page
    gid[0, 0, 3] = 99                                      # not a group
    freq = _freq(64)
    keep = cr.copy(c)
    ok = cr.copy(c)
    ok["table"][2, 0] = c["table"][0, -1] if c["table"][0, -1] >= 0 else 0
    p, dt, cache = _params(fz, 3, 2, H_kv, T, d, 5, 1, 8), _type(fz, "bf16"), _cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    q, k = _dev(Q, dt), _dev(Kn, dt)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    fz.focus_cache_append_rotary(p, _rot(fz, freq), k, _dev(Vn, dt), _dev(gid), cache, ws, Q=q, Q_out=qo, K_out=ko)
    assert fz.focus_check_errors(ws) == 6                  # the group id is reported first
    got = _host(cache)
    assert list(got["len"][:, 0]) == [70, mp * 64 - 4, 13] and list(got["next"]) == [keep["next"][0] + T, keep["next"][1], keep["next"][2] + T]
    assert (qo[1] == 7.0).all() and (ko[1] == 7.0).all() and not (qo[0] == 7.0).any()
    page, row = cr.slots(got, 0, 0)
    assert got["gid"][page[63], 0, row[63]] == 4           # clamped
    used = set(got["table"][0, :2])
    for g in range(c["k"].shape[0]):                       # nothing but sequence 0's pages changed
        if g not in used:
            assert all(np.array_equal(got[n][g], keep[n][g], equal_nan=True) for n in ("k", "v", "k_scale", "pos", "gid", "mass"))
    # rows outside the drafted tokens
    cache = _cache(fz, keep)
    rows = np.tile(np.arange(T, dtype=np.int32), (3, 1))
    rows[0, 2], rows[0, 3] = -4, T
    gid[0, 0, 3] = 1
    fz.focus_cache_append_rotary(p, _rot(fz, freq), k, _dev(Vn, dt), _dev(gid), cache, ws, rows=_dev(rows))
    assert fz.focus_check_errors(ws) in (7, 8)
    n_new = _dev(np.int32([T, 0, 0]))
    cache = _cache(fz, keep)
    fz.focus_cache_append_rotary(p, _rot(fz, freq), k, _dev(Vn, dt), _dev(gid), cache, ws, rows=_dev(rows), n_new=n_new)
    assert fz.focus_check_errors(ws) == 8


# ----------------------------------------------------------------- accept ---

@pytest.mark.parametrize("B,T,V", [(1, 1, 2), (1, 16, 2), (5, 33, 3), (130, 64, 2), (513, 64, 4), (7, 64, 1)])
@pytest.mark.parametrize("pad", [False, True])
def test_accept_matches_the_oracle(fz, B, T, V, pad):
    import torch
    rng = np.random.default_rng(B + T)
    parent = _random_tree(rng, B, T)
    if T == 64 and V == 1:
        parent = np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))     # a chain that is accepted whole
    token, target = (rng.integers(0, V, (B, T)).astype(np.int32) for _ in range(2))
    prev = rng.integers(0, V, B).astype(np.int32)
    n_new = rng.integers(0, T + 1, B).astype(np.int32) if pad else None
    paths, last = tr.accept(token, target, prev, parent, n_new)
    if pad:
        for b in range(B):
            parent[b, n_new[b]:] = 1000                    # not read
    p = fz.make_params(B, 1, 1, T, 64, 64, 64, 4, 1, 8)
    ws = fz.alloc_workspace_tree(p)
    rows = torch.full((B, T), -3, dtype=torch.int32, device="cuda")
    count, pv = torch.full((B,), -3, dtype=torch.int32, device="cuda"), _dev(prev)
    nn = None if n_new is None else _dev(n_new)
    fz.focus_tree_accept(p, _dev(token), _dev(target), pv, _dev(parent), rows, count, pv, ws, n_new=nn)    # last in prev's place
    assert fz.focus_check_errors(ws) == 0
    got = rows.cpu().numpy()
    assert list(count.cpu().numpy()) == [len(x) for x in paths] and np.array_equal(pv.cpu().numpy(), last)
    for b, path in enumerate(paths):
        assert list(got[b, :len(path)]) == path and (got[b, len(path):] == -3).all()


def test_accept_flags_bad_parents_and_counts(fz):
    import torch
    p = fz.make_params(2, 1, 1, 4, 64, 64, 64, 4, 1, 8)
    ws = fz.alloc_workspace_tree(p)
    z = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    one, rows, count, last = z[:, 0].contiguous(), z.clone(), z[:, 0].contiguous(), z[:, 0].contiguous()
    fz.focus_tree_accept(p, z, z, one, _dev(np.int32([[-1, 0, 1, 3], [-1, 0, 1, 2]])), rows, count, last, ws)
    assert fz.focus_check_errors(ws) == 8 and list(count.cpu()) == [3, 4]       # node 3 counts as one below the root
    fz.focus_tree_accept(p, z, z, one, _dev(np.int32([[-1, 0, 1, 2]] * 2)), rows, count, last, ws, n_new=_dev(np.int32([5, -1])))
    assert fz.focus_check_errors(ws) == 7 and list(count.cpu()) == [4, 0]
