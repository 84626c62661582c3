"""The paged 8-bit key/value cache on the GPU against its fp64 oracle.

Append and eviction are compared exactly: codes as the numbers they stand for,
scales, positions, group ids, mass and counts; rows that no call may touch have
to come back as they were.

Attention bounds, per output, from the arithmetic (u = 2^-24):
  logit     |ds| <= (d + 8) 2 u D, D = scale * sum |q||k| of the row's worst key
            (exact products, d sums in fp32 that may truncate, three scalings);
  weight    relative error r = 2 ds + kept 2 u + 2^-20 (logits of the weight and
            of its sum, the sum's roundings, exp2 and the join's factors);
  lse       ds + kept 2 u + 2^-22 (1 + |lse|);
  O         half a step of the output type, and (r + w) sum P|v| for the weights,
            w = 2^-11 (one f16 rounding) for bf16 tensors and 2^-22 for fp32; and
            kept 2^-26 M for the weights' floor: weights p = 2^(s + e) times page
            exponents e multiply codes of at most 448 and are cut off at 2^-16 where
            the largest is 2^10 or more; that one, in a page of exponent e0, adds at
            least 2^10 2^-e0 to the sum, so the cut-offs move O by at most
            kept 2^-16 448 / (2^10 2^-e0) = kept 2^-26 M, M = 448 2^e0;
  mass      r times what was added, and a step of the total.
"""
import numpy as np
import pytest

import oracle.cache_ref as cr
from learned_group_sparse_focus_gb300 import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NAMES = ("k", "v", "k_scale", "v_scale", "pos", "gid", "mass", "table", "len", "next")


@pytest.fixture(scope="module")
def fz():
    from learned_group_sparse_focus_gb300 import focus
    return focus


def _dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def _cache(fz, c):
    return fz.Cache(**{k: _dev(c[k]) for k in NAMES})


def _type(fz, dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _host(cache):
    return {k: getattr(cache, k).cpu().numpy() for k in NAMES}


def _same(got, want):
    """Equal caches, every slot of the pool and the unused ones too."""
    for k in ("pos", "gid", "table", "len", "next"):
        assert np.array_equal(got[k], want[k]), k
    for k in ("k_scale", "v_scale", "mass"):
        assert np.array_equal(got[k], want[k].astype(np.float32), equal_nan=True), k
    for k in ("k", "v"):
        a, b = cr.VALUES[got[k]], cr.VALUES[want[k]]
        assert np.array_equal(a, b, equal_nan=True), (k, np.argwhere(~((a == b) | (np.isnan(a) & np.isnan(b))))[:5])


def _rows(rng, shape, dtype, spread=1.0):
    x = (rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))).astype(np.float32)
    return synth.round_bf16(x) if dtype == "bf16" else x


def _params(fz, B, G, H_kv, T, d, K, A, w, dtype="bf16"):
    return fz.make_params(B, G * H_kv, H_kv, T, d, 64, 64, K, A, w, dtype=dtype)


def _make(seed, B, H_kv, d, lens, K, A, dtype="bf16", spare=3, room=0):
    """A cache filled with `lens` tokens a sequence by the oracle."""
    rng = np.random.default_rng(seed)
    T = max(max(lens), 1)
    mp = -(-(T + room) // 64) + 1
    c = cr.empty(B, H_kv, d, B * mp + spare, mp, seed)
    gid = rng.integers(0, K, (B, A, T)).astype(np.int32)
    c = cr.append(c, _rows(rng, (B, H_kv, T, d), dtype), _rows(rng, (B, H_kv, T, d), dtype), gid, np.array(lens))
    live = np.isfinite(c["mass"])
    c["mass"][live] = np.exp(2 * rng.standard_normal(live.sum())).astype(np.float32) * (rng.random(live.sum()) > 0.4)
    return c


# ----------------------------------------------------------------- append ---

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,lens,T,A,pad", [
    (64, [0, 0], 1, 1, False), (64, [1, 63, 64, 65], 1, 1, False), (128, [0, 5, 63, 130], 64, 2, True),
    (128, [200, 0, 64], 65, 1, False), (64, [7], 300, 2, True), (128, [64, 1], 129, 1, True)])
def test_append_matches_the_oracle(fz, dtype, d, lens, T, A, pad):
    import torch
    rng = np.random.default_rng(len(lens) * T + d)
    B, H_kv, K = len(lens), 2, 5
    c = _make(T + d, B, H_kv, d, lens, K, A, dtype, room=T)
    Kn, Vn = _rows(rng, (B, H_kv, T, d), dtype), _rows(rng, (B, H_kv, T, d), dtype, 2.5)
    gid = rng.integers(0, K, (B, A, T)).astype(np.int32)
    n_new = None
    if pad:
        n_new = rng.integers(0, T + 1, B).astype(np.int32)
        n_new[0] = 0
        for b in range(B):                                # rows behind n_new are not read
            Kn[b, :, n_new[b]:] = Vn[b, :, n_new[b]:] = np.nan
            gid[b, :, n_new[b]:] = -7
    want = cr.append(c, Kn, Vn, gid, n_new)
    p = _params(fz, B, 2, H_kv, T, d, K, A, 8, dtype)
    dt = _type(fz, dtype)
    a = [_dev(Kn, dt), _dev(Vn, dt), _dev(gid)]
    nn = None if n_new is None else _dev(n_new)
    # counts to other arrays: the cache's own stay
    cache = _cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    ln, nx = torch.full_like(cache.len, -1), torch.full_like(cache.next, -1)
    fz.focus_cache_append(p, *a, cache, ws, n_new=nn, len_out=ln, next_out=nx)
    assert fz.focus_check_errors(ws) == 0
    assert np.array_equal(ln.cpu().numpy(), want["len"]) and np.array_equal(nx.cpu().numpy(), want["next"])
    _same(_host(cache), {**want, "len": c["len"], "next": c["next"]})
    # again, in place: the same contents
    fz.focus_cache_append(p, *a, cache, ws, n_new=nn)
    assert fz.focus_check_errors(ws) == 0
    _same(_host(cache), want)


def test_append_special_values_and_growing_scales(fz):
    d, H_kv = 64, 2
    rng = np.random.default_rng(0)
    x = _rows(rng, (1, H_kv, 12, d), "bf16")
    x[:, :, 1] *= 2.0 ** 20                               # the page's scale grows, older rows round again
    x[:, :, 2, :4] = [np.inf, -np.inf, np.nan, -0.0]
    x[:, :, 3] = 0.0
    x[:, :, 4] *= 2.0 ** -60
    x[:, :, 5, 0] = 3.3e38
    x[:, :, 6] = np.nan
    x[0, 0, 7] = 448.0
    x = synth.round_bf16(x)
    c = cr.empty(1, H_kv, d, 3, 2, 4)
    p = _params(fz, 1, 1, H_kv, 1, d, 4, 1, 8)
    cache = _cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    import torch
    for t in range(12):
        one, gid = x[:, :, t:t + 1], np.full((1, 1, 1), t % 4, np.int32)
        flip = np.ascontiguousarray(one[..., ::-1])
        c = cr.append(c, one, flip, gid)
        fz.focus_cache_append(p, _dev(one, torch.bfloat16), _dev(flip, torch.bfloat16), _dev(gid), cache, ws)
        _same(_host(cache), c)
    assert fz.focus_check_errors(ws) == 0


def test_append_without_mass_and_shared_pool(fz):
    """Two caches with disjoint tables over one pool, no mass array."""
    import torch
    d, H_kv, T, K = 64, 2, 70, 4
    rng = np.random.default_rng(2)
    c = cr.empty(1, H_kv, d, 6, 2, 4)
    other = cr.copy(c)
    other["table"] = np.array([[p for p in range(6) if p not in c["table"]][:2]], np.int32)
    pool = {k: _dev(c[k]) for k in NAMES[:6]}
    p = _params(fz, 1, 1, H_kv, T, d, K, 1, 8)
    want = c
    for who in (c, other):
        x = _rows(rng, (1, H_kv, T, d), "bf16")
        gid = rng.integers(0, K, (1, 1, T)).astype(np.int32)
        cache = fz.Cache(**pool, mass=None, **{k: _dev(who[k]) for k in NAMES[7:]})
        ws = fz.alloc_workspace_cache(p, cache)
        assert ws.numel() == 256
        fz.focus_cache_append(p, _dev(x, torch.bfloat16), _dev(x, torch.bfloat16), _dev(gid), cache, ws)
        assert fz.focus_check_errors(ws) == 0
        want = cr.append({**want, **{k: who[k] for k in NAMES[7:]}}, x, x, gid)
    got = {k: v.cpu().numpy() for k, v in pool.items()}
    _same({**want, **got}, want)


def test_append_errors_are_flagged_and_contained(fz):
    import torch
    d, H_kv, K = 64, 2, 4
    c = _make(3, 3, H_kv, d, [100, 120, 3], K, 1)        # three pages a sequence
    c["len"][1, 1] = 150                                 # one head of sequence 1 has no room for 50 more
    T = 50
    rng = np.random.default_rng(5)
    x = _rows(rng, (3, H_kv, T, d), "bf16")
    gid = rng.integers(0, K, (3, 1, T)).astype(np.int32)
    p = _params(fz, 3, 1, H_kv, T, d, K, 1, 8)
    want = cr.append(c, x, x, gid)
    assert np.array_equal(want["len"][1], c["len"][1])
    cache = _cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    a = _dev(x, torch.bfloat16)
    fz.focus_cache_append(p, a, a, _dev(gid), cache, ws)
    assert fz.focus_check_errors(ws) == 7
    assert fz.focus_check_errors(ws) == 0
    _same(_host(cache), want)
    # a group id outside [0, K) is clamped
    bad = gid.copy()
    bad[0, 0, 3], bad[2, 0, 4] = -1, K
    fixed = np.clip(bad, 0, K - 1)
    cache = _cache(fz, c)
    fz.focus_cache_append(p, a, a, _dev(bad), cache, ws)
    assert fz.focus_check_errors(ws) == 6               # reported before the overflow of sequence 1
    _same(_host(cache), cr.append(c, x, x, fixed))
    # page ids outside the pool: their rows are dropped, the others stored
    for page in (-1, 1 << 30, int(c["k"].shape[0])):
        broken = cr.copy(c)
        broken["table"][0, 2] = page
        cache = _cache(fz, broken)
        fz.focus_cache_append(p, a, a, _dev(gid), cache, ws)
        assert fz.focus_check_errors(ws) == 7
        got, ok = _host(cache), c["table"][0][:2]
        for k in ("k", "pos", "gid"):
            assert np.array_equal(got[k][ok], want[k][ok]), k
        skipped = c["table"][0][2]
        assert np.array_equal(got["k"][skipped], c["k"][skipped])


# -------------------------------------------------------------- attention ---

def _bounds(ref, d, dtype):
    """(logit, weight, O) bounds of the module's docstring."""
    ds = (d + 8) * 2 * U * ref["dot"]
    r = 2 * ds + ref["kept"] * 2 * U + 2.0 ** -20
    step, wt = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -22)
    return ds, r, step * np.abs(ref["O"]) + (r[..., None] + wt) * ref["pv"] * (1 + step) + \
        (ref["kept"] * 2.0 ** -26 * ref["page"])[..., None] + 1e-38


def _o_within(O, ref, d, dtype, there=...):
    over = np.abs(O.float().cpu().numpy().astype(np.float64) - ref["O"]) - _bounds(ref, d, dtype)[2]
    assert over[there].max(initial=0) <= 0, over[there].max()


def _check_attention(fz, c, Q, gid, K, w, dtype, n_new=None, accumulate=True, want_lse=True):
    import torch
    B, H, T, d = Q.shape
    H_kv, A = c["k"].shape[1], gid.shape[1]
    p = fz.make_params(B, H, H_kv, T, d, 64, 64, K, A, w, dtype=dtype)
    cache = _cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    dt = _type(fz, dtype)
    q = _dev(Q, dt)
    Q = q.float().cpu().numpy()                          # what the device holds
    O = torch.full((B, H, T, d), 7.0, dtype=dt, device="cuda")
    lse = torch.full((B, H, T), 7.0, device="cuda") if want_lse else None
    nn = None if n_new is None else _dev(n_new)
    fz.focus_cache_attention_fwd(p, q, _dev(gid), cache, O, lse, ws, n_new=nn, accumulate=accumulate)
    assert fz.focus_check_errors(ws) == 0
    ref = cr.attention(c, Q, gid, w, p.scale, n_new)
    got = O.float().cpu().numpy().astype(np.float64)
    behind = np.isnan(ref["lse"])
    assert (got[behind] == 7.0).all()
    ds, r, tol = _bounds(ref, d, dtype)
    err = np.abs(got - ref["O"])[~behind] - tol[~behind]
    assert np.isfinite(got).all() and err.max(initial=0) <= 0, ("O", err.max())
    if want_lse:
        lg = lse.cpu().numpy().astype(np.float64)
        assert (lg[behind] == 7.0).all()
        none = np.isneginf(ref["lse"])
        assert (lg[none] == -np.inf).all() and (got[none] == 0).all()
        there = ~behind & ~none
        bound = (ds + ref["kept"] * 2 * U + 2.0 ** -22 * (1 + np.abs(np.where(there, ref["lse"], 0))))[there]
        assert (np.abs(lg[there] - ref["lse"][there]) <= bound).all(), "lse"
    after = _host(cache)
    if accumulate:
        live = np.zeros(c["mass"].shape, bool)
        for b in range(B):
            for h in range(H_kv):
                pg, row = cr.slots(c, b, h)
                live[pg, h, row] = True
        m0, m1 = c["mass"].astype(np.float64), after["mass"].astype(np.float64)
        assert np.array_equal(after["mass"][~live], c["mass"][~live], equal_nan=True)
        bound = r.max() * ref["got"][live] + 2.0 ** -23 * np.abs(m1[live]) + 1e-30
        off = np.abs(m1[live] - m0[live] - ref["got"][live]) - bound
        assert off.max(initial=0) <= 0, ("mass", off.max())
        after["mass"] = c["mass"]
    _same(after, c)
    return O


CASES = [
    # G, H_kv, d, lens, T, K, A, w
    (1, 1, 64, [1], 1, 1, 1, 1),
    (1, 2, 64, [1, 2, 63, 64, 65], 1, 3, 1, 4),
    (4, 2, 128, [500, 1, 129], 1, 4, 1, 32),
    (8, 1, 128, [1000], 1, 8, 1, 64),
    (2, 3, 64, [777, 300], 3, 5, 3, 33),
    (4, 2, 128, [400, 650], 4, 6, 2, 50),
    (3, 2, 64, [200, 90], 7, 2, 1, 0),
    (16, 1, 128, [350], 2, 3, 1, 20),
    (1, 4, 128, [300], 64, 4, 1, 30),
    (5, 1, 64, [130, 64], 13, 500, 1, 1000),
    # more than 8, 16, 32 and 64 rows a head, tokens that straddle blocks of rows, more
    # groups than the table holds, an empty sequence, windows of one and of everything
    (12, 2, 128, [600, 0, 70], 1, 3, 1, 40),
    (24, 1, 128, [500], 1, 2, 1, 1),
    (40, 1, 128, [300, 64], 2, 3, 1, 500),
    (3, 2, 128, [700, 65], 5, 4, 2, 30),
    (8, 1, 128, [900, 1], 4, 6, 1, 0),
    (6, 1, 128, [400], 13, 3, 1, 25),
    (2, 1, 128, [333], 31, 1500, 1, 10),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,H_kv,d,lens,T,K,A,w", CASES)
def test_attention_matches_the_oracle(fz, dtype, G, H_kv, d, lens, T, K, A, w):
    rng = np.random.default_rng(G * 1000 + T * 10 + d)
    B = len(lens)
    c = _make(T + G, B, H_kv, d, lens, K, A, dtype)
    Q = _rows(rng, (B, G * H_kv, T, d), dtype, 0.3)
    gid = rng.integers(0, K, (B, A, T)).astype(np.int32)
    _check_attention(fz, c, Q, gid, K, w, dtype)
    n_new = rng.integers(0, T + 1, B).astype(np.int32)
    n_new[-1] = T
    _check_attention(fz, c, Q, gid, K, w, dtype, n_new=n_new, accumulate=bool(T % 2), want_lse=bool(G % 2))


@pytest.mark.parametrize("G,d,T,K,dtype", [(2, 64, 1, 1, "bf16"), (4, 128, 1, 1, "bf16"), (1, 128, 3, 2, "f32"),
                                           (12, 128, 1, 1, "bf16"), (8, 128, 4, 2, "bf16"), (1, 128, 64, 3, "bf16")])
def test_attention_over_more_slots_than_the_lists_hold(fz, G, d, T, K, dtype):
    """So many kept slots that the kernels' lists wrap around and the weights' pass scans
    again: two sequences, one of 30,000 slots, random codes."""
    rng = np.random.default_rng(d + T)
    n = [30000, 9001]
    mp = -(-n[0] // 64)
    c = cr.empty(2, 1, d, 2 * mp, mp, 5)
    c["k"] = (c["k"] & 0xbf).astype(np.uint8)                # below 2 in magnitude, no NaN
    c["v"] &= 0xbf
    c["k_scale"][:] = 2.0 ** rng.integers(-3, 1, c["k_scale"].shape)
    c["v_scale"][:] = 2.0 ** rng.integers(-5, 6, c["v_scale"].shape)
    for b in range(2):
        c["pos"][c["table"][b], 0] = np.arange(mp * 64).reshape(mp, 64)
    c["gid"][:] = rng.integers(0, K, c["gid"].shape)
    c["mass"][:] = 0.0
    c["len"][:, 0], c["next"][:] = n, n
    Q = _rows(rng, (2, G, T, d), dtype, 0.2)
    _check_attention(fz, c, Q, rng.integers(0, K, (2, 1, T)).astype(np.int32), K, 300, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_after_heads_were_evicted_differently(fz, dtype):
    """Heads of different lengths, one empty, gaps in the positions."""
    c = _make(21, 2, 3, 64, [700, 420], 4, 1, dtype)
    dst = cr.empty(2, 3, 64, 12, 5, 8)
    c = cr.evict(c, dst, 290, 40)
    c["len"][0, 1], c["len"][1, 2], c["len"][1, 0] = 0, 65, 1
    rng = np.random.default_rng(3)
    Q = _rows(rng, (2, 6, 3, 64), dtype, 0.3)
    gid = rng.integers(0, 4, (2, 1, 3)).astype(np.int32)
    _check_attention(fz, c, Q, gid, 4, 30, dtype)
    _check_attention(fz, c, Q, np.full((2, 1, 3), 9, np.int32), 10, 1, dtype)    # a group that no slot has


def test_attention_with_no_cached_token_and_early_positions(fz):
    c = cr.empty(2, 2, 64, 3, 1, 1)
    Q = np.ones((2, 4, 5, 64), np.float32)
    _check_attention(fz, c, Q, np.zeros((2, 1, 5), np.int32), 3, 8, "bf16")      # positions -5 .. -1, no slots
    c = _make(2, 2, 2, 64, [2, 70], 3, 1)
    _check_attention(fz, c, Q, np.zeros((2, 1, 5), np.int32), 3, 8, "bf16")      # three of five before the first


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_over_pages_of_very_different_scales(fz, dtype):
    """Value pages 2^-50 to 2^70 apart from each other, large logits, tiny and huge queries."""
    rng = np.random.default_rng(8)
    d, H_kv, n = 128, 2, 640
    c = cr.empty(1, H_kv, d, 12, 11, 3)
    gid = rng.integers(0, 3, (1, 1, n)).astype(np.int32)
    x, v = _rows(rng, (1, H_kv, n, d), dtype, 0.0), _rows(rng, (1, H_kv, n, d), dtype, 0.0)
    for j in range(10):
        v[:, :, 64 * j:64 * j + 64] *= np.float32(2.0 ** rng.integers(-50, 71))
        x[:, :, 64 * j:64 * j + 64] *= np.float32(2.0 ** rng.integers(-6, 2))
    c = cr.append(c, x, v, gid)
    c["mass"][:] = 0
    Q = _rows(rng, (1, 8, 2, d), dtype, 0.0)
    for h, f in enumerate((1.0, 2.0 ** -100, 6.0, 0.0, 2.0 ** -20, 2.0, 3.0, 1.0)):
        Q[:, h] *= np.float32(f)
    _check_attention(fz, c, Q, gid[:, :, -2:].copy(), 3, 100, dtype)


@pytest.mark.parametrize("H,d", [(4, 64), (4, 128), (8, 128)])
def test_nan_and_infinite_queries_stay_in_their_rows(fz, H, d):
    import torch
    c = _make(4, 1, 1, d, [300], 2, 1)
    Q = _rows(np.random.default_rng(1), (1, H, 2, d), "bf16", 0.2)
    gid = np.array([[[0, 1]]], np.int32)
    p = fz.make_params(1, H, 1, 2, d, 64, 64, 2, 1, 20)
    cache = _cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    outs = []
    for bad in (False, True):
        q = Q.copy()
        if bad:
            q[0, 1, 0, 3], q[0, 2, 1, 5] = np.nan, np.inf
        O = torch.zeros((1, H, 2, d), dtype=torch.bfloat16, device="cuda")
        fz.focus_cache_attention_fwd(p, _dev(q, torch.bfloat16), _dev(gid), cache, O, None, ws)
        outs.append(O.float().cpu().numpy())
    same = np.ones((H, 2), bool)
    same[1, 0] = same[2, 1] = False
    assert np.array_equal(outs[0][0][same], outs[1][0][same])
    assert np.isnan(outs[1][0, 1, 0]).all() and np.isnan(outs[1][0, 2, 1]).all()


@pytest.mark.parametrize("H,d", [(2, 64), (2, 128), (6, 128), (20, 128), (32, 128)])
def test_nan_key_reaches_only_the_rows_that_keep_it(fz, H, d):
    import torch
    c = _make(6, 1, 1, d, [200], 2, 1)
    page, row = cr.slots(c, 0, 0)
    c["gid"][page, 0, row] = 0
    c["gid"][page[10], 0, row[10]] = 1
    c["v"][page[10], 0, row[10], 0] = 127
    c["v"][page[150], 0, row[150], d - 1] = 255
    c["gid"][page[150], 0, row[150]] = 1
    Q = _rows(np.random.default_rng(1), (1, H, 2, d), "bf16", 0.2)
    p = fz.make_params(1, H, 1, 2, d, 64, 64, 2, 1, 20)
    cache = _cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    O = torch.zeros((1, H, 2, d), dtype=torch.bfloat16, device="cuda")
    fz.focus_cache_attention_fwd(p, _dev(Q, torch.bfloat16), _dev(np.array([[[0, 1]]], np.int32)), cache, O, None, ws)
    o = O.float().cpu().numpy()[0]
    assert np.isfinite(o[:, 0]).all() and np.isfinite(o[:, 1, 1:-1]).all()
    assert np.isnan(o[:, 1, 0]).all() and np.isnan(o[:, 1, -1]).all()


def test_attention_with_bad_pages_and_lengths(fz):
    """Bad ids and counts are skipped, clamped and flagged; the rest is unharmed."""
    import torch
    c = _make(7, 2, 2, 64, [200, 200], 1, 1)
    c["mass"][:] = 0
    for page, ln in ((-5, None), (1 << 30, None), (None, 1 << 20), (None, -3)):
        broken = cr.copy(c)
        if page is not None:
            broken["table"][0, 1] = page
        if ln is not None:
            broken["len"][0, 1] = ln
        Q = _rows(np.random.default_rng(1), (2, 4, 1, 64), "bf16", 0.2)
        p = fz.make_params(2, 4, 2, 1, 64, 64, 64, 1, 1, 20)
        cache = _cache(fz, broken)
        ws = fz.alloc_workspace_cache(p, cache)
        O = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
        gid = np.zeros((2, 1, 1), np.int32)
        fz.focus_cache_attention_fwd(p, _dev(Q, torch.bfloat16), _dev(gid), cache, O, None, ws, accumulate=True)
        assert fz.focus_check_errors(ws) == 7
        ref = cr.attention({**c, "table": c["table"]}, Q, gid, 20, p.scale)
        _o_within(O, ref, 64, "bf16", there=1)


def test_long_cache_positions_near_the_limit(fz):
    """Positions close to 2^31 and a window longer than the cache."""
    c = _make(9, 1, 1, 64, [150], 2, 1)
    far = (1 << 31) - 1 - 150
    page, row = cr.slots(c, 0, 0)
    c["pos"][page, 0, row] += far
    c["next"] += far
    rng = np.random.default_rng(1)
    Q = _rows(rng, (1, 2, 2, 64), "bf16", 0.2)
    for w in (5, 1 << 30):
        _check_attention(fz, c, Q, np.array([[[0, 1]]], np.int32), 2, w, "bf16")


@pytest.mark.parametrize("H,T", [(4, 1), (8, 4)])
def test_pages_past_four_gigabytes_of_a_pool(fz, H, T):
    """The same calls over the last pages of a 5 GB pool and over a small pool: same bits."""
    import torch
    B, H_kv, d, K, w, n = 2, 2, 128, 3, 20, 700
    p = fz.make_params(B, H, H_kv, n, d, 64, 64, K, 1, w)
    q = fz.make_params(B, H, H_kv, T, d, 64, 64, K, 1, w)
    rng = np.random.default_rng(H)
    bf, mp = torch.bfloat16, -(-(n + T) // 64)
    k, v = (_dev(_rows(rng, (B, H_kv, n, d), "bf16"), bf) for _ in range(2))
    k1, v1 = (_dev(_rows(rng, (B, H_kv, T, d), "bf16"), bf) for _ in range(2))
    Q = _dev(_rows(rng, (B, H, T, d), "bf16", 0.3), bf)
    gid, gid1 = (_dev(rng.integers(0, K, (B, 1, m)).astype(np.int32)) for m in (n, T))
    outs = []
    for pages in (64, 5 * 2 ** 30 // (H_kv * 64 * d)):
        def pool(shape, dtype):
            return torch.zeros((pages, H_kv) + shape, dtype=dtype, device="cuda")

        part = dict(k=pool((64, d), torch.uint8), v=pool((64, d), torch.uint8), k_scale=pool((), torch.float32),
                    v_scale=pool((), torch.float32), pos=pool((64,), torch.int32), gid=pool((64,), torch.int16),
                    mass=pool((64,), torch.float32))

        def cache(last):
            table = torch.arange(last - B * mp, last, dtype=torch.int32, device="cuda").flip(0).reshape(B, mp)
            return fz.Cache(**part, table=table, len=torch.zeros((B, H_kv), dtype=torch.int32, device="cuda"),
                            next=torch.zeros((B,), dtype=torch.int32, device="cuda"))

        src, dst = cache(pages), cache(pages - 30)
        ws = fz.alloc_workspace_cache(p, src)
        fz.focus_cache_append(p, k, v, gid, src, ws)
        fz.focus_cache_append(q, k1, v1, gid1, src, ws)
        O, lse = torch.zeros_like(Q), torch.zeros(Q.shape[:3], device="cuda")
        fz.focus_cache_attention_fwd(q, Q, gid1, src, O, lse, ws, accumulate=True)
        fz.focus_cache_evict(q, 200, 30, src, dst, ws)
        O2 = torch.zeros_like(Q)
        fz.focus_cache_attention_fwd(q, Q, gid1, dst, O2, None, ws)
        assert fz.focus_check_errors(ws) == 0
        tail = {m: x[pages - 60:].cpu() for m, x in part.items()}
        outs.append([O.float().cpu(), lse.cpu(), O2.float().cpu(), src.len.cpu(), dst.len.cpu(), *tail.values()])
        if len(outs) == 2:                               # nothing was written below those pages
            assert not any(part[m][:pages - 60].view(-1)[::7].any() for m in ("k", "v", "k_scale", "pos"))
    assert outs[0][0].abs().max() > 0
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# --------------------------------------------------------------- eviction ---

@pytest.mark.parametrize("H_kv,d,lens,budget,recent,ties", [
    (1, 64, [1], 1, 0, False), (2, 64, [65, 64, 63], 64, 64, False), (2, 128, [1000, 300, 5], 257, 31, False),
    (3, 64, [700, 500], 400, 0, True), (2, 128, [129], 128, 1, True), (1, 128, [2500], 1000, 300, False),
    (2, 64, [90, 64], 3, 2, True)])
def test_eviction_matches_the_oracle(fz, H_kv, d, lens, budget, recent, ties):
    rng = np.random.default_rng(budget)
    B = len(lens)
    c = _make(budget, B, H_kv, d, lens, 4, 1)
    live = np.isfinite(c["mass"])
    if ties:
        c["mass"][live] = rng.integers(0, 3, live.sum())
    c["mass"].flat[np.flatnonzero(live)[3::17]] = np.float32(-0.0)
    c["mass"].flat[np.flatnonzero(live)[5::29]] = np.nan
    c["mass"].flat[np.flatnonzero(live)[7::31]] = np.inf
    c["mass"].flat[np.flatnonzero(live)[9::37]] = -1.5
    pages = -(-budget // 64)
    dst = cr.empty(B, H_kv, d, B * pages + 2, pages, 77)
    want = cr.evict(c, dst, budget, recent)
    p = _params(fz, B, 1, H_kv, 1, d, 4, 1, 8)
    src, to = _cache(fz, c), _cache(fz, dst)
    ws = fz.alloc_workspace_cache(p, src)
    for _ in range(2):                                   # twice: src stays, so does the answer
        fz.focus_cache_evict(p, budget, recent, src, to, ws)
        assert fz.focus_check_errors(ws) == 0
        _same(_host(to), want)
        _same(_host(src), c)


def test_eviction_of_a_long_head(fz):
    """More slots than the blocks of a cluster hold as keys in shared memory."""
    rng = np.random.default_rng(1)
    n, d, budget, recent = 400_000, 64, 1500, 700
    pages = -(-n // 64)
    c = cr.empty(1, 1, d, pages, pages, 5)
    c["k"] &= 0x7e                                       # no NaN codes
    c["v"] &= 0x7e
    c["k_scale"][:] = 2.0 ** rng.integers(-9, 3, (pages, 1))
    c["v_scale"][:] = 0.25
    page = c["table"][0]
    c["pos"][page, 0] = 3 * np.arange(pages * 64, dtype=np.int32).reshape(pages, 64)
    c["mass"][:] = rng.integers(0, 300, c["mass"].shape)     # hundreds of ties at the threshold
    c["len"][:], c["next"][:] = n, 3 * n
    dst = cr.empty(1, 1, d, 30, 24, 6)
    want = cr.evict(c, dst, budget, recent)
    p = _params(fz, 1, 1, 1, 1, d, 4, 1, 8)
    src, to = _cache(fz, c), _cache(fz, dst)
    ws = fz.alloc_workspace_cache(p, src)
    fz.focus_cache_evict(p, budget, recent, src, to, ws)
    assert fz.focus_check_errors(ws) == 0
    _same(_host(to), want)


def test_eviction_within_one_pool_updates_the_counts_in_place(fz):
    c = _make(31, 2, 2, 64, [600, 350], 4, 1, spare=20)
    free = [x for x in range(c["k"].shape[0]) if x not in c["table"]]
    d = {**c, "table": np.array(free[:8], np.int32).reshape(2, 4)}
    want = cr.evict(c, d, 200, 20)
    p = _params(fz, 2, 1, 2, 1, 64, 4, 1, 8)
    src = _cache(fz, c)
    dst = fz.Cache(**{**{k: getattr(src, k) for k in NAMES}, "table": _dev(d["table"])})
    ws = fz.alloc_workspace_cache(p, src)
    fz.focus_cache_evict(p, 200, 20, src, dst, ws)
    assert fz.focus_check_errors(ws) == 0
    _same(_host(dst), want)


# ------------------------------------------------------------ as they run ---

def _decode_inputs(rng, p, steps, dtype):
    for _ in range(steps):
        yield (_rows(rng, (p.B, p.H_kv, p.n, p.d), dtype, 0.3), _rows(rng, (p.B, p.H_kv, p.n, p.d), dtype, 0.3),
               _rows(rng, (p.B, p.H, p.n, p.d), dtype, 0.3), rng.integers(0, p.K, (p.B, p.A, p.n)).astype(np.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_observation_eviction_and_decoding(fz, dtype):
    """A prompt goes into the cache, its last tokens weigh the keys, the cache is cut
    down into fresh pages of the pool, and decoding goes on over what is left."""
    import torch
    rng = np.random.default_rng(17)
    B, G, H_kv, d, K, w, n = 2, 2, 2, 64, 4, 24, 300
    dt = _type(fz, dtype)
    c = cr.empty(B, H_kv, d, 24, 6, 5)
    c["mass"][:] = 0
    free = [x for x in range(24) if x not in c["table"]]
    pool = _cache(fz, c)
    p = _params(fz, B, G, H_kv, n, d, K, 1, w, dtype)
    ws = fz.alloc_workspace_cache(p, pool)
    lens = np.array([300, 211], np.int32)
    k, v, q, gid = next(_decode_inputs(rng, p, 1, dtype))
    fz.focus_cache_append(p, _dev(k, dt), _dev(v, dt), _dev(gid), pool, ws, n_new=_dev(lens))
    c = cr.append(c, k, v, gid, lens)
    _same(_host(pool), c)
    T = 16                                               # the last 16 prompt tokens of each sequence
    po = _params(fz, B, G, H_kv, T, d, K, 1, w, dtype)
    qo = np.stack([q[b, :, lens[b] - T:lens[b]] for b in range(B)])
    go = np.stack([gid[b, :, lens[b] - T:lens[b]] for b in range(B)])
    O = torch.empty((B, G * H_kv, T, d), dtype=dt, device="cuda")
    fz.focus_cache_attention_fwd(po, _dev(qo, dt), _dev(go), pool, O, None, ws, accumulate=True)
    got = _host(pool)["mass"]
    ref = cr.attention(c, qo, go, w, p.scale)
    assert np.abs(got - ref["got"]).max() < 1e-4
    c["mass"] = got.copy()                               # select on the same numbers
    small = fz.Cache(**{**{x: getattr(pool, x) for x in NAMES},
                        "table": _dev(np.array(free[:8], np.int32).reshape(2, 4))})
    fz.focus_cache_evict(p, 128, w, pool, small, ws)
    c = cr.evict(c, {**c, "table": small.table.cpu().numpy()}, 128, w)
    _same(_host(small), c)
    p1 = _params(fz, B, G, H_kv, 1, d, K, 1, w, dtype)
    for k, v, q, gid in _decode_inputs(rng, p1, 5, dtype):
        fz.focus_cache_append(p1, _dev(k, dt), _dev(v, dt), _dev(gid), small, ws)
        c = cr.append(c, k, v, gid)
        mass = _host(small)["mass"]
        assert np.allclose(mass, c["mass"], rtol=1e-5, atol=1e-6)
        c["mass"] = mass
        _same(_host(small), c)
        _check_attention(fz, c, q, gid, K, w, dtype)
        O = torch.empty((B, G * H_kv, 1, d), dtype=dt, device="cuda")
        fz.focus_cache_attention_fwd(p1, _dev(q, dt), _dev(gid), small, O, None, ws, accumulate=True)
        c["mass"] = (c["mass"] + cr.attention(c, q, gid, w, p.scale)["got"]).astype(np.float32)
    assert fz.focus_check_errors(ws) == 0


def test_decode_step_from_hidden_states(fz):
    """run_decode_step: assign -> append -> attention, padded rows left 0, against the
    oracle with the group ids that the step returned."""
    import torch
    rng = np.random.default_rng(23)
    B, G, H_kv, d, K, w, D, T = 3, 2, 2, 64, 6, 12, 96, 3
    c = _make(12, B, H_kv, d, [100, 30, 64], K, 1, room=20)
    p = fz.make_params(B, G * H_kv, H_kv, T, d, D, 32, K, 1, w)
    cache = _cache(fz, c)
    ws, wc = fz.alloc_workspace(p), fz.alloc_workspace_cache(p, cache)
    bf = torch.bfloat16
    W, C = _dev(rng.standard_normal((1, 32, D)) / D ** 0.5, bf), _dev(rng.standard_normal((1, K, 32)), bf)
    stream = torch.cuda.Stream()
    for step, n_new in enumerate((None, np.array([3, 0, 1], np.int32))):
        k, v, q, _ = next(_decode_inputs(rng, p, 1, "bf16"))
        h = _dev(rng.standard_normal((B, T, D)), bf)
        a = [_dev(q, bf), _dev(k, bf), _dev(v, bf)]
        nn = None if n_new is None else _dev(n_new)
        torch.cuda.synchronize()
        O, gid, lse = fz.run_decode_step(p, h, W, C, *a, cache, ws, wc, n_new=nn, want_lse=True,
                                         accumulate=bool(step), stream=stream)
        stream.synchronize()
        assert fz.focus_check_errors(ws, stream) == 0 and fz.focus_check_errors(wc, stream) == 0
        g = gid.cpu().numpy()
        c = cr.append(c, k, v, g, n_new)
        ref = cr.attention(c, q, g, w, p.scale, n_new)
        there = ~np.isnan(ref["lse"])
        o = O.float().cpu().numpy()
        _o_within(O, ref, d, "bf16", there)
        assert (o[~there] == 0).all()
        assert np.abs(lse.cpu().numpy()[there] - ref["lse"][there]).max() < 1e-3
        c["mass"] = _host(cache)["mass"]
        _same(_host(cache), c)


def test_captured_step_replays_with_growing_counts(fz):
    """append + attention + eviction captured once and replayed: the counts live on the device."""
    import torch
    rng = np.random.default_rng(29)
    B, G, H_kv, d, K, w = 2, 4, 2, 128, 4, 16
    c = _make(14, B, H_kv, d, [120, 70], K, 1, room=40, spare=10)
    c["mass"][:] = 0
    p = _params(fz, B, G, H_kv, 1, d, K, 1, w)
    cache = _cache(fz, c)
    dst = cr.empty(B, H_kv, d, 8, 2, 6)
    to = _cache(fz, dst)
    ws = fz.alloc_workspace_cache(p, cache)
    bf = torch.bfloat16
    k, v, q = (torch.zeros(s, dtype=bf, device="cuda") for s in ((B, H_kv, 1, d), (B, H_kv, 1, d), (B, G * H_kv, 1, d)))
    gid = torch.zeros((B, 1, 1), dtype=torch.int32, device="cuda")
    O, lse = torch.zeros_like(q), torch.zeros((B, G * H_kv, 1), device="cuda")

    def step():
        fz.focus_cache_append(p, k, v, gid, cache, ws)
        fz.focus_cache_attention_fwd(p, q, gid, cache, O, lse, ws, accumulate=True)
        fz.focus_cache_evict(p, 100, w, cache, to, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for kn, vn, qn, gn in _decode_inputs(rng, p, 12, "bf16"):
        for t, x in ((k, kn), (v, vn), (q, qn), (gid, gn)):
            t.copy_(torch.from_numpy(np.ascontiguousarray(x)))
        graph.replay()
        torch.cuda.synchronize()
        c = cr.append(c, kn, vn, gn)
        ref = cr.attention(c, qn, gn, w, p.scale)
        _o_within(O, ref, d, "bf16")
        got = _host(cache)
        assert np.allclose(got["mass"], c["mass"] + ref["got"], rtol=1e-5, atol=1e-5, equal_nan=True)
        c["mass"] = got["mass"]
        _same(got, c)
        dst = cr.evict(c, dst, 100, w)
        _same(_host(to), dst)
    assert fz.focus_check_errors(ws) == 0


def test_attention_is_the_same_bits_again_and_on_another_stream(fz):
    import torch
    c = _make(41, 3, 2, 128, [900, 64, 333], 4, 2)
    rng = np.random.default_rng(1)
    Q, gid = _rows(rng, (3, 8, 6, 128), "bf16", 0.3), rng.integers(0, 4, (3, 2, 6)).astype(np.int32)
    p = fz.make_params(3, 8, 2, 6, 128, 64, 64, 4, 2, 40)
    q, g = _dev(Q, torch.bfloat16), _dev(gid)
    outs = []
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        cache = _cache(fz, c)
        ws = fz.alloc_workspace_cache(p, cache)
        O, lse = torch.zeros_like(q), torch.zeros((3, 8, 6), device="cuda")
        torch.cuda.synchronize()
        fz.focus_cache_attention_fwd(p, q, g, cache, O, lse, ws, accumulate=True, stream=stream)
        torch.cuda.synchronize()
        outs.append([x.clone() for x in (O, lse, cache.mass)])
    for o in outs[1:]:
        assert all(torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                               b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))
                   for a, b in zip(o, outs[0]))


def _cycle(fz, seed):
    """Append, attention and eviction over buffers of their own, and what they leave."""
    import torch
    B, H, H_kv, L, T, d, K = 2, 16, 2, 3000, 4, 128, 8
    rng = np.random.default_rng(seed)
    p = fz.make_params(B, H, H_kv, L, d, 64, 64, K, 1, 64)
    q = fz.make_params(B, H, H_kv, T, d, 64, 64, K, 1, 64)
    bf = torch.bfloat16
    k, v = (_dev(_rows(rng, (B, H_kv, L, d), "bf16"), bf) for _ in range(2))
    Q = _dev(_rows(rng, (B, H, T, d), "bf16", 0.3), bf)
    gid = _dev(rng.integers(0, K, (B, 1, L)).astype(np.int32))
    gid1 = gid[:, :, -T:].contiguous()
    src, dst = fz.alloc_cache(p, L, mass=True), fz.alloc_cache(p, 640, mass=True)
    ws, O = fz.alloc_workspace_cache(p, src), torch.zeros_like(Q)

    def run():
        src.len.zero_()
        src.next.zero_()
        fz.focus_cache_append(p, k, v, gid, src, ws)
        fz.focus_cache_attention_fwd(q, Q, gid1, src, O, None, ws, accumulate=True)
        fz.focus_cache_evict(p, 600, 64, src, dst, ws)

    return run, ws, lambda: [x.cpu().clone() for x in (O.float(), src.mass, dst.k, dst.pos, dst.mass, dst.len)]


def test_two_threads_on_two_streams(fz):
    import threading

    import torch
    jobs = [_cycle(fz, seed) for seed in (2, 3)]
    want = []
    for run, ws, out in jobs:
        run()
        want.append(out())

    def work(run):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                run()
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(run,)) for run, _, _ in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (_, ws, out), w in zip(jobs, want):
        assert fz.focus_check_errors(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(out(), w))


FIRST_CALL = """
import sys
import torch
sys.path[:0] = [{root!r}, {tests!r}]
from learned_group_sparse_focus_gb300 import focus as fz
import test_gpu_cache as t
run, ws, out = t._cycle(fz, 1)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
a = out()
run()
assert fz.focus_check_errors(ws) == 0 and a[0].abs().max() > 0
assert all(torch.equal(x, y) for x, y in zip(a, out()))
"""


def test_a_process_may_capture_its_first_call():
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_writes_stay_inside_their_buffers(fz):
    """Every buffer that a call writes sits between guard bytes."""
    import torch
    from test_gpu_canary import Guarded
    B, G, H_kv, d, K, w, T = 2, 3, 2, 64, 3, 10, 5
    c = _make(51, B, H_kv, d, [130, 63], K, 1, spare=8, room=T)
    g = {k: Guarded(c[k].shape, _dev(c[k]).dtype, _dev(c[k])) for k in NAMES}
    cache = fz.Cache(**{k: x.t for k, x in g.items()})
    dst = cr.empty(B, H_kv, d, 5, 2, 6)
    gd = {k: Guarded(dst[k].shape, _dev(dst[k]).dtype, _dev(dst[k])) for k in NAMES}
    to = fz.Cache(**{k: x.t for k, x in gd.items()})
    p = _params(fz, B, G, H_kv, T, d, K, 1, w)
    ws = Guarded((fz.focus_cache_workspace_bytes(p, cache),), torch.uint8)
    fz.focus_workspace_init(ws.t)
    bf = torch.bfloat16
    k, v, q, gid = next(_decode_inputs(np.random.default_rng(1), p, 1, "bf16"))
    O, lse = Guarded(q.shape, bf), Guarded(q.shape[:3], torch.float32)
    fz.focus_cache_append(p, _dev(k, bf), _dev(v, bf), _dev(gid), cache, ws.t)
    fz.focus_cache_attention_fwd(p, _dev(q, bf), _dev(gid), cache, O.t, lse.t, ws.t, accumulate=True)
    fz.focus_cache_evict(p, 100, 10, cache, to, ws.t)
    assert fz.focus_check_errors(ws.t) == 0
    for x in (*g.values(), *gd.values(), ws, O, lse):
        assert x.intact()
