"""Rotary positions and drafted trees without a GPU: pins of their fp64 oracle, the
refusals of the C entry points and the Python binding's checks of tensors."""
import ctypes
import itertools
import os
from fractions import Fraction

import numpy as np
import pytest

import oracle.cache_ref as cr
import oracle.tree_ref as tr


@pytest.fixture(scope="module")
def fz():
    from learned_group_sparse_focus_gb300 import _build
    if not os.path.exists(_build.LIB):
        _build.build()
    from learned_group_sparse_focus_gb300 import focus
    return focus


# ----------------------------------------------------------------- oracle ---

def test_angles_of_far_positions():
    """Against exact whole-number arithmetic with 200 bits of 1 / (2 pi)."""
    # pi by Machin's formula, in units of 2^-260
    one = 1 << 260

    def arctan_inv(x):
        total, term, n, sign = 0, one // x, 1, 1
        while term:
            total += sign * (term // n)
            term //= x * x
            n += 2
            sign = -sign
        return total

    pi = 4 * (4 * arctan_inv(5) - arctan_inv(239))
    freq = np.float32([1.0, 0.7498942, 1e-3, 7.3e-8])
    for pos in (0, 1, 12345, (1 << 20) + 7, (1 << 31) - 1):
        c, s = tr.cos_sin(np.array([pos]), freq)
        for j, f in enumerate(freq):
            angle = Fraction(float(f)) * pos * one                     # radians in units of 2^-260
            rest = float((angle - 2 * pi * round(angle / (2 * pi))) / one)
            assert abs(c[0, j] - np.cos(rest)) < 1e-9 and abs(s[0, j] - np.sin(rest)) < 1e-9


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_hand_and_its_transpose(interleaved):
    freq = np.float32([np.pi / 2, 0.5] + [0.0] * 6)
    x = np.arange(1.0, 33.0)[None]
    y = tr.rotate(x, np.array([1]), freq, interleaved)[0]
    i, j = (0, 1) if interleaved else (0, 8)
    assert abs(y[i] + x[0, j]) < 1e-6 and abs(y[j] - x[0, i]) < 1e-6       # a quarter turn: (a, b) -> (-b, a)
    i, j = (2, 3) if interleaved else (1, 9)
    a, b = x[0, i], x[0, j]
    assert abs(y[i] - (a * np.cos(0.5) - b * np.sin(0.5))) < 1e-12
    assert abs(y[j] - (a * np.sin(0.5) + b * np.cos(0.5))) < 1e-12
    assert np.array_equal(y[16:], x[0, 16:])
    rng = np.random.default_rng(0)
    u, v, at = rng.standard_normal((5, 32)), rng.standard_normal((5, 32)), rng.integers(0, 1 << 20, 5)
    fwd, back = tr.rotate(u, at, freq, interleaved, 1.5), tr.rotate(v, at, freq, interleaved, 1.5, transpose=True)
    assert abs((fwd * v).sum() - (u * back).sum()) < 1e-9                  # <R u, v> = <u, R' v>
    again = tr.rotate(tr.rotate(u, at, freq, interleaved), at, freq, interleaved, transpose=True)
    assert np.abs(again - u).max() < 1e-12


def test_scores_of_turned_rows_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    freq = np.float32(10000.0 ** (-np.arange(32) / 32))
    q, k = rng.standard_normal((1, 64)), rng.standard_normal((1, 64))
    s = [(tr.rotate(q, np.array([x + 77]), freq) * tr.rotate(k, np.array([x]), freq)).sum() for x in (0, 5, 10 ** 6)]
    assert abs(s[0] - s[1]) < 1e-9 and abs(s[0] - s[2]) < 1e-9


def test_accept_against_brute_force():
    rng = np.random.default_rng(2)
    for _ in range(200):
        T = int(rng.integers(1, 9))
        parent = np.array([[int(rng.integers(-1, t)) if t else -1 for t in range(T)]])
        token, target = rng.integers(0, 2, (1, T)), rng.integers(0, 2, (1, T))
        prev = rng.integers(0, 2, 1)
        (path,), last = tr.accept(token, target, prev, parent)
        # every ascending subset of nodes that is a chain from a root and follows the choices
        best = []
        for size in range(T, 0, -1):
            good = []
            for sub in itertools.combinations(range(T), size):
                ups = (-1,) + sub[:-1]
                if all(parent[0, t] == u for t, u in zip(sub, ups)) and \
                        all(token[0, t] == (prev[0] if u < 0 else target[0, u]) for t, u in zip(sub, ups)):
                    good.append(sub)
            if good:
                best = list(min(good, key=lambda g: g[-1]))
                break
        assert path == best and last[0] == (target[0, best[-1]] if best else prev[0])


def test_a_chain_is_what_an_append_and_attention_give():
    """A tree without branches over exact values: the same as appending first."""
    rng = np.random.default_rng(3)
    H_kv, d, n, T, G = 2, 64, 90, 5, 2
    gid = rng.integers(0, 3, (1, 1, n + T)).astype(np.int32)
    x = rng.integers(-3, 4, (2, 1, H_kv, n + T, d)).astype(np.float64)      # e4m3 at scale 2^-7 holds these
    c = cr.append(cr.empty(1, H_kv, d, 4, 3, 0), x[0][:, :, :n], x[1][:, :, :n], gid[:, :, :n])
    Q = rng.standard_normal((1, G * H_kv, T, d))
    tree = tr.attention(c, Q, x[0][:, :, n:], x[1][:, :, n:], gid[:, :, n:], np.arange(-1, T - 1)[None], 4, 0.125)
    full = cr.append(c, x[0][:, :, n:], x[1][:, :, n:], gid[:, :, n:])
    want = cr.attention(full, Q, gid[:, :, n:], 4, 0.125)
    assert np.abs(tree["O"] - want["O"]).max() < 1e-12 and np.abs(tree["lse"] - want["lse"]).max() < 1e-12


# --------------------------------------------------------------- refusals ---

def _struct(fz, **over):
    c = fz.CacheStruct(n_pages=4, max_pages=2)
    for i, name in enumerate(("k", "v", "k_scale", "v_scale", "pos", "gid", "mass", "table", "len", "next")):
        setattr(c, name, (i + 1) << 20)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def _params(fz, **kw):
    f = dict(B=2, H=4, H_kv=2, n=3, d=64, D=64, d_g=32, K=4, A=1, w=8)
    f.update(kw)
    return fz.make_params(**f)


def _rot(fz, inv_freq=1 << 24, dim=64, interleaved=0, scale=1.0):
    return fz.RotaryStruct(inv_freq, dim, interleaved, scale)


BAD_ROTATIONS = (dict(inv_freq=None), dict(inv_freq=8), dict(dim=0), dict(dim=8), dict(dim=24), dict(dim=80), dict(dim=-16),
                 dict(interleaved=2), dict(interleaved=-1), dict(scale=float("nan")), dict(scale=float("inf")))
X = [(64 + i) << 20 for i in range(16)]        # aligned, never dereferenced


def test_structs_and_status(fz):
    assert ctypes.sizeof(fz.RotaryStruct) == 24
    assert fz.lib().focus_status_string(8) == b"parent or row of a drafted tree out of range"


def test_rotary_refusals(fz):
    def call(p=None, rot=None, base=None, parent=None, n_new=None, Q=X[0], K=X[1], Qo=X[2], Ko=X[3], ws=1 << 26, nbytes=256):
        p, rot = p or _params(fz), rot or _rot(fz)
        return fz.lib().focus_rotary(ctypes.byref(p), ctypes.byref(rot), 0, base, parent, n_new, Q, K, Qo, Ko, ws, nbytes, None)

    for bad in BAD_ROTATIONS:
        assert call(rot=_rot(fz, **bad)) == 1, bad
    assert fz.lib().focus_rotary(ctypes.byref(_params(fz)), None, 0, None, None, None, X[0], None, X[0], None, 1 << 26, 256, None) == 1
    p = _params(fz)
    p.H_kv = 3
    assert call(p=p) == 1 and call(ws=None) == 1 and call(ws=(1 << 26) + 64) == 1 and call(nbytes=255) == 3
    for kw in (dict(Q=None), dict(K=None), dict(Qo=None), dict(Ko=None), dict(Q=None, K=None, Qo=None, Ko=None),
               dict(Qo=X[1]), dict(Ko=X[0]), dict(Qo=X[3]), dict(Q=X[0] + 8), dict(Ko=X[3] + 4), dict(base=4), dict(parent=8),
               dict(n_new=2)):
        assert call(**kw) == 1, kw
    assert call(p=_params(fz, d=96)) == 2 and call(p=_params(fz, n=65), parent=X[4]) == 2


def test_append_rotary_refusals(fz):
    def call(p=None, rot=_rot(fz), cache=None, Q=X[0], K=X[1], V=X[2], gid=X[3], rows=None, n_new=None, Qo=X[4], Ko=X[5],
             ln=X[6], nx=X[7], ws=1 << 26, nbytes=1 << 40):
        p, cache = p or _params(fz), cache or _struct(fz)
        return fz.lib().focus_cache_append_rotary(ctypes.byref(p), None if rot is None else ctypes.byref(rot), Q, K, V, gid, rows,
                                                  n_new, ctypes.byref(cache), Qo, Ko, ln, nx, ws, nbytes, None)

    for bad in BAD_ROTATIONS:
        assert call(rot=_rot(fz, **bad)) == 1, bad
    for over in (dict(k=0), dict(v=8), dict(table=0), dict(mass=4), dict(n_pages=0)):
        assert call(cache=_struct(fz, **over)) == 1, over
    for kw in (dict(K=None), dict(V=None), dict(gid=None), dict(ln=None), dict(nx=None), dict(K=X[1] + 8), dict(Q=None), dict(Qo=None),
               dict(Q=X[0] + 8), dict(Qo=X[4] + 8), dict(Ko=X[5] + 8), dict(rows=X[8] + 4), dict(n_new=4), dict(rows=X[8]),
               dict(rows=X[8], Q=None, Qo=None), dict(rows=X[8], Ko=None), dict(rot=None), dict(Ko=X[2]), dict(Ko=X[0]), dict(Ko=X[4]),
               dict(Qo=X[1]), dict(Qo=X[2]), dict(ln=X[7]), dict(ws=None), dict(ws=(1 << 26) + 16)):
        assert call(**kw) == 1, kw
    c = _struct(fz)
    assert call(ln=c.next) == call(nx=c.len) == 1 and call(nbytes=256) == 3 and call(p=_params(fz, d=32)) == 2


def test_accept_refusals(fz):
    def call(p=None, token=X[0], target=X[1], prev=X[2], parent=X[3], n_new=None, rows=X[4], count=X[5], last=X[6], ws=1 << 26,
             nbytes=256):
        p = p or _params(fz)
        return fz.lib().focus_tree_accept(ctypes.byref(p), token, target, prev, parent, n_new, rows, count, last, ws, nbytes, None)

    for name in ("token", "target", "prev", "parent", "rows", "count", "last"):
        assert call(**{name: None}) == 1 and call(**{name: X[9] + 4}) == 1, name
    for kw in (dict(rows=X[0]), dict(rows=X[3]), dict(count=X[2]), dict(last=X[1]), dict(rows=X[5]), dict(rows=X[6]), dict(count=X[6]),
               dict(n_new=X[4]), dict(n_new=4), dict(ws=None), dict(ws=128)):
        assert call(**kw) == 1, kw
    assert call(nbytes=255) == 3 and call(p=_params(fz, n=65)) == 2


def test_python_binding_checks_tensors(fz):
    import torch
    p = _params(fz)
    for bad in (torch.zeros(12), torch.zeros(0), torch.zeros(2, 16), torch.zeros(16).double(), torch.zeros(32)[::2], None):
        with pytest.raises(ValueError):
            fz.Rotary(bad)
    rot = fz.Rotary(torch.ones(16), interleaved=True, scale=2.0)
    assert rot.struct.dim == 32 and rot.struct.interleaved == 1 and rot.struct.scale == 2.0
    c = fz.alloc_cache(p, 100, mass=True, device="cpu")
    q, k = (torch.zeros((2, h, 3, 64), dtype=torch.bfloat16) for h in (4, 2))
    gid, rows = torch.zeros((2, 1, 3), dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    one, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        fz.focus_cache_append_rotary(p, rot, k, k, gid, c, ws)
    with pytest.raises(ValueError, match="CUDA"):
        fz.focus_rotary(p, rot, ws, K=k, K_out=k)
    with pytest.raises(ValueError, match="CUDA"):
        fz.focus_tree_accept(p, rows, rows, one, rows, rows, one, one, ws)
    for kw in (dict(Q=k, Q_out=q), dict(Q=q, Q_out=q.float()), dict(K_out=q), dict(rows=one), dict(n_new=rows), dict(rows=rows.long())):
        with pytest.raises(ValueError, match="must be"):
            fz.focus_cache_append_rotary(p, rot, k, k, gid, c, ws, **kw)
    for kw in (dict(Q=k, Q_out=q), dict(K=k, K_out=q), dict(base=rows), dict(parent=one), dict(n_new=rows), dict(K=k.transpose(2, 3))):
        with pytest.raises(ValueError, match="must be"):
            fz.focus_rotary(p, rot, ws, **kw)
    for i in range(7):
        x = [rows, rows, one, rows, rows, one, one]
        x[i] = x[i].long()
        with pytest.raises(ValueError, match="must be"):
            fz.focus_tree_accept(p, *x, ws)


def test_tree_attention_refusals(fz):
    lib = fz.lib()

    def call(p=None, Q=X[0], K=X[1], V=X[2], gid=X[3], parent=X[4], n_new=None, cache=None, O=X[5], lse=None, ws=1 << 26,
             nbytes=1 << 40):
        p, cache = p or _params(fz), cache or _struct(fz)
        return lib.focus_cache_attention_tree_fwd(ctypes.byref(p), Q, K, V, gid, parent, n_new, ctypes.byref(cache), O, lse, ws,
                                                  nbytes, None)

    for name in ("Q", "K", "V", "gid", "parent", "O"):
        assert call(**{name: None}) == 1 and call(**{name: X[9] + 8}) == 1, name
    for kw in (dict(n_new=4), dict(lse=8), dict(O=X[0]), dict(O=X[1]), dict(O=X[2]), dict(ws=None), dict(ws=(1 << 26) + 128),
               dict(cache=_struct(fz, k=0)), dict(cache=_struct(fz, table=8)), dict(cache=_struct(fz, max_pages=0))):
        assert call(**kw) == 1, kw
    p = _params(fz)
    p.w = -1
    assert call(p=p) == 1 and lib.focus_tree_workspace_bytes(ctypes.byref(p)) == 0
    assert call(nbytes=lib.focus_tree_workspace_bytes(ctypes.byref(_params(fz))) - 1) == 3
    assert call(p=_params(fz, d=96)) == 2 and call(p=_params(fz, n=65)) == 2
    assert call(cache=_struct(fz, n_pages=(1 << 23) + 1)) == 2              # pools past 2^36 bytes


def test_python_binding_checks_tree_tensors(fz):
    import torch
    p = _params(fz)
    c = fz.alloc_cache(p, 100, device="cpu")
    q, k = (torch.zeros((2, h, 3, 64), dtype=torch.bfloat16) for h in (4, 2))
    gid, parent = torch.zeros((2, 1, 3), dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    good = [q, k, k, gid, parent, c, q, None, ws]
    with pytest.raises(ValueError, match="CUDA"):
        fz.focus_cache_attention_tree_fwd(p, *good)
    for i, bad in ((0, k), (1, q), (2, k.float()), (3, gid.long()), (4, gid), (6, k), (7, parent)):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError, match="must be"):
            fz.focus_cache_attention_tree_fwd(p, *args)
    with pytest.raises(ValueError, match="must be"):
        fz.focus_cache_attention_tree_fwd(p, *good, n_new=parent)
