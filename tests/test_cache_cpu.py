"""The key/value cache without a GPU: pins of its fp64 oracle, the refusals of
the C entry points and the Python binding's checks of tensors."""
import ctypes
import os

import numpy as np
import pytest

import oracle.cache_ref as cr
import oracle.focus_ref as ref
from learned_group_sparse_focus_gb300 import synth


@pytest.fixture(scope="module")
def fz():
    from learned_group_sparse_focus_gb300 import _build
    if not os.path.exists(_build.LIB):
        _build.build()
    from learned_group_sparse_focus_gb300 import focus
    return focus


# ----------------------------------------------------------------- oracle ---

def test_e4m3_table_and_rounding_match_torch():
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(cr.VALUES.astype(np.float32), want, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 2.0 ** np.arange(-12, 8).repeat(200),
                        (cr.VALUES[1:127] + cr.VALUES[:126]) / 2, [0.0, -0.0, 448.0, -448.0, 2.0 ** -10, 2.0 ** -11]])
    x = np.clip(x, -448, 448).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(cr.encode(x), got)
    assert list(cr.encode(np.array([np.inf, -np.inf, np.nan, 1e9]))) == [126, 254, 127, 126]


def test_page_exponent_is_the_least_that_holds_the_rows():
    for x in (1e-30, 2.0 ** -56, 448 * 2.0 ** -64, 449 * 2.0 ** -64, 1.0, 1.75, 1.7500001, 448.0, 448.1, 3e38):
        e = cr.need_exp(np.array([x, -x / 3, np.inf, np.nan]))
        assert 448 * 2.0 ** e >= x and (e == cr.MIN_EXP or 448 * 2.0 ** (e - 1) < x)
    assert cr.need_exp(np.zeros(3)) == cr.need_exp(np.array([np.nan, np.inf])) == cr.MIN_EXP


def _filled(B, H_kv, d, lens, K, A, seed, extra=1):
    rng = np.random.default_rng(seed)
    T = max(lens)
    mp = -(-T // 64) + extra
    c = cr.empty(B, H_kv, d, B * mp + 2, mp, seed)
    Kx, Vx = (synth.round_bf16(rng.standard_normal((B, H_kv, T, d)).astype(np.float32)) for _ in range(2))
    gid = rng.integers(0, K, (B, A, T)).astype(np.int32)
    return cr.append(c, Kx, Vx, gid, np.array(lens)), Kx, Vx, gid


def test_appended_values_are_within_half_a_step_of_the_inputs():
    c, Kx, _, _ = _filled(2, 3, 64, [200, 77], 4, 1, 5)
    for b, n in enumerate((200, 77)):
        for h in range(3):
            page, row = cr.slots(c, b, h)
            got = cr.values(c, "k", page, h, row)
            x = Kx[b, h, :n].astype(np.float64)
            low = c["k_scale"][page, h].astype(np.float64)[:, None] * 2.0 ** -10     # half a subnormal step
            assert (np.abs(got - x) <= np.maximum(np.abs(x) * 2.0 ** -4, low)).all()
            assert list(c["pos"][page, h, row]) == list(range(n))


def test_token_by_token_append_ends_in_the_same_scales():
    rng = np.random.default_rng(3)
    x = synth.round_bf16((rng.standard_normal((1, 2, 100, 64)) * np.exp(rng.standard_normal((1, 2, 100, 1)))).astype(np.float32))
    gid = np.zeros((1, 1, 100), np.int32)
    one = cr.append(cr.empty(1, 2, 64, 2, 2, 0), x, x, gid)
    many = cr.empty(1, 2, 64, 2, 2, 0)
    for t in range(100):
        many = cr.append(many, x[:, :, t:t + 1], x[:, :, t:t + 1], gid[:, :, t:t + 1])
    assert np.array_equal(one["k_scale"][one["table"][0]], many["k_scale"][many["table"][0]])
    for h in range(2):
        page, row = cr.slots(one, 0, h)
        a, b = cr.values(one, "k", page, h, row), cr.values(many, "k", page, h, row)
        step = one["k_scale"][page, h].astype(np.float64)[:, None] * 2.0 ** -9
        assert (np.abs(a - b) <= step).all()         # rounded twice only below the normals


@pytest.mark.parametrize("A,w", [(1, 9), (2, 40), (1, 0)])
def test_attention_over_the_cache_is_focus_attention_of_its_values(A, w):
    H, H_kv, d, n = 4, 2, 64, 150
    c, _, _, gid = _filled(1, H_kv, d, [n], 5, A, 11)
    page, row = cr.slots(c, 0, 0)
    k = np.stack([cr.values(c, "k", page, h, row) for h in range(H_kv)])[None]
    v = np.stack([cr.values(c, "v", page, h, row) for h in range(H_kv)])[None]
    q = np.random.default_rng(1).standard_normal((1, H, n, d))
    T = 7
    got = cr.attention(c, q[:, :, n - T:], gid[:, :, n - T:], w, 0.125)
    O, lse = ref.attention_rows(q, k, v, gid, max(w, 1), 0.125, np.arange(n - T, n), A)
    assert np.abs(got["O"] - O).max() < 1e-12 and np.abs(got["lse"] - lse).max() < 1e-12
    assert abs(got["got"].sum() - H * T) < 1e-9      # every row's weights sum to 1


def test_eviction_keeps_the_recent_and_the_heaviest():
    mass = np.array([0, 5, 1, np.nan, 5, -0.0, 2, 9, 0, 0], np.float32)
    pos = np.array([3, 4, 8, 9, 12, 13, 14, 20, 21, 22])
    assert list(cr.stays(mass, pos, 23, 5, 2)) == [1, 3, 7, 8, 9]       # 21, 22 recent; NaN, 9, then the first 5
    assert list(cr.stays(mass, pos, 23, 4, 0)) == [1, 3, 4, 7]
    assert list(cr.stays(mass, pos, 23, 8, 1)) == [0, 1, 2, 3, 4, 6, 7, 9]   # 0 before -0 and 0: the lowest slot
    assert list(cr.stays(mass, pos, 23, 10, 0)) == list(range(10))


def test_evicting_nothing_copies_the_cache_exactly():
    c, _, _, _ = _filled(2, 2, 64, [130, 40], 4, 1, 9)
    c["mass"][:] = 1.0
    out = cr.evict(c, cr.empty(2, 2, 64, 8, 3, 4), 192, 0)
    for b in range(2):
        for h in range(2):
            (p0, r0), (p1, r1) = cr.slots(c, b, h), cr.slots(out, b, h)
            for x in ("k", "v"):
                assert np.array_equal(cr.values(c, x, p0, h, r0), cr.values(out, x, p1, h, r1))


# --------------------------------------------------------------- refusals ---

def _struct(fz, **over):
    c = fz.CacheStruct(n_pages=4, max_pages=2)
    for i, name in enumerate(("k", "v", "k_scale", "v_scale", "pos", "gid", "mass", "table", "len", "next")):
        setattr(c, name, (i + 1) << 20)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def _calls(fz, p, c, ws=1 << 26, nbytes=1 << 40, bad=None, n_new=None, dst=None, budget=64, recent=8, accumulate=1):
    """Status of the three calls with aligned, never-dereferenced addresses."""
    lib, P, C, ok = fz.lib(), ctypes.byref(p), ctypes.byref(c), 1 << 27
    x = [ok] * 5
    if bad is not None:
        x[bad[0]] = bad[1]
    dst = _struct(fz, table=1 << 25) if dst is None else dst
    return (lib.focus_cache_append(P, x[0], x[1], x[2], n_new, C, x[3], x[4], ws, nbytes, None),
            lib.focus_cache_attention_fwd(P, x[0], x[1], n_new, C, x[2], None, accumulate, ws, nbytes, None),
            lib.focus_cache_evict(P, budget, recent, C, ctypes.byref(dst), ws, nbytes, None))


def _params(fz, **kw):
    f = dict(B=2, H=4, H_kv=2, n=1, d=64, D=64, d_g=32, K=4, A=1, w=8)
    f.update(kw)
    return fz.make_params(**f)


def test_bad_params_and_caches_are_refused(fz):
    p = _params(fz)
    p.H_kv = 3
    assert _calls(fz, p, _struct(fz)) == (1, 1, 1)
    p = _params(fz)
    for over in (dict(k=0), dict(v=8), dict(k_scale=4), dict(pos=0), dict(gid=2), dict(table=0), dict(len=1),
                 dict(next=0), dict(mass=4), dict(n_pages=0), dict(max_pages=0), dict(n_pages=(1 << 24) + 1),
                 dict(max_pages=-1)):
        assert _calls(fz, p, _struct(fz, **over)) == (1, 1, 1), over
        assert fz.lib().focus_cache_workspace_bytes(ctypes.byref(p), ctypes.byref(_struct(fz, **over))) == 0
    assert fz.lib().focus_cache_append(ctypes.byref(p), 16, 16, 16, None, None, 16, 16, 256, 1 << 30, None) == 1
    assert _calls(fz, p, _struct(fz), ws=(1 << 26) + 128) == (1, 1, 1)
    assert _calls(fz, p, _struct(fz), ws=None) == (1, 1, 1)
    for i in range(5):
        for v in (None, (1 << 27) + 8):
            st = _calls(fz, p, _struct(fz), bad=(i, v), nbytes=0 if i > 2 else 1 << 40)
            assert st[0] == (1 if i <= 2 else 3) and (i > 2 or st[1] == 1)
    assert _calls(fz, p, _struct(fz), n_new=(1 << 27) + 4)[:2] == (1, 1)


def test_unsupported_and_small_workspace(fz):
    p = _params(fz, d=96)
    assert _calls(fz, p, _struct(fz)) == (2, 2, 2)
    p = _params(fz)
    need = fz.lib().focus_cache_workspace_bytes(ctypes.byref(p), ctypes.byref(_struct(fz)))
    # error block + per (sequence, head) a count and the kept slots of two pages
    assert need == 256 + -(-2 * 2 * (2 * 64 + 1) * 4 // 256) * 256
    assert _calls(fz, p, _struct(fz), nbytes=need - 256) == (3, 3, 3)
    assert fz.lib().focus_cache_workspace_bytes(ctypes.byref(p), ctypes.byref(_struct(fz, mass=None))) == 256
    lib, c = fz.lib(), _struct(fz)
    big = _struct(fz, n_pages=1 << 23)                   # 2^23 pages x 2 heads x 64 slots x 64 bytes: 2^36
    assert _calls(fz, p, big, nbytes=0) == (3, 3, 3)
    big.n_pages += 1
    assert _calls(fz, p, big) == (2, 2, 2)
    q = _params(fz, n=65)
    assert lib.focus_cache_attention_fwd(ctypes.byref(q), 16, 16, None, ctypes.byref(c), 16, None, 0, 256, 1 << 40,
                                         None) == 2


def test_eviction_and_accumulation_arguments(fz):
    p, lib = _params(fz), fz.lib()
    assert _calls(fz, p, _struct(fz, mass=None), nbytes=1 << 40)[2] == 1

    def evict(budget=64, recent=8, **dst):
        d = _struct(fz, **{"table": 1 << 25, **dst})
        return lib.focus_cache_evict(ctypes.byref(p), budget, recent, ctypes.byref(_struct(fz)), ctypes.byref(d),
                                     1 << 26, 1 << 40, None)

    assert evict(budget=0) == evict(recent=-1) == evict(budget=64, recent=65) == 1
    assert evict(budget=129) == 1                        # dst has two pages a sequence
    assert evict(mass=None) == evict(table=8 << 20) == evict(k=0) == 1
    assert lib.focus_cache_attention_fwd(ctypes.byref(p), 16, 16, None, ctypes.byref(_struct(fz, mass=None)), 16,
                                         None, 1, 256, 1 << 40, None) == 1


def test_append_counts_that_overlap_are_refused(fz):
    p, lib, c = _params(fz), fz.lib(), _struct(fz)

    def append(len_out, next_out):
        return lib.focus_cache_append(ctypes.byref(p), 1 << 27, 1 << 27, 1 << 27, None, ctypes.byref(c), len_out,
                                      next_out, 1 << 26, 1 << 40, None)

    assert append(1 << 28, 1 << 28) == append(c.next, 1 << 28) == append(1 << 28, c.len) == append(c.next, c.len) == 1


def test_eviction_counts_that_overlap_are_refused(fz):
    """dst's counts may be src's own, not each other nor the other one's source: blocks
    still read a sequence's next while others write their counts."""
    p, lib, src = _params(fz), fz.lib(), _struct(fz)

    def evict(length, nxt):
        d = _struct(fz, table=1 << 25, len=length, next=nxt)
        return lib.focus_cache_evict(ctypes.byref(p), 64, 8, ctypes.byref(src), ctypes.byref(d), 1 << 26, 1 << 40, None)

    assert evict(1 << 28, 1 << 28) == evict(src.next, 1 << 28) == evict(1 << 28, src.len) == evict(src.next, src.len) == 1


def test_cache_struct_matches_the_header(fz):
    assert ctypes.sizeof(fz.CacheStruct) == 10 * 8 + 2 * 4
    assert fz.lib().focus_status_string(7) == b"cache page, length or position out of range"


def test_python_binding_checks_tensors(fz):
    import torch
    p = _params(fz, n=3)
    c = fz.alloc_cache(p, 100, mass=True, device="cpu")
    assert c.table.shape == (2, 2) and c.k.shape == (4, 2, 64, 64) and c.dims == (2, 2, 64)
    fields = {k: getattr(c, k) for k in ("k", "v", "k_scale", "v_scale", "pos", "gid", "mass", "table", "len", "next")}
    for name, bad in (("v", c.v[:, :, :32]), ("pos", c.pos.long()), ("gid", c.gid[..., ::2]), ("len", c.len[0]),
                      ("k_scale", c.k_scale.t()), ("k", c.k[0]), ("table", c.table[0]), ("mass", c.mass.double())):
        with pytest.raises(ValueError):
            fz.Cache(**{**fields, name: bad})
    with pytest.raises(ValueError):
        fz.alloc_cache(p, 0, device="cpu")
    x = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16)
    gid = torch.zeros((2, 1, 3), dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):                    # a cache in host memory
        fz.focus_cache_append(p, x, x, gid, c, ws)
    for K, g, kw in ((x[:, :, :2], gid, {}), (x.float(), gid, {}), (x.transpose(0, 1), gid, {}), (x, gid.long(), {}),
                     (x, gid, dict(n_new=gid)), (x, gid, dict(len_out=c.next)), (x, gid, dict(next_out=c.len))):
        with pytest.raises(ValueError):
            fz.focus_cache_append(p, K, x, g, c, ws, **kw)
    Q = torch.zeros((2, 4, 3, 64), dtype=torch.bfloat16)
    for q, O, lse in ((x, Q, None), (Q, x, None), (Q, Q, gid), (Q, None, None)):
        with pytest.raises(ValueError):
            fz.focus_cache_attention_fwd(p, q, gid, c, O, lse, ws)
    other = fz.alloc_cache(_params(fz, H=8, H_kv=4), 64, mass=True, device="cpu")
    with pytest.raises(ValueError):
        fz.focus_cache_evict(p, 64, 0, c, other, ws)
    with pytest.raises(ValueError):
        fz.focus_cache_append(_params(fz, B=1, n=3), x[:1], x[:1], gid[:1], c, ws)
