"""Attention over the paged cache at the ends of its contract, against the fp64
oracle: the bits that the softmax weights keep, pages whose scales lie as far
apart as the format allows, the smallest and largest queries, NaN rows beside
sound ones with the weights accumulated, and bad pages, guard zones and group ids
per head in every form of the kernels.  Bounds are those of test_gpu_cache.py;
where one is tighter, the test derives it.
"""
import numpy as np
import pytest

import oracle.cache_ref as cr
import test_gpu_cache as base

pytestmark = pytest.mark.gpu
U = base.U


@pytest.fixture(scope="module")
def fz():
    from learned_group_sparse_focus_gb300 import focus
    return focus


def _random_cache(seed, B, H_kv, d, pages, K, spare=2):
    """Full pages of random codes (no NaN) at scale 1, anywhere in the pool."""
    rng = np.random.default_rng(seed)
    c = cr.empty(B, H_kv, d, B * pages + spare, pages, seed)
    for x in ("k", "v"):
        c[x] = np.where(c[x] & 127 == 127, 0x38, c[x]).astype(np.uint8)
        c[x + "_scale"][:] = 1.0
    for b in range(B):
        c["pos"][c["table"][b]] = np.arange(pages * 64).reshape(pages, 1, 64)
    c["gid"][:] = rng.integers(0, K, c["gid"].shape)
    c["mass"][:] = 0.0
    c["len"][:], c["next"][:] = pages * 64, pages * 64
    return c


# (G, d, T): the mma.sync kernel with one token and with several, eight rows and
# more; the tcgen05 kernel with 16, 32 and 64 rows, one token and several
FORMS = [(4, 128, 1), (2, 64, 3), (4, 64, 5), (12, 128, 1), (24, 128, 1), (40, 128, 1), (8, 128, 2), (4, 128, 7),
         (1, 128, 64)]


# ---------------------------------------------------------------- weights ---

@pytest.mark.parametrize("G,d,T", FORMS)
def test_weights_keep_sixteen_bits(fz, G, d, T):
    """bf16 outputs are within half a step and (r + 2^-16) sum P|v|: the weights enter the
    value product with a relative error of at most 2^-16 (the tcgen05 kernel's four e4m3
    parts: the first leaves at most 2^-4 of a weight, and an f16 number of that size is off
    by at most 2^-16; the other kernel's two f16 halves hold 22 bits).
    Small queries keep r, the error of the logits and of the sum, near 2^-16 too."""
    import torch
    rng = np.random.default_rng(G + T)
    B, H_kv, K, w, pages = 2, 2, 40, 4, 6
    c = _random_cache(3, B, H_kv, d, pages, K)
    c["v_scale"][:] = 2.0 ** rng.integers(-2, 3, c["v_scale"].shape)
    c["k_scale"][:] = 2.0 ** -6
    Q = base._rows(rng, (B, G * H_kv, T, d), "bf16", 0.0) * np.float32(2.0 ** -6)
    gid = rng.integers(0, K, (B, 1, T)).astype(np.int32)
    p = fz.make_params(B, G * H_kv, H_kv, T, d, 64, 64, K, 1, w)
    cache = base._cache(fz, c)
    ws = fz.alloc_workspace_cache(p, cache)
    O = torch.zeros((B, G * H_kv, T, d), dtype=torch.bfloat16, device="cuda")
    fz.focus_cache_attention_fwd(p, base._dev(Q, torch.bfloat16), base._dev(gid), cache, O, None, ws)
    assert fz.focus_check_errors(ws) == 0
    ref = cr.attention(c, Q, gid, w, p.scale)
    r = 2 * (d + 8) * 2 * U * ref["dot"] + ref["kept"] * 2 * U + 2.0 ** -20
    assert r.max() < 2.0 ** -14
    tol = 2.0 ** -9 * _power(ref["O"]) + (r[..., None] + 2.0 ** -16) * ref["pv"] * (1 + 2.0 ** -8) + \
        (ref["kept"] * 2.0 ** -26 * ref["page"])[..., None]
    over = np.abs(O.float().cpu().numpy().astype(np.float64) - ref["O"]) - tol
    assert over.max() <= 0, (over.max(), (over > 0).mean())


def _power(x):
    """Twice the power of two at or below |x|: a bf16 rounding is off by at most 2^-9 of it."""
    return 2.0 * 2.0 ** np.floor(np.log2(np.maximum(np.abs(x), 1e-38)))


# ----------------------------------------------------------------- scales ---

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,d,T", FORMS)
@pytest.mark.parametrize("pages", [4, 300])
def test_value_scales_as_far_apart_as_the_format_allows(fz, dtype, G, d, T, pages):
    """Exponents -64 to 120 side by side, in rising, falling and random order: every slot
    counts in the sum, the lse and the mass, however small its page's values are.  With
    300 pages a warp or a block meets several scales itself."""
    rng = np.random.default_rng(pages + G)
    K = 1 if pages == 4 else 3
    for order in ("up", "down", "any"):
        c = _random_cache(G, 1, 1, d, pages, K)
        e = np.array([-64, 0, 75, 118])[np.arange(pages) * 4 // pages]
        if order != "up":
            e = e[::-1] if order == "down" else rng.permutation(np.tile(np.array([-64, -63, 3, 60, 70, 118]), pages)[:pages])
        c["v_scale"][c["table"][0], 0] = 2.0 ** e.astype(np.float64)
        c["v"] = np.where(c["v"] & 127 > 0x70, 0x38, c["v"]).astype(np.uint8)      # at most 128: |v| <= 2^125
        c["k_scale"][:] = 2.0 ** -8
        if order == "any":
            c["v"][c["table"][0][e == -64]] = 0
        Q = base._rows(rng, (1, G, T, d), dtype, 0.2)
        Q[:, 0] = 0.0                                                              # a row of equal logits
        gid = rng.integers(0, K, (1, 1, T)).astype(np.int32)
        base._check_attention(fz, c, Q, gid, K, 100, dtype)


# ---------------------------------------------------------------- queries ---

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,d,T", FORMS)
def test_smallest_and_largest_queries(fz, dtype, G, d, T):
    """Rows down to the least normal numbers against keys near the largest, and the other
    way round: logits of order one."""
    rng = np.random.default_rng(G * T + d)
    for e in (120, 114, 100, 70, 0, -64):
        c = _random_cache(G + e + 64, 1, 1, d, 5, 2)
        c["k"] = np.where(c["k"] & 127 > 0x70, 0x38, c["k"]).astype(np.uint8)
        c["k_scale"][:] = 2.0 ** e
        c["v_scale"][:] = 2.0 ** -3
        Q = base._rows(rng, (1, G, T, d), dtype, 0.0)
        Q = (Q.astype(np.float64) * 2.0 ** max(-e - 4, -122)).astype(np.float32)
        gid = rng.integers(0, 2, (1, 1, T)).astype(np.int32)
        base._check_attention(fz, c, Q, gid, 2, 60, dtype)


# -------------------------------------------------------------------- NaN ---

def _nan_case(fz, c, Q, gid, K, w, bad_rows, what):
    """Attention with accumulate over a cache or queries with NaN: rows outside bad_rows
    [H, T] have the outputs and lse of the sound call bit for bit, the others are NaN;
    returns the mass."""
    import torch
    _, H, T, d = Q.shape
    p = fz.make_params(1, H, 1, T, d, 64, 64, K, 1, w)
    outs = []
    for bad in (False, True):
        cache = base._cache(fz, c[bad])
        ws = fz.alloc_workspace_cache(p, cache)
        O = torch.zeros((1, H, T, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((1, H, T), device="cuda")
        q = what[bad]
        fz.focus_cache_attention_fwd(p, base._dev(q, torch.bfloat16), base._dev(gid), cache, O, lse, ws, accumulate=True)
        assert fz.focus_check_errors(ws) == 0
        outs.append((O.float().cpu().numpy()[0], lse.cpu().numpy()[0], cache.mass.cpu().numpy()))
    (o0, l0, _), (o1, l1, mass) = outs
    assert np.array_equal(o0[~bad_rows], o1[~bad_rows]) and np.array_equal(l0[~bad_rows], l1[~bad_rows])
    assert np.isnan(o1[bad_rows]).all() and np.isnan(l1[bad_rows]).all()
    return mass


def _mass_of_others(c, Q, gid, w, mass):
    """NaN where token 0 (group 0: the even slots) keeps the slot, the oracle's elsewhere."""
    T, d, n = Q.shape[2], Q.shape[3], len(mass)
    ref = cr.attention(c, Q, gid, w, 1 / d ** 0.5)
    got, slot, pos0 = ref["got"][cr.slots(c, 0, 0)[0], 0, cr.slots(c, 0, 0)[1]], np.arange(n), n - T
    kept_by_0 = (slot <= pos0) & ((slot % 2 == 0) | (pos0 - slot < w))
    assert np.isnan(mass[kept_by_0]).all()
    off = np.abs(mass - got) - base._bounds(ref, d, "bf16")[1].max() * got - 2.0 ** -23 * np.abs(mass)
    assert (off[~kept_by_0] <= 0).all() and (got[~kept_by_0] > 0).any()


NAN_FORMS = [(2, 64, 2), (4, 128, 2), (8, 64, 2), (6, 128, 2), (16, 128, 2), (32, 128, 2), (1, 128, 16)]


@pytest.mark.parametrize("H,d,T", NAN_FORMS)
def test_nan_queries_leave_the_mass_of_other_tokens_slots(fz, H, d, T):
    """Token 0 has group 0, the others group 1, and one query row of token 0 is NaN: slots
    that only the other tokens keep have the mass of a call without it."""
    n, w = 300, 4
    c = base._make(4, 1, 1, d, [n], 2, 1)
    c["mass"][:] = 0
    page, row = cr.slots(c, 0, 0)
    c["gid"][page, 0, row] = np.arange(n) % 2
    gid = np.array([[[0] + [1] * (T - 1)]], np.int32)
    Q = base._rows(np.random.default_rng(1), (1, H, T, d), "bf16", 0.2)
    for v in (np.nan, np.inf):
        q = Q.copy()
        q[0, H // 2, 0, 3] = v
        bad = np.zeros((H, T), bool)
        bad[H // 2, 0] = True
        mass = _nan_case(fz, (c, c), Q, gid, 2, w, bad, (Q, q))[page, 0, row]
        _mass_of_others(c, Q, gid, w, mass)


@pytest.mark.parametrize("H,d,T", NAN_FORMS)
def test_nan_key_codes_leave_the_mass_of_other_tokens_slots(fz, H, d, T):
    """A NaN in a key that only token 0 keeps: that token's rows and slots are NaN, every
    other row, lse and mass is as without it."""
    n, w = 300, 4
    c = base._make(5, 1, 1, d, [n], 2, 1)
    c["mass"][:] = 0
    page, row = cr.slots(c, 0, 0)
    c["gid"][page, 0, row] = np.arange(n) % 2
    gid = np.array([[[0] + [1] * (T - 1)]], np.int32)
    Q = base._rows(np.random.default_rng(1), (1, H, T, d), "bf16", 0.2)
    broken = cr.copy(c)
    broken["k"][page[10], 0, row[10], 5] = 127
    broken["k"][page[200], 0, row[200], d - 1] = 255
    bad = np.zeros((H, T), bool)
    bad[:, 0] = True
    mass = _nan_case(fz, (c, broken), Q, gid, 2, w, bad, (Q, Q))[page, 0, row]
    _mass_of_others(c, Q, gid, w, mass)


# ----------------------------------------------- heads, pages and buffers ---

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,H_kv,d,T", [(1, 3, 64, 1), (4, 2, 128, 1), (12, 2, 128, 1), (40, 2, 128, 1), (2, 2, 128, 3),
                                        (8, 2, 128, 3), (2, 2, 128, 64), (70, 2, 128, 2)])
def test_a_group_id_for_each_key_value_head(fz, dtype, G, H_kv, d, T):
    """A = H_kv: every head keeps by its own ids; two sequences, ragged new tokens, up to
    three blocks of 64 rows."""
    rng = np.random.default_rng(G + T)
    c = base._make(G, 2, H_kv, d, [260, 131], 4, H_kv, dtype)
    Q = base._rows(rng, (2, G * H_kv, T, d), dtype, 0.3)
    gid = np.stack([rng.permutation(4)[:H_kv] for _ in range(2 * T)]).reshape(2, T, H_kv).transpose(0, 2, 1)
    gid = np.ascontiguousarray(gid, np.int32)                 # heads of a token never share an id
    base._check_attention(fz, c, Q, gid, 4, 9, dtype)
    base._check_attention(fz, c, Q, gid, 4, 9, dtype, n_new=np.array([T, T // 2], np.int32))


def test_lists_that_wrap_in_several_blocks_of_rows(fz):
    """256 rows over more kept slots than the list holds: every block of rows scans again
    for its second pass."""
    rng = np.random.default_rng(9)
    c = _random_cache(8, 1, 1, 128, 60, 2)
    c["k_scale"][:] = 2.0 ** -8
    Q = base._rows(rng, (1, 4, 64, 128), "bf16", 0.2)
    base._check_attention(fz, c, Q, rng.integers(0, 2, (1, 1, 64)).astype(np.int32), 2, 30, "bf16")


ALL_FORMS = FORMS + [(4, 128, 64)]


@pytest.mark.parametrize("G,d,T", ALL_FORMS)
def test_bad_pages_and_lengths_in_every_form(fz, G, d, T):
    """A bad page's slots are skipped, a bad count is clamped, both are flagged; the other
    sequence's outputs, lse and mass are the oracle's."""
    import torch
    n, w, H_kv = 333, 20, 2
    c = base._make(7, 2, H_kv, d, [n, n], 2, 1)
    c["mass"][:] = 0
    rng = np.random.default_rng(1)
    Q = base._rows(rng, (2, G * H_kv, T, d), "bf16", 0.2)
    gid = rng.integers(0, 2, (2, 1, T)).astype(np.int32)
    p = fz.make_params(2, G * H_kv, H_kv, T, d, 64, 64, 2, 1, w)
    without = cr.copy(c)
    without["gid"][c["table"][0, 1]] = 2                      # nobody keeps that page's slots
    for page, ln in ((-5, None), (1 << 30, None), (None, 1 << 20), (None, -3)):
        broken = cr.copy(c)
        if page is not None:
            broken["table"][0, 1] = page
        if ln is not None:
            broken["len"][0, 1] = ln
        cache = base._cache(fz, broken)
        ws = fz.alloc_workspace_cache(p, cache)
        O = torch.zeros((2, G * H_kv, T, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((2, G * H_kv, T), device="cuda")
        fz.focus_cache_attention_fwd(p, base._dev(Q, torch.bfloat16), base._dev(gid), cache, O, lse, ws, accumulate=True)
        assert fz.focus_check_errors(ws) == 7
        ref = cr.attention(without if page is not None else c, Q, gid, w, p.scale)
        ds, r, _ = base._bounds(ref, d, "bf16")
        sound = (0, 1) if page is not None else (1,)
        mass, off = cache.mass.cpu().numpy(), lse.cpu().numpy() - ref["lse"]
        for b in sound:
            base._o_within(O, ref, d, "bf16", there=b)
            assert (np.abs(off[b]) <= ds[b] + ref["kept"][b] * 2 * U + 2.0 ** -22 * (1 + np.abs(ref["lse"][b]))).all()
            for h in range(H_kv):
                at = c["table"][b, :-(-n // 64)], h
                assert (np.abs(mass[at] - ref["got"][at]) <= r.max() * ref["got"][at] + 2.0 ** -23 * mass[at]).all()


@pytest.mark.parametrize("G,d,T", ALL_FORMS)
def test_attention_writes_stay_inside_their_buffers_in_every_form(fz, G, d, T):
    """O, lse, mass and the workspace sit between guard bytes, the last tile is partial."""
    import torch
    from test_gpu_canary import Guarded
    B, H_kv, w = 2, 2, 10
    c = base._make(51, B, H_kv, d, [333, 63], 3, 1, spare=0)
    c["mass"][:] = 0
    mass = Guarded(c["mass"].shape, torch.float32, base._dev(c["mass"]))
    cache = fz.Cache(**{k: mass.t if k == "mass" else base._dev(c[k]) for k in base.NAMES})
    p = fz.make_params(B, G * H_kv, H_kv, T, d, 64, 64, 3, 1, w)
    ws = Guarded((fz.focus_cache_workspace_bytes(p, cache),), torch.uint8)
    fz.focus_workspace_init(ws.t)
    rng = np.random.default_rng(2)
    q = base._dev(base._rows(rng, (B, G * H_kv, T, d), "bf16"), torch.bfloat16)
    gid = base._dev(rng.integers(0, 3, (B, 1, T)).astype(np.int32))
    O, lse = Guarded(q.shape, torch.bfloat16), Guarded(q.shape[:3], torch.float32)
    fz.focus_cache_attention_fwd(p, q, gid, cache, O.t, lse.t, ws.t, accumulate=True)
    assert fz.focus_check_errors(ws.t) == 0
    for x in (mass, ws, O, lse):
        assert x.intact()


@pytest.mark.parametrize("G,d,dtype", [(2, 64, "bf16"), (4, 128, "bf16"), (1, 128, "f32")])
def test_a_long_chunk_goes_in_by_turns(fz, G, d, dtype):
    """150 tokens behind prefixes of 70 and 0: appends and attentions of 64, 64 and 22 give
    every token the oracle's output over the whole."""
    import torch
    rng = np.random.default_rng(d + G)
    B, H_kv, n, K, w = 2, 2, 150, 3, 25
    c = base._make(3, B, H_kv, d, [70, 0], K, 1, dtype, room=n)
    k, v = (base._rows(rng, (B, H_kv, n, d), dtype, 0.3) for _ in range(2))
    Q, gid = base._rows(rng, (B, G * H_kv, n, d), dtype, 0.3), rng.integers(0, K, (B, 1, n)).astype(np.int32)
    cache, dt = base._cache(fz, c), base._type(fz, dtype)
    for t in range(0, n, 64):
        m = min(64, n - t)
        p = fz.make_params(B, G * H_kv, H_kv, m, d, 64, 64, K, 1, w, dtype=dtype)
        part = [np.ascontiguousarray(x[:, :, t:t + m]) for x in (k, v, Q, gid)]
        ws = fz.alloc_workspace_cache(p, cache)
        O = torch.zeros((B, G * H_kv, m, d), dtype=dt, device="cuda")
        ids = base._dev(part[3])
        fz.focus_cache_append(p, base._dev(part[0], dt), base._dev(part[1], dt), ids, cache, ws)
        fz.focus_cache_attention_fwd(p, base._dev(part[2], dt), ids, cache, O, None, ws)
        assert fz.focus_check_errors(ws) == 0
        c = cr.append(c, part[0], part[1], part[3])
        base._o_within(O, cr.attention(c, part[2], part[3], w, p.scale), d, dtype)
    assert (cache.len.cpu().numpy() == c["len"]).all() and c["len"].min() == n


# ----------------------------------------------------------------- set-up ---

PREFILL_FIRST = """
import sys
import time
import torch
sys.path.insert(0, {root!r})
from learned_group_sparse_focus_gb300 import focus as fz
bf = torch.bfloat16
p = fz.make_params(1, 4, 2, 256, 64, 64, 32, 4, 1, 16)
h, W, C = (torch.zeros(s, dtype=bf, device="cuda") for s in ((1, 256, 64), (1, 32, 64), (1, 4, 32)))
gid = torch.zeros((1, 1, 256), dtype=torch.int32, device="cuda")
ws = fz.alloc_workspace(p)
fz.focus_assign(p, h, W, C, gid, ws)
q = fz.make_params(1, 4, 2, 4, 64, 64, 32, 4, 1, 16)
cache = fz.alloc_cache(q, 512)
wc = fz.alloc_workspace_cache(q, cache)
Q = torch.zeros((1, 4, 4, 64), dtype=bf, device="cuda")
O, ids = torch.zeros_like(Q), gid[:, :, :4].contiguous()
took = []
for _ in range(20):
    torch.cuda.synchronize()
    start = time.perf_counter()
    fz.focus_cache_attention_fwd(q, Q, ids, cache, O, None, wc)
    took.append(time.perf_counter() - start)
print(took[0] / sorted(took)[10])
"""


def test_the_prefill_does_not_set_up_the_cache_kernels():
    """The cache's kernels are loaded and asked for their cluster figures by the first call
    that launches them: it takes many times a later call's time on the host, also where
    the process has already run the prefill."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", PREFILL_FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
    assert float(done.stdout) > 6, done.stdout
