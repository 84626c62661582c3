"""Attention over the paged cache at the ends of its contract, against the fp64
oracle: the bits that the softmax weights keep.  Bounds are those of
test_gpu_cache.py; where one is tighter, the test derives it.
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
