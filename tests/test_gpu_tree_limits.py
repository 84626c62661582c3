"""Drafted trees and rotary appends at the edges of what their documentation allows: guard
zones, first calls under capture, threads, pools past 4 GiB, positions past 32 bits, many rows a
head, many sequences."""
import numpy as np
import pytest

import oracle.cache_ref as cr
import oracle.tree_ref as tr
from test_gpu_cache import NAMES, _cache, _dev, _make, _params, _rows, _type
from test_gpu_rotary import _freq, _random_tree, _rot
from test_gpu_tree import _check, _draft, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fz():
    from learned_group_sparse_focus_gb300 import focus
    return focus


def _step(fz, seed, G=4, d=128, T=12, dtype="bf16"):
    """One speculative step as a callable, the workspaces and what it left."""
    import torch
    rng = np.random.default_rng(seed)
    B, H_kv, K = 2, 2, 3
    c = _make(seed, B, H_kv, d, [100, 63], K, 1, dtype, room=T)
    Q, Kd, Vd, gid, parent = _draft(rng, B, G * H_kv, H_kv, T, d, K, 1, dtype)
    p, dt = _params(fz, B, G, H_kv, T, d, K, 1, 9, dtype), _type(fz, dtype)
    q, k, v, g, par = _dev(Q, dt), _dev(Kd, dt), _dev(Vd, dt), _dev(gid), _dev(parent)
    token, target = (_dev(rng.integers(0, 2, (B, T)).astype(np.int32)) for _ in range(2))
    prev = _dev(np.zeros(B, np.int32))
    last, count, rows = torch.zeros_like(prev), torch.zeros_like(prev), torch.zeros_like(par)
    start, cache, rot = _cache(fz, c), _cache(fz, c), _rot(fz, _freq(d))
    qr, kr, O = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q)
    lse = torch.zeros(q.shape[:3], device="cuda")
    wc, wt = fz.alloc_workspace_cache(p, cache), fz.alloc_workspace_tree(p)

    def run():
        for n in NAMES:                                   # every run begins with the same cache
            getattr(cache, n).copy_(getattr(start, n))
        fz.focus_rotary(p, rot, wt, Q=q, K=k, Q_out=qr, K_out=kr, base=cache.next, parent=par)
        fz.focus_cache_attention_tree_fwd(p, qr, kr, v, g, par, cache, O, lse, wt)
        fz.focus_tree_accept(p, token, target, prev, par, rows, count, last, wt)
        fz.focus_cache_append_rotary(p, rot, k, v, g, cache, wc, rows=rows, n_new=count)

    def out():
        return [x.cpu().clone() for x in (O.float(), lse, qr.float(), rows, count, last, cache.k, cache.v, cache.pos, cache.len, cache.next)]

    return run, (wc, wt), out


def test_two_threads_on_two_streams(fz):
    import threading

    import torch
    jobs = [_step(fz, 2), _step(fz, 3, 2, 64, 20), _step(fz, 4, 1, 64, 5, "f32")]
    want = []
    for run, _, out in jobs:
        run()
        want.append(out())

    def work(run):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
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
        assert all(fz.focus_check_errors(x) == 0 for x in ws)
        assert all(torch.equal(a, b) for a, b in zip(out(), w))


FIRST_CALL = """
import sys
import torch
sys.path[:0] = [{root!r}, {tests!r}]
from learned_group_sparse_focus_gb300 import focus as fz
import test_gpu_tree_limits as t
for args in ((1,), (2, 2, 64, 20), (3, 2, 64, 5, "f32")):
    run, ws, out = t._step(fz, *args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    g.replay()
    torch.cuda.synchronize()
    a = out()
    run()
    assert all(fz.focus_check_errors(x) == 0 for x in ws) and a[0].abs().max() > 0
    assert all(torch.equal(x, y) for x, y in zip(a, out()))
"""


def test_a_process_may_capture_its_first_calls():
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL.format(root=os.path.dirname(tests), tests=tests)
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


@pytest.mark.parametrize("dtype,d,dim,T", [("bf16", 128, 64, 70), ("f32", 64, 64, 5), ("bf16", 64, 16, 1)])
def test_rotary_writes_stay_inside_their_buffers(fz, dtype, d, dim, T):
    import torch
    from test_gpu_canary import Guarded
    B, G, H_kv, K = 2, 3, 2, 3
    c = _make(51, B, H_kv, d, [130, 63], K, 1, dtype, spare=8, room=T)
    g = {k: Guarded(c[k].shape, _dev(c[k]).dtype, _dev(c[k])) for k in NAMES}
    cache = fz.Cache(**{k: x.t for k, x in g.items()})
    p, dt = _params(fz, B, G, H_kv, T, d, K, 1, 10, dtype), _type(fz, dtype)
    ws = Guarded((fz.focus_cache_workspace_bytes(p, cache),), torch.uint8)
    fz.focus_workspace_init(ws.t)
    rng = np.random.default_rng(1)
    q, k, v = (_dev(_rows(rng, (B, h, T, d), dtype), dt) for h in (G * H_kv, H_kv, H_kv))
    gid = _dev(rng.integers(0, K, (B, 1, T)).astype(np.int32))
    rot = _rot(fz, _freq(dim))
    outs = [Guarded(x.shape, dt) for x in (q, k, q, k)]
    fz.focus_cache_append_rotary(p, rot, k, v, gid, cache, ws.t, Q=q, Q_out=outs[0].t, K_out=outs[1].t)
    fz.focus_rotary(p, rot, ws.t, Q=q, K=k, Q_out=outs[2].t, K_out=outs[3].t)
    ints = [Guarded((B, T) if i == 0 else (B,), torch.int32) for i in range(3)]
    if T <= 64:
        z = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        fz.focus_tree_accept(p, z, z, z[:, 0].contiguous(), _dev(_random_tree(rng, B, T)), *[x.t for x in ints], ws.t)
    assert fz.focus_check_errors(ws.t) == 0
    for x in (*g.values(), ws, *outs, *ints):
        assert x.intact()


@pytest.mark.parametrize("H,T", [(4, 4), (8, 20)])
def test_pages_past_four_gigabytes_of_a_pool(fz, H, T):
    """The same calls over the last pages of a 5 GB pool and over a small pool: same bits."""
    import torch
    B, H_kv, d, K, w, n = 2, 2, 128, 3, 20, 700
    p, q = (fz.make_params(B, H, H_kv, m, d, 64, 64, K, 1, w) for m in (n, T))
    rng = np.random.default_rng(H)
    bf, mp = torch.bfloat16, -(-(n + T) // 64)
    k, v = (_dev(_rows(rng, (B, H_kv, n, d), "bf16"), bf) for _ in range(2))
    k1, v1 = (_dev(_rows(rng, (B, H_kv, T, d), "bf16"), bf) for _ in range(2))
    Q = _dev(_rows(rng, (B, H, T, d), "bf16", 0.3), bf)
    gid, gid1 = (_dev(rng.integers(0, K, (B, 1, m)).astype(np.int32)) for m in (n, T))
    parent, rot = _dev(_random_tree(rng, B, T)), _rot(fz, _freq(d))
    outs = []
    for pages in (64, 5 * 2 ** 30 // (H_kv * 64 * d)):
        def pool(shape, dtype):
            return torch.zeros((pages, H_kv) + shape, dtype=dtype, device="cuda")

        part = dict(k=pool((64, d), torch.uint8), v=pool((64, d), torch.uint8), k_scale=pool((), torch.float32),
                    v_scale=pool((), torch.float32), pos=pool((64,), torch.int32), gid=pool((64,), torch.int16),
                    mass=pool((64,), torch.float32))
        table = torch.arange(pages - B * mp, pages, dtype=torch.int32, device="cuda").flip(0).reshape(B, mp)
        cache = fz.Cache(**part, table=table, len=torch.zeros((B, H_kv), dtype=torch.int32, device="cuda"),
                         next=torch.zeros((B,), dtype=torch.int32, device="cuda"))
        ws, wt = fz.alloc_workspace_cache(p, cache), fz.alloc_workspace_tree(q)
        fz.focus_cache_append_rotary(p, rot, k, v, gid, cache, ws)
        O, lse = torch.zeros_like(Q), torch.zeros(Q.shape[:3], device="cuda")
        fz.focus_cache_attention_tree_fwd(q, Q, k1, v1, gid1, parent, cache, O, lse, wt)
        assert fz.focus_check_errors(ws) == 0 and fz.focus_check_errors(wt) == 0
        tail = {m: x[pages - 60:].cpu() for m, x in part.items()}
        outs.append([O.float().cpu(), lse.cpu(), cache.len.cpu(), *tail.values()])
        if len(outs) == 2:                               # nothing was written below those pages
            assert not any(part[m][:pages - 60].view(-1)[::7].any() for m in ("k", "v", "k_scale", "pos"))
    assert outs[0][0].abs().max() > 0
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("G,T", [(2, 4), (4, 20)])
def test_positions_that_would_pass_32_bits_are_flagged(fz, G, T):
    rng = np.random.default_rng(5)
    c = _make(6, 2, 1, 128, [100, 100], 3, 1)
    Q, Kd, Vd, gid, parent = _draft(rng, 2, G, 1, T, 128, 3, 1, "bf16", "chain")
    _, _, ws, want, _ = _run(fz, c, Q, Kd, Vd, gid, parent, 3, 9, "bf16")
    assert fz.focus_check_errors(ws) == 0
    for bad in ((1 << 31) - 1 - T + 1, -1):
        c2 = cr.copy(c)
        c2["next"][0] = bad
        _, _, ws, O, _ = _run(fz, c2, Q, Kd, Vd, gid, parent, 3, 9, "bf16")
        assert fz.focus_check_errors(ws) == 7 and (O[1] == want[1]).all()


@pytest.mark.parametrize("G,d,T,lens", [(96, 128, 3, [200]), (33, 64, 2, [70, 0]), (128, 128, 1, [130])])
def test_many_query_heads_a_head(fz, G, d, T, lens):
    rng = np.random.default_rng(G)
    B = len(lens)
    c = _make(G, B, 1, d, lens, 3, 1)
    Q, Kd, Vd, gid, parent = _draft(rng, B, G, 1, T, d, 3, 1, "bf16")
    _check(fz, c, Q, Kd, Vd, gid, parent, 3, 40, "bf16")


@pytest.mark.parametrize("d,G,T", [(64, 1, 3), (128, 6, 4)])
def test_more_sequences_than_blocks_at_once(fz, d, G, T):
    rng = np.random.default_rng(d)
    B = 200
    lens = rng.integers(0, 130, B)
    c = _make(d, B, 1, d, lens, 4, 1)
    Q, Kd, Vd, gid, parent = _draft(rng, B, G, 1, T, d, 4, 1, "bf16")
    n_new = rng.integers(0, T + 1, B).astype(np.int32)
    _check(fz, c, Q, Kd, Vd, gid, parent, 4, 11, "bf16", n_new=n_new)


def test_no_node_at_all(fz):
    rng = np.random.default_rng(9)
    for G, T in ((2, 5), (4, 30)):
        c = _make(9, 2, 2, 128, [100, 64], 3, 1)
        Q, Kd, Vd, gid, parent = _draft(rng, 2, 2 * G, 2, T, 128, 3, 1, "bf16")
        _check(fz, c, Q, Kd, Vd, gid, parent, 3, 9, "bf16", n_new=np.zeros(2, np.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_drafted_rows(fz, dtype):
    """Smallest and largest keys, queries and values beside ordinary ones."""
    rng = np.random.default_rng(10)
    for G, T in ((2, 6), (4, 12)):
        c = _make(11, 1, 1, 128, [90], 2, 1, dtype)
        Q, Kd, Vd, gid, parent = _draft(rng, 1, G, 1, T, 128, 2, 1, dtype, "star")
        Q[0, 0] *= 2.0 ** -60
        Q[0, 1] *= 2.0 ** 20
        Kd[0, 0, 0] *= 2.0 ** -40
        Kd[0, 0, 2] *= 2.0 ** -21
        Kd[0, 0, 3] = 0.0
        Vd[0, 0, 1] *= 2.0 ** 100
        Vd[0, 0, 4] = 0.0
        _check(fz, c, Q, Kd, Vd, gid, parent, 2, 5, dtype)


def test_gid_outside_the_groups_matches_nothing_cached(fz):
    rng = np.random.default_rng(12)
    for G, T in ((2, 4), (4, 10)):
        c = _make(13, 1, 1, 128, [200], 3, 1)
        Q, Kd, Vd, gid, parent = _draft(rng, 1, G, 1, T, 128, 3, 1, "bf16")
        gid[0, 0, 1], gid[0, 0, 2] = 5000, -3
        _check(fz, c, Q, Kd, Vd, gid, parent, 3, 2, "bf16")


@pytest.mark.parametrize("size", [0, 6, 12, 18, 40])
def test_weights_of_huge_logits_still_sum_to_one(fz, size):
    """Values are all one, so outputs are, however large the logits and their rounding: off by bf16's half
    step, and 2^-12 for the weights' and the sum's roundings."""
    import torch
    rng = np.random.default_rng(21)
    G, T, d = 4, 12, 128
    for shape in ("star", "chain"):
        for lens in ([0], [100]):
            c = _make(22, 1, 1, d, lens, 2, 1)
            Q, Kd, Vd, gid, parent = _draft(rng, 1, G, 1, T, d, 2, 1, "bf16", shape)
            Q, Kd = Q * 2.0 ** (size + 4), Kd * 2.0 ** size
            p, cache = _params(fz, 1, G, 1, T, d, 2, 1, 9, "bf16"), _cache(fz, c)
            cache.v.copy_(torch.ones_like(cache.v, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8))
            cache.v_scale.fill_(1.0)
            q, k = _dev(Q, torch.bfloat16), _dev(Kd, torch.bfloat16)
            O, lse, ws = torch.zeros_like(q), torch.zeros(1, G, T, device="cuda"), fz.alloc_workspace_tree(p)
            fz.focus_cache_attention_tree_fwd(p, q, k, torch.ones_like(k), _dev(gid), _dev(parent), cache, O, lse, ws)
            assert fz.focus_check_errors(ws) == 0 and torch.isfinite(lse).all()
            assert ((O.float() - 1).abs() <= 2.0 ** -8 + 2.0 ** -12).all()
