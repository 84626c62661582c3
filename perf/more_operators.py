"""Decoding several tokens a step with drafted trees and rotary positions: the
cases that are measured.

Four operators beside the paged 8-bit key/value cache:

  append   new keys are rotated to their positions and quantised into the cache's
           pages with their values, in one call that also rotates the queries (and
           may write the rotated keys, which a prompt's own attention reads);
           with `rows`, the appended tokens are picked from a drafted tree.
  rotary   the rotation alone, of the nodes of a drafted tree, and its transpose,
           which is the rotation's gradient.
  tree     attention of the nodes of a drafted tree over the cached slots that the
           keep rule leaves and over each node's ancestors, whose keys and values
           are not in the cache.
  accept   the accepted path of a drafted tree, its length and the next choice.

A cache page holds 64 slots of one sequence.  Per page and key/value head: e4m3
codes of K and V, one power-of-two scale for each, and per slot the token's
position, group id and accumulated attention weight.  `table` lists a
sequence's pages, `len` the slots in use per head (heads differ after an
eviction), `next` the position that the next token gets.  A tree's node t hangs
below node parent[t] < t, or below the last cached token (-1); its position is
next + its depth.

`run` computes a case in plain torch operations, or, with `own` set, through
learned_group_sparse_focus_gb300.focus.
"""
import math

import torch

own = False

PAGE = 64
MIN_EXP = -64          # smallest scale exponent of a page


# ------------------------------------------------------------------ cases ---

def _case(name, op, B, H, H_kv, d, n, T, **more):
    c = dict(name=name, op=op, B=B, H=H, H_kv=H_kv, d=d, n=n, T=T, K=64, w=512, A=1, dtype="bf16", groups="zipf",
             ragged=False, evicted=False, pad=False, first=0, tree="random", theta=10000.0, dim=d, interleaved=False,
             factor=1.0, queries=True, keys_out=False, path=False, transpose=False, V=8)
    c.update(more)
    return c


def listed():
    return [
        # the append of one decode step of a serving batch, queries rotated in the same call: latency
        _case("append_step", "append", 16, 32, 8, 128, 8192, 1, ragged=True, theta=500000.0),
        # a right-padded chunk behind a cached prefix of a model that rotates half of each head, in neighbouring pairs
        _case("append_chunk", "append", 4, 32, 32, 128, 1500, 777, K=32, w=256, ragged=True, pad=True, dim=64,
              interleaved=True, keys_out=True),
        # a whole 32K prompt of the GQA layer; the prompt's attention reads the rotated keys as well
        _case("append_prompt_32k", "append", 1, 32, 8, 128, 0, 32768, theta=500000.0, keys_out=True),
        # the accepted nodes of trees of 64, picked by row, for a batch of long sequences
        _case("append_accepted", "append", 16, 32, 8, 128, 16384, 64, ragged=True, path=True, pad=True, queries=False),
        # queries and keys of drafted trees of an fp32 model, at positions past a million
        _case("rotary_tree_f32", "rotary", 8, 64, 8, 128, 1, 64, dtype="f32", first=1 << 20, pad=True),
        # the gradient with respect to the queries and keys of two sequences of 8K tokens
        _case("rotary_grad_8k", "rotary", 2, 32, 32, 128, 0, 8192, transpose=True, tree="chain"),
        # sixteen drafted nodes for each of eight short sequences of a small model
        _case("tree_small", "tree", 8, 12, 12, 64, 1024, 16, K=16, w=64, groups="uniform", ragged=True),
        # sixteen drafted nodes for one user at 32K tokens
        _case("tree_32k", "tree", 1, 32, 8, 128, 32768, 16),
        # trees of up to 64 nodes for a serving batch at up to 32K tokens
        _case("tree_batch", "tree", 16, 32, 8, 128, 32768, 64, ragged=True, pad=True),
        # an fp32 model over a cache that was evicted from: heads of different lengths, gaps in the positions
        _case("tree_f32", "tree", 3, 6, 3, 64, 777, 7, K=5, w=33, A=3, dtype="f32", ragged=True, evicted=True),
        # one user's tree: the launch itself
        _case("accept_one", "accept", 1, 1, 1, 64, 0, 16),
        # trees of up to 64 nodes for a large batch, several nodes with the same token among them
        _case("accept_batch", "accept", 512, 1, 1, 64, 0, 64, pad=True, V=3),
    ]


def draw(rng):
    def lg(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(("append", "rotary", "tree", "tree", "accept"))
    H_kv = rng.choice((1, 2, 3, 4, 8, 12, 32))
    G = rng.choice((1, 2, 4, 8))
    d = rng.choice((64, 128))
    n = rng.choice((0, lg(1, 65536), lg(1, 65536), lg(1, 65536)))
    B = min(rng.randint(1, 16), max(1, (1 << 21) // (max(n, 1) * H_kv)))
    n = min(n, (1 << 21) // H_kv)
    more = dict(dtype=rng.choice(("bf16", "bf16", "bf16", "f32")), groups=rng.choice(("zipf", "uniform")),
                ragged=rng.random() < 0.5, evicted=rng.random() < 0.4, pad=rng.random() < 0.4, K=lg(1, 512),
                w=lg(1, 1024), A=rng.choice((1, H_kv)), tree=rng.choice(("random", "random", "chain")),
                first=rng.choice((0, lg(1, 1 << 24))))
    if op in ("append", "rotary"):
        more.update(theta=rng.choice((10000.0, 500000.0)), dim=rng.choice((16, d // 2, d, d)),
                    interleaved=rng.random() < 0.4, factor=rng.choice((1.0, 1.0, 1.1387)))
    if op == "append":
        more["path"] = rng.random() < 0.3
        T = rng.randint(1, 64) if more["path"] else rng.choice((1, lg(1, 8192)))
        T = max(1, min(T, (1 << 18) // (B * G * H_kv)))
        more["queries"] = not more["path"] and rng.random() < 0.7
        more["keys_out"] = not more["path"] and rng.random() < 0.5
    elif op == "rotary":
        more["transpose"] = rng.random() < 0.5
        T = rng.randint(1, 64) if more["tree"] == "random" else lg(1, 16384)
        T = max(1, min(T, (1 << 19) // (B * G * H_kv)))
    elif op == "tree":
        T = rng.choice((1, rng.randint(1, 16), rng.randint(1, 64)))
        T = max(1, min(T, (1 << 26) // (B * H_kv * max(n, 64) * G)))
    else:
        T, B, n = rng.randint(1, 64), lg(1, 1024), 0
        more["V"] = rng.choice((2, 3, 8))
    c = _case("", op, B, G * H_kv, H_kv, d, n, T, **more)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs ---

def _need_exp(amax):
    """Least e >= MIN_EXP with amax <= 448 * 2^e, for finite amax >= 0 (exact)."""
    f, x = torch.frexp(amax)                                   # amax = f 2^x, f in [0.5, 1)
    e = torch.where(f > 0.875, x - 8, x - 9)                   # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp_(min=MIN_EXP)


def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127], exact: the exponent's bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(gen, shape):
    """Codes and scales of N(0, 1) rows, page by page: [.., PAGE, d] -> uint8, fp32 [..]."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).float()
    s = _pow2(_need_exp(x.abs().amax(dim=(-1, -2))))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def _cache(case, gen, rand, room):
    """A filled cache whose pages lie anywhere in the pool, and the group ids of every position."""
    B, H_kv, d, K, A, n, first = (case[x] for x in ("B", "H_kv", "d", "K", "A", "n", "first"))
    dev = "cuda"
    # slots in use: [B, H_kv], ragged over sequences, and over heads where slots were evicted
    lens = torch.full((B, H_kv), n, dtype=torch.int32, device=dev)
    if case["ragged"]:
        lens = (n - (rand(B, 1) * 0.75 * n).int()).int().expand(B, H_kv).contiguous()
    if case["evicted"]:
        lens = torch.maximum(lens - (rand(B, H_kv) * 0.25 * lens).int(), lens.clamp(max=1)).int()
    max_pages = max(1, -(-(n + room) // PAGE))
    cap = max_pages * PAGE
    # positions rise along the slots; an evicted cache has gaps in all but its last 256 slots
    slot = torch.arange(cap, device=dev)
    inc = torch.ones((B, H_kv, cap), dtype=torch.int64, device=dev)
    if case["evicted"]:
        inc += torch.where(slot < lens[..., None] - 256, (-2.0 * torch.log(1.0 - rand(B, H_kv, cap))).long(), 0)
    live = slot < lens[..., None]
    run_up = torch.where(live, inc, 0).cumsum(-1)
    total = run_up[..., -1]
    span = total.amax(1)                                                       # [B] positions since `first`
    rel = torch.where(live, span[:, None, None] - total[..., None] + run_up - 1, 0)
    # group ids by position, one assignment for all heads or one a head
    far = (int(span.max()) if n else 0) + case["T"] + 1
    p = torch.arange(1, K + 1, device=dev, dtype=torch.float32) ** (-1.1 if case["groups"] == "zipf" else 0.0)
    cdf = (p / p.sum()).cumsum(0)
    ids = torch.randperm(K, generator=gen, device=dev)
    of_token = ids[torch.searchsorted(cdf, rand(B, A, far)).clamp_(max=K - 1)].int()
    gid = torch.gather(of_token.expand(B, H_kv, far), 2, rel).short()
    n_pages = B * max_pages
    table = torch.randperm(n_pages, generator=gen, device=dev).int().view(B, max_pages)
    c = dict(k=torch.empty((n_pages, H_kv, PAGE, d), dtype=torch.uint8, device=dev),
             v=torch.empty((n_pages, H_kv, PAGE, d), dtype=torch.uint8, device=dev),
             k_scale=torch.empty((n_pages, H_kv), device=dev), v_scale=torch.empty((n_pages, H_kv), device=dev))
    step = max(1, (1 << 26) // (H_kv * PAGE * d))
    for a in range(0, n_pages, step):
        b = min(n_pages, a + step)
        for x in ("k", "v"):
            c[x][a:b], c[x + "_scale"][a:b] = _codes(gen, (b - a, H_kv, PAGE, d))
    at = table.long().view(-1)

    def spread(x):
        out = torch.empty((n_pages, H_kv, PAGE), dtype=x.dtype, device=dev)
        out[at] = x.view(B, H_kv, max_pages, PAGE).transpose(1, 2).reshape(n_pages, H_kv, PAGE)
        return out

    # weight that a key has gathered: long-tailed, none for two keys in five
    mass = torch.exp(2.0 * torch.randn((B, H_kv, cap), generator=gen, device=dev)) * (rand(B, H_kv, cap) > 0.4) * live
    c.update(pos=spread(torch.where(live, rel + first, 0).int()), gid=spread(gid), mass=spread(mass), table=table,
             len=lens, next=(span + first).int())
    return c, of_token, span


def prepare(case, seed):
    B, H, H_kv, d, A, T = (case[x] for x in ("B", "H", "H_kv", "d", "A", "T"))
    op, dev = case["op"], "cuda"
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt)

    s = dict(case=case, scale=1.0 / math.sqrt(d))
    s["n_new"] = (1 + (rand(B) * T).int()).clamp_(max=T).int() if case["pad"] else None
    # a node hangs below any node before it, each as likely (so depths grow as log T), or below the one before
    s["parent"] = None
    if op in ("tree", "accept") or (op == "rotary" and case["tree"] == "random"):
        t = torch.arange(T, device=dev)
        up = (rand(B, T) * t).int().clamp_(max=T - 1)
        up = torch.where(rand(B, T) < 0.1, -1, up).int() if case["tree"] == "random" else (t - 1).int().expand(B, T)
        s["parent"] = torch.where(t == 0, -1, up).int().contiguous()
    if op == "accept":
        # a drafted token is often the one that the model chose after its parent
        s["target"] = torch.randint(0, case["V"], (B, T), generator=gen, device=dev, dtype=torch.int32)
        s["prev"] = torch.randint(0, case["V"], (B,), generator=gen, device=dev, dtype=torch.int32)
        after = torch.where(s["parent"] < 0, s["prev"][:, None], torch.gather(s["target"], 1, s["parent"].clamp(min=0).long()))
        other = torch.randint(0, case["V"], (B, T), generator=gen, device=dev, dtype=torch.int32)
        s["token"] = torch.where(rand(B, T) < 0.7, after, other).int()
        s["rows"] = torch.full((B, T), -1, dtype=torch.int32, device=dev)
        s["count"], s["last"] = torch.empty_like(s["prev"]), torch.empty_like(s["prev"])
        return s
    i = torch.arange(case["dim"] // 2, device=dev, dtype=torch.float64)
    s["inv_freq"] = (case["theta"] ** (-2.0 * i / case["dim"])).float()
    if op == "rotary":
        s["Q"], s["K"] = normal(B, H, T, d), normal(B, H_kv, T, d)
        s["Q_out"], s["K_out"] = torch.zeros_like(s["Q"]), torch.zeros_like(s["K"])
        s["base"] = (case["first"] + (rand(B) * max(case["n"], 1)).int()).int()
        return s
    cache, of_token, span = _cache(case, gen, rand, T if op == "append" else 0)
    s["cache"] = cache
    s["K"], s["V"] = normal(B, H_kv, T, d), normal(B, H_kv, T, d)
    where = (span[:, None] + torch.arange(T, device=dev)).expand(B, T)
    s["gid"] = torch.gather(of_token, 2, where[:, None].expand(B, A, T)).contiguous()
    if op == "append":
        s["len"], s["next"] = torch.empty_like(cache["len"]), torch.empty_like(cache["next"])
        s["rows"] = None
        if case["path"]:
            # an accepted path rises through the tree; few of many drafted nodes are accepted
            if case["pad"]:
                s["n_new"] = (1 + (rand(B) ** 3 * T).int()).clamp_(max=T).int()
            m = torch.full((B,), T, device=dev) if s["n_new"] is None else s["n_new"]
            order = rand(B, T).argsort(1)
            taken = torch.where(torch.arange(T, device=dev) < m[:, None], order, T).sort(1).values
            s["rows"] = torch.where(taken < T, taken, 0).int()
        s["Q"] = normal(B, H, T, d) if case["queries"] else None
        s["Q_out"] = torch.zeros_like(s["Q"]) if case["queries"] else None
        s["K_out"] = torch.zeros_like(s["K"]) if case["keys_out"] else None
    else:
        s["Q"] = normal(B, H, T, d)
        s["O"] = torch.zeros_like(s["Q"])
        s["lse"] = torch.zeros((B, H, T), device=dev)
    return s


# ------------------------------------------------------------ plain forms ---

def _fresh(s):
    c = s["case"]
    return torch.full((c["B"],), c["T"], dtype=torch.int32, device="cuda") if s["n_new"] is None else s["n_new"]


def _lineage(parent):
    """[B, T, T]: whether node j is node t or one of its ancestors."""
    B, T = parent.shape
    node = torch.arange(T, device=parent.device)
    up = (parent[..., None] == node).float()                   # one step towards the root
    up = up + torch.eye(T, device=parent.device)
    return torch.matrix_power(up, T) > 0                       # counts of walks, all of them at least 0


def _rotate(x, at, s, transpose=False):
    """Rows x [B, h, T, d] turned to positions `at` [B, T], in x's own precision; angles in 64 bits."""
    c = s["case"]
    r = c["dim"]
    angle = at.double()[..., None] * s["inv_freq"].double()                    # [B, T, r / 2]
    cos, sin = ((f(angle) * c["factor"]).to(x.dtype)[:, None] for f in (torch.cos, torch.sin))
    if transpose:
        sin = -sin
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _put(out, x, there):
    """Rows of valid tokens into out, rounded once; the others stay."""
    out.copy_(torch.where(there[:, None, :, None], x.to(out.dtype), out))


def _plain_rotary(s):
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    depth = t if s["parent"] is None else _lineage(s["parent"]).sum(-1) - 1
    at = s["base"][:, None] + depth
    there = t < _fresh(s)[:, None]
    _put(s["Q_out"], _rotate(s["Q"].float(), at, s, c["transpose"]), there)
    _put(s["K_out"], _rotate(s["K"].float(), at, s, c["transpose"]), there)


def _rows(x, table):
    """[n_pages, H_kv, PAGE, ...] -> [B, H_kv, slots, ...] through the table."""
    y = x[table.long()].transpose(1, 2)
    return y.reshape(y.shape[0], y.shape[1], -1, *y.shape[4:])


def _values(x, scale, table):
    y = x.view(torch.float8_e4m3fn)[table.long()].float() * scale[table.long()][..., None, None]
    y = y.transpose(1, 2)
    return y.reshape(y.shape[0], y.shape[1], -1, y.shape[-1])


def _quantise(x, e):
    """x [.., PAGE, d] in 64 bits at page exponents e [..] -> codes, each value rounded once."""
    y = (x * torch.exp2(-e.double())[..., None, None]).clamp(-448.0, 448.0)
    step = torch.exp2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].double() - 4)
    return (torch.round(y / step) * step).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c, T = s["cache"], s["case"]["T"]
    B, H_kv = c["len"].shape
    dev = c["len"].device
    n_new = _fresh(s)
    K, V, gid = s["K"], s["V"], s["gid"]
    if s["rows"] is not None:
        pick = s["rows"].long()
        K, V = (torch.gather(x, 2, pick[:, None, :, None].expand(-1, H_kv, -1, x.shape[-1])) for x in (K, V))
        gid = torch.gather(gid, 2, pick[:, None].expand(-1, gid.shape[1], -1))
    new_at = c["next"].long()[:, None] + torch.arange(T, device=dev)                          # [B, T]
    there = torch.arange(T, device=dev) < n_new[:, None]
    K64 = _rotate(K.double(), new_at, s)          # a rounding border of e4m3 decides a whole step: 64 bits
    if s["Q"] is not None:
        _put(s["Q_out"], _rotate(s["Q"].float(), new_at, s), there)
    if s["K_out"] is not None:
        _put(s["K_out"], K64, there)
    touched = (T + PAGE - 2) // PAGE + 1
    page = c["len"].long()[..., None] // PAGE + torch.arange(touched, device=dev)             # [B, H_kv, touched]
    slot = page[..., None] * PAGE + torch.arange(PAGE, device=dev)                            # [.., PAGE]
    t = slot - c["len"].long()[..., None, None]
    new = (t >= 0) & (t < n_new[:, None, None, None])
    old = t < 0
    used = new.any(-1)
    where = torch.gather(c["table"].long()[:, None].expand(B, H_kv, -1), 2, page.clamp(max=c["table"].shape[1] - 1))
    head = torch.arange(H_kv, device=dev)[None, :, None].expand_as(where)
    tc = t.clamp(0, T - 1)

    def one(x, codes, scale):
        rows = torch.gather(x, 2, tc.view(B, H_kv, -1, 1).expand(-1, -1, -1, x.shape[-1]))
        rows = rows.view(*t.shape, -1) * new[..., None]
        was = codes[where, head]
        e_old = torch.frexp(scale[where, head])[1] - 1
        need = _need_exp(rows.abs().amax(dim=(-1, -2)))
        e = torch.where(old.any(-1), torch.maximum(need, e_old), need)
        kept = was.view(torch.float8_e4m3fn).double() * scale[where, head].double()[..., None, None]
        both = _quantise(torch.where(old[..., None], kept, rows), e)
        codes[where[used], head[used]] = torch.where((new | old)[..., None], both, was)[used]
        scale[where[used], head[used]] = _pow2(e)[used]

    one(K64, c["k"], c["k_scale"])
    one(V.double(), c["v"], c["v_scale"])
    at, h, r = where[..., None].expand_as(t)[new], head[..., None].expand_as(t)[new], (slot % PAGE)[new]
    c["pos"][at, h, r] = (c["next"].long()[:, None, None, None] + t)[new].int()
    ids = gid.expand(B, H_kv, T)
    c["gid"][at, h, r] = torch.gather(ids, 2, tc.view(B, H_kv, -1)).view_as(t)[new].short()
    c["mass"][at, h, r] = 0.0
    s["len"].copy_(c["len"] + n_new[:, None])
    s["next"].copy_(c["next"] + n_new)


def _plain_tree(s):
    c, k = s["cache"], s["case"]
    B, H, T, d = s["Q"].shape
    H_kv, G, w = k["H_kv"], H // k["H_kv"], max(k["w"], 1)
    dev = s["Q"].device
    t = torch.arange(T, device=dev)
    there = t < _fresh(s)[:, None]                                                             # [B, T]
    line = _lineage(s["parent"])
    depth = line.sum(-1) - 1
    i = c["next"][:, None] + depth
    mine = s["gid"].expand(B, H_kv, T)
    pos, gid = _rows(c["pos"], c["table"]), _rows(c["gid"], c["table"])                        # [B, H_kv, S]
    slot = torch.arange(pos.shape[-1], device=dev)
    ahead = i[:, None, :, None] - pos[:, :, None, :]                                           # [B, H_kv, T, S]
    cached = (ahead >= 0) & ((ahead < w) | (mine[..., None] == gid[:, :, None, :])) & (slot < c["len"][:, :, None, None])
    near = (depth[:, None, :, None] - depth[:, None, None, :] < w) | (mine[..., None] == mine[:, :, None, :])
    keep = torch.cat((cached, near & line[:, None]), -1)                                       # [B, H_kv, T, S + T]
    ks = torch.cat((_values(c["k"], c["k_scale"], c["table"]), s["K"].float()), 2)
    vs = torch.cat((_values(c["v"], c["v_scale"], c["table"]), s["V"].float()), 2)
    score = torch.matmul(s["Q"].float().view(B, H_kv, G * T, d), ks.transpose(2, 3))
    score = (score * s["scale"]).view(B, H_kv, G, T, -1).masked_fill(~keep[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)                                 # finite: a node keeps itself
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul((p / total).view(B, H_kv, G * T, -1), vs).view(B, H, T, d)
    _put(s["O"], out, there)
    lse = (top + torch.log(total)).view(B, H, T)
    s["lse"].copy_(torch.where(there[:, None], lse, s["lse"]))


def _plain_accept(s):
    parent, T = s["parent"], s["case"]["T"]
    t = torch.arange(T, device=parent.device)
    after = torch.where(parent < 0, s["prev"][:, None], torch.gather(s["target"], 1, parent.clamp(min=0).long()))
    right = (s["token"] == after) & (t < _fresh(s)[:, None])
    line = _lineage(parent)
    good = (right[:, None, :] | ~line).all(-1)                         # the node and all of its ancestors
    depth = torch.where(good, line.sum(-1), 0)
    best = (depth * T + (T - 1 - t)).argmax(1)                         # the deepest, ties: the lowest index
    count = torch.gather(depth, 1, best[:, None])[:, 0]
    on = torch.gather(line, 1, best[:, None, None].expand(-1, 1, T))[:, 0] & (count > 0)[:, None]
    path = torch.where(on, t, T).sort(1).values                        # a parent comes before its children
    s["rows"].copy_(torch.where(t < count[:, None], path, s["rows"]))
    s["count"].copy_(count)
    s["last"].copy_(torch.where(count > 0, torch.gather(s["target"], 1, best[:, None])[:, 0], s["prev"]))


# -------------------------------------------------------------------- run ---

def _handle(s):
    """What a program keeps between calls: problem description, rotation, cache handle and workspace."""
    from learned_group_sparse_focus_gb300 import focus as fz
    k = s["case"]
    p = fz.make_params(k["B"], k["H"], k["H_kv"], k["T"], k["d"], 64, 64, k["K"], k["A"], k["w"], scale=s["scale"],
                       dtype=k["dtype"])
    rot = None
    if "inv_freq" in s:
        rot = fz.Rotary(s["inv_freq"], interleaved=k["interleaved"], scale=k["factor"])
    if "cache" not in s:
        return fz, p, rot, None, fz.alloc_workspace_tree(p)
    cache = fz.Cache(**s["cache"])
    ws = fz.alloc_workspace_tree(p) if k["op"] == "tree" else fz.alloc_workspace_cache(p, cache)
    return fz, p, rot, cache, ws


def _own(s):
    if "handle" not in s:
        s["handle"] = _handle(s)
    fz, p, rot, cache, ws = s["handle"]
    op = s["case"]["op"]
    if op == "append":
        fz.focus_cache_append_rotary(p, rot, s["K"], s["V"], s["gid"], cache, ws, Q=s["Q"], Q_out=s["Q_out"],
                                     K_out=s["K_out"], rows=s["rows"], n_new=s["n_new"], len_out=s["len"],
                                     next_out=s["next"])
    elif op == "rotary":
        fz.focus_rotary(p, rot, ws, Q=s["Q"], K=s["K"], Q_out=s["Q_out"], K_out=s["K_out"], base=s["base"],
                        parent=s["parent"], n_new=s["n_new"], transpose=s["case"]["transpose"])
    elif op == "tree":
        fz.focus_cache_attention_tree_fwd(p, s["Q"], s["K"], s["V"], s["gid"], s["parent"], cache, s["O"], s["lse"], ws,
                                          n_new=s["n_new"])
    else:
        fz.focus_tree_accept(p, s["token"], s["target"], s["prev"], s["parent"], s["rows"], s["count"], s["last"], ws,
                             n_new=s["n_new"])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        _own(s)
    else:
        {"append": _plain_append, "rotary": _plain_rotary, "tree": _plain_tree, "accept": _plain_accept}[op](s)
    if op == "rotary":
        return dict(Q=s["Q_out"], K=s["K_out"])
    if op == "tree":
        return dict(O=s["O"], lse=s["lse"])
    if op == "accept":
        return dict(rows=s["rows"], count=s["count"], last=s["last"])
    c = s["cache"]
    out = dict(k=c["k"].view(torch.float8_e4m3fn), v=c["v"].view(torch.float8_e4m3fn), k_scale=c["k_scale"],
               v_scale=c["v_scale"], pos=c["pos"], gid=c["gid"], mass=c["mass"], len=s["len"], next=s["next"])
    out.update({x: s[x] for x in ("Q_out", "K_out") if s[x] is not None})
    return out


def work(case):
    B, H, H_kv, d, K, n, T = (case[x] for x in ("B", "H", "H_kv", "d", "K", "n", "T"))
    es, G, w = (2 if case["dtype"] == "bf16" else 4), H // H_kv, max(case["w"], 1)
    new = (T + 1) / 2 if case["pad"] else T
    if case["op"] == "accept":
        return {"bytes": B * (4 * 3 * new + 12), "flops": B * new}
    if case["op"] == "rotary":
        return {"bytes": B * (H + H_kv) * new * 2 * d * es, "flops": 3 * B * (H + H_kv) * new * case["dim"]}
    if case["op"] == "append":
        if case["path"] and case["pad"]:
            new = 1 + T / 4
        bytes_ = B * H_kv * new * (2 * d * es + 2 * d + 4 + 2 + 4 + 4 + (d * es if case["keys_out"] else 0))
        heads = H_kv + (H if case["queries"] else 0)
        return {"bytes": bytes_ + (2 * B * H * new * d * es if case["queries"] else 0),
                "flops": 3 * B * heads * new * case["dim"]}
    if case["ragged"]:
        n = 0.625 * n
    if case["evicted"]:
        n = 0.875 * n
    p = [1.0 / i ** (1.1 if case["groups"] == "zipf" else 0.0) for i in range(1, K + 1)]
    z = sum(p)
    one = sum((x / z) ** 2 for x in p)                                  # a far key shares one node's group
    some = sum(x / z * (1 - (1 - x / z) ** new) for x in p)             # ... or any of the nodes' groups
    near = min(n, w)
    far = max(0.0, n - near)
    depth = (new + 1) / 2 if case["tree"] == "chain" else 1 + math.log(new + 1)
    bytes_ = B * H_kv * (2 * n + 8 * n / PAGE + 4 * near + (near + far * some) * 2 * d + new * 2 * d * es)
    return {"bytes": bytes_ + B * H * new * (2 * d * es + 4), "flops": 4 * d * B * H * new * (near + far * one + depth)}


# ------------------------------------------------------------------ exact ---

def _two_to(e):
    """2^e in 64 bits, exact (a power of two from pow() may be off in its last place)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(codes):
    """The numbers that e4m3 codes stand for, in 64 bits, from the format's definition."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    size = torch.where(e > 0, (1 + m / 8) * _two_to(e - 7), m / 512)
    return torch.where(c >= 128, -size, size)


def _to_e4m3(x):
    """The nearest e4m3 numbers to |x| <= 448 (halves to even), in 64 bits."""
    step = _two_to(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _page_scale(rows):
    """Least power of two >= 2^MIN_EXP that brings the rows to at most 448."""
    a = rows.abs().amax().clamp(min=448.0 * 2.0 ** MIN_EXP)
    s = _two_to(torch.frexp(a / 512.0)[1])                               # 256 s <= a < 512 s
    return float(torch.where(a > 448.0 * s, 2.0 * s, s))


def _turn(x, at, s, back=False):
    """Rows [.., T, d] in 64 bits times the rotation matrices of positions `at` [T], as complex numbers."""
    c = s["case"]
    h = c["dim"] // 2
    phase = torch.outer(at.double(), s["inv_freq"].double())
    by = torch.polar(torch.full_like(phase, c["factor"]), -phase if back else phase)
    lo, hi = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if c["interleaved"] else (slice(0, h), slice(h, 2 * h))
    out = x.double().clone()
    z = torch.complex(out[..., lo].contiguous(), out[..., hi].contiguous()) * by
    out[..., lo], out[..., hi] = z.real, z.imag
    return out


def _paths(s, b):
    """Of sequence b: each node's path from the root, itself included, as lists."""
    out = []
    for t, up in enumerate(s["parent"][b].tolist()):
        out.append((out[up] if up >= 0 else []) + [t])
    return out


def _counts(s):
    return [s["case"]["T"]] * s["case"]["B"] if s["n_new"] is None else s["n_new"].tolist()


def _exact_rotary(s):
    k = s["case"]
    out = dict(Q=s["Q_out"].double().clone(), K=s["K_out"].double().clone())
    for b, m in enumerate(_counts(s)):
        depth = torch.arange(k["T"], device="cuda")
        if s["parent"] is not None:
            depth = torch.tensor([len(p) - 1 for p in _paths(s, b)], device="cuda")
        at = int(s["base"][b]) + depth[:m]
        for x in ("Q", "K"):
            out[x][b, :, :m] = _turn(s[x][b, :, :m], at, s, k["transpose"])
    return out


def _exact_append(s):
    c = s["cache"]
    codes = {x: _e4m3(c[x]) for x in ("k", "v")}
    sc = {x: c[x + "_scale"].double().clone() for x in ("k", "v")}
    mass = c["mass"].double().clone()
    more = {x: s[x].double().clone() for x in ("Q_out", "K_out") if s[x] is not None}
    lens, table = c["len"].tolist(), c["table"].tolist()
    for b, m in enumerate(_counts(s)):
        at = int(c["next"][b]) + torch.arange(m, device="cuda")
        pick = torch.arange(m, device="cuda") if s["rows"] is None else s["rows"][b, :m].long()
        new = {"k": _turn(s["K"][b][:, pick], at, s), "v": s["V"][b][:, pick].double()}
        if "K_out" in more:
            more["K_out"][b, :, :m] = new["k"]
        if "Q_out" in more:
            more["Q_out"][b, :, :m] = _turn(s["Q"][b, :, :m], at, s)
        for h, n in enumerate(lens[b]):
            for j in range(n // PAGE, (n + m - 1) // PAGE + 1):
                g, lo, hi = table[b][j], max(n, j * PAGE), min(n + m, (j + 1) * PAGE)
                r = lo - j * PAGE
                mass[g, h, r:hi - j * PAGE] = 0.0
                for x in ("k", "v"):
                    rows = new[x][h, lo - n:hi - n]
                    scale = _page_scale(rows)
                    if r:
                        was = float(sc[x][g, h])
                        scale = max(scale, was)
                        codes[x][g, h, :r] = _to_e4m3(codes[x][g, h, :r] * (was / scale))
                    codes[x][g, h, r:r + hi - lo] = _to_e4m3(rows / scale)
                    sc[x][g, h] = scale
    return dict(k=codes["k"], v=codes["v"], k_scale=sc["k"], v_scale=sc["v"], pos=None, gid=None, mass=mass, len=None,
                next=None, **more)


def _exact_tree(s):
    c, k = s["cache"], s["case"]
    B, H, T, d = s["Q"].shape
    G, w = H // k["H_kv"], max(k["w"], 1)
    O, lse = s["O"].double().clone(), s["lse"].double().clone()
    for b, m in enumerate(_counts(s)):
        paths = _paths(s, b)[:m]
        depth = torch.tensor([len(p) - 1 for p in paths], device="cuda")
        on_path = torch.tensor([[j in p for j in range(m)] for p in paths], device="cuda")
        i = int(c["next"][b]) + depth
        for h in range(k["H_kv"]):
            j = torch.arange(int(c["len"][b, h]), device="cuda")
            page, row = c["table"][b].long()[j // PAGE], j % PAGE
            pos, gid = c["pos"][page, h, row], c["gid"][page, h, row]
            mine = s["gid"][b, h if k["A"] > 1 else 0, :m]
            far = i[:, None] - pos[None].long()
            keep = (far >= 0) & ((far < w) | (mine[:, None] == gid[None]))                    # [m, slots]
            any_ = keep.any(0).nonzero()[:, 0]
            page, row = page[any_], row[any_]
            tree = on_path & ((depth[:, None] - depth[None] < w) | (mine[:, None] == mine[None]))
            keep = torch.cat((keep[:, any_], tree), 1)
            ks, vs = (torch.cat((_e4m3(c[x][page, h, row]) * c[x + "_scale"].double()[page, h][:, None],
                                 s[x.upper()][b, h, :m].double())) for x in ("k", "v"))
            q = s["Q"][b, h * G:(h + 1) * G, :m].double()                                      # [G, m, d]
            z = torch.einsum("gtd,sd->gts", q, ks) * s["scale"]
            z = torch.where(keep[None], z, -math.inf)
            l = torch.logsumexp(z, -1)
            O[b, h * G:(h + 1) * G, :m] = torch.einsum("gts,sd->gtd", torch.exp(z - l[..., None]), vs)
            lse[b, h * G:(h + 1) * G, :m] = l
    return dict(O=O, lse=lse)


def exact(case, seed):
    if case["op"] == "accept":
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "rotary": _exact_rotary, "tree": _exact_tree}[case["op"]](s)
