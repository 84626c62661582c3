"""Decoding with a paged 8-bit key/value cache: the cases that are measured.

Three operators around one cache: the append that quantises new keys and values
into its pages, the Focus attention of new tokens over it, and the eviction of
the slots with the least accumulated attention weight into fresh pages.

A cache page holds 64 slots of one sequence.  Per page and key/value head: e4m3
codes of K and V, one power-of-two scale for each, and per slot the token's
position, group id and accumulated attention weight.  `table` lists a
sequence's pages, `len` the slots in use per head (heads differ after an
eviction), `next` the position that the next appended token gets.

`run` computes a case in plain torch operations, or, with `own` set, through
learned_group_sparse_focus_gb300.focus.
"""
import math

import torch

own = False

PAGE = 64
MIN_EXP = -64          # smallest scale exponent of a page


# ------------------------------------------------------------------ cases ---

def _case(name, op, B, H, H_kv, d, K, w, A, n, T, **more):
    c = dict(name=name, op=op, B=B, H=H, H_kv=H_kv, d=d, K=K, w=w, A=A, n=n, T=T, dtype="bf16", groups="zipf",
             ragged=False, evicted=False, pad=False, accumulate=False, budget=0, recent=0)
    c.update(more)
    return c


def listed():
    return [
        # one decode step's append of a small model, eight sequences of different lengths: the launch itself
        _case("append_step_small", "append", 8, 12, 12, 64, 16, 64, 1, 1024, 1, groups="uniform", ragged=True),
        # a right-padded chunk behind a cached prefix, pages half full on both ends
        _case("append_chunk_ragged", "append", 4, 32, 32, 128, 32, 256, 1, 1500, 777, ragged=True, pad=True),
        # a whole 32K prompt of the GQA layer
        _case("append_prompt_32k", "append", 1, 32, 8, 128, 64, 512, 1, 0, 32768),
        # an fp32 model, odd sizes
        _case("append_f32", "append", 3, 6, 3, 64, 5, 33, 3, 201, 95, dtype="f32", ragged=True),
        # one decode step of the small model
        _case("attend_step_small", "attend", 8, 12, 12, 64, 16, 64, 1, 1024, 1, groups="uniform", ragged=True),
        # one decode step at 32K tokens, one sequence: latency of a single user
        _case("attend_step_32k", "attend", 1, 32, 8, 128, 64, 512, 1, 32768, 1),
        # a serving batch at up to 32K tokens that keeps each key's weight for eviction
        _case("attend_batch_mass", "attend", 16, 32, 8, 128, 64, 512, 1, 32768, 1, ragged=True, accumulate=True),
        # four drafted tokens to verify, 64K tokens, a group id per key/value head
        _case("attend_draft_64k", "attend", 4, 64, 8, 128, 64, 1024, 8, 65536, 4, groups="uniform", pad=True),
        # the last 64 prompt tokens weigh the cached keys before an eviction
        _case("attend_observe_8k", "attend", 2, 32, 32, 128, 32, 256, 1, 8192, 64, accumulate=True),
        # an fp32 model over a cache that was evicted from: heads of different lengths, gaps in the positions
        _case("attend_f32", "attend", 3, 6, 3, 64, 5, 33, 3, 777, 3, dtype="f32", ragged=True, evicted=True,
              accumulate=True),
        # a 32K prompt cut down to 4,096 slots a head
        _case("evict_prompt_32k", "evict", 1, 32, 8, 128, 64, 512, 1, 32768, 1, budget=4096, recent=512),
        # a serving batch brought back to its budget after 512 more tokens
        _case("evict_batch", "evict", 16, 32, 8, 128, 64, 256, 1, 8704, 1, budget=8192, recent=256, evicted=True),
    ]


def draw(rng):
    def lg(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(("append", "attend", "evict"))
    H_kv = rng.choice((1, 2, 3, 4, 8, 12, 32))
    G = rng.choice((1, 2, 4, 8))
    d = rng.choice((64, 128))
    n = lg(1, 65536)
    B = min(rng.randint(1, 16), max(1, (1 << 21) // (n * H_kv)))
    n = min(n, (1 << 21) // H_kv)
    K = lg(1, 512)
    w = lg(1, 1024)
    A = rng.choice((1, H_kv))
    T = 1
    more = dict(dtype=rng.choice(("bf16", "bf16", "bf16", "f32")), groups=rng.choice(("zipf", "uniform")),
                ragged=rng.random() < 0.5, evicted=rng.random() < 0.4)
    if op == "append":
        T = rng.choice((1, lg(1, 4096)))
        T = max(1, min(T, (1 << 18) // (B * H_kv)))
        more["pad"] = rng.random() < 0.5
    elif op == "attend":
        T = max(1, min(rng.choice((1, 1, rng.randint(2, 8), lg(8, 64))), (1 << 25) // (B * H_kv * n * G), n))
        more["accumulate"] = rng.random() < 0.5
        more["pad"] = rng.random() < 0.3
    else:
        more["budget"] = max(1, min(n, lg(1, n)))
        more["recent"] = rng.randint(0, more["budget"])
    c = _case("", op, B, G * H_kv, H_kv, d, K, w, A, n, T, **more)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs ---

def _need_exp(amax):
    """Least e >= MIN_EXP with amax <= 448 * 2^e, for finite amax >= 0 (fp32, exact)."""
    f, x = torch.frexp(amax)                                   # amax = f 2^x, f in [0.5, 1)
    e = torch.where(f > 0.875, x - 8, x - 9)                   # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp_(min=MIN_EXP)


def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127], exact: the exponent's bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(gen, shape):
    """Codes and scales of N(0, 1) rows, page by page: [.., PAGE, d] -> uint8, fp32 [..]."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).float()
    e = _need_exp(x.abs().amax(dim=(-1, -2)))
    s = _pow2(e)
    return (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def _pool(gen, n_pages, H_kv, d, fill):
    dev = "cuda"
    c = dict(k=torch.zeros((n_pages, H_kv, PAGE, d), dtype=torch.uint8, device=dev),
             v=torch.zeros((n_pages, H_kv, PAGE, d), dtype=torch.uint8, device=dev),
             k_scale=torch.ones((n_pages, H_kv), device=dev), v_scale=torch.ones((n_pages, H_kv), device=dev),
             pos=torch.zeros((n_pages, H_kv, PAGE), dtype=torch.int32, device=dev),
             gid=torch.zeros((n_pages, H_kv, PAGE), dtype=torch.int16, device=dev),
             mass=torch.zeros((n_pages, H_kv, PAGE), device=dev))
    if fill:
        step = max(1, (1 << 26) // (H_kv * PAGE * d))
        for a in range(0, n_pages, step):
            b = min(n_pages, a + step)
            for x in ("k", "v"):
                c[x][a:b], c[x + "_scale"][a:b] = _codes(gen, (b - a, H_kv, PAGE, d))
    return c


def prepare(case, seed):
    B, H, H_kv, d, K, A, n, T = (case[x] for x in ("B", "H", "H_kv", "d", "K", "A", "n", "T"))
    op, dev = case["op"], "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    # slots in use: [B, H_kv], ragged over sequences, and over heads where slots were evicted
    lens = torch.full((B, H_kv), n, dtype=torch.int32, device=dev)
    if case["ragged"]:
        lens = (n - (rand(B, 1) * 0.75 * n).int()).int().expand(B, H_kv).contiguous()
    if case["evicted"] and op != "evict":
        lens = torch.maximum(lens - (rand(B, H_kv) * 0.25 * lens).int(), lens.clamp(max=1)).int()
    room = n + T if op == "append" else n
    max_pages = max(1, -(-room // PAGE))
    cap = max_pages * PAGE
    # positions rise along the slots; an evicted cache has gaps in all but its last 256 slots
    slot = torch.arange(cap, device=dev)
    inc = torch.ones((B, H_kv, cap), dtype=torch.int64, device=dev)
    if case["evicted"]:
        gap = (-2.0 * torch.log(1.0 - rand(B, H_kv, cap))).long()
        inc += torch.where(slot < lens[..., None] - 256, gap, 0)
    live = slot < lens[..., None]
    run_up = torch.where(live, inc, 0).cumsum(-1)
    total = run_up[..., -1]
    nxt = total.amax(1)                                                        # [B]
    pos = torch.where(live, nxt[:, None, None] - total[..., None] + run_up - 1, 0)
    # group ids by position, one assignment for all heads or one a head
    span = int(nxt.max()) + T + 1 if n else T + 1
    p = torch.arange(1, K + 1, device=dev, dtype=torch.float32) ** (-1.1 if case["groups"] == "zipf" else 0.0)
    cdf = (p / p.sum()).cumsum(0)
    ids = torch.randperm(K, generator=gen, device=dev)
    of_token = ids[torch.searchsorted(cdf, rand(B, A, span)).clamp_(max=K - 1)].int()
    gid = torch.gather(of_token.expand(B, H_kv, span), 2, pos).short()
    # pages of a sequence lie anywhere in the pool
    n_pages = B * max_pages
    table = torch.randperm(n_pages, generator=gen, device=dev).int().view(B, max_pages)
    cache = _pool(gen, n_pages, H_kv, d, True)
    at = table.long().view(-1)

    def spread(x):
        return x.view(B, H_kv, max_pages, PAGE).transpose(1, 2).reshape(n_pages, H_kv, PAGE)

    # weight that a key has gathered: long-tailed, none for two keys in five
    mass = torch.exp(2.0 * torch.randn((B, H_kv, cap), generator=gen, device=dev)) * (rand(B, H_kv, cap) > 0.4)
    cache["pos"][at] = spread(pos.int())
    cache["gid"][at] = spread(gid)
    cache["mass"][at] = spread(mass * live)
    cache.update(table=table, len=lens, next=nxt.int())
    s = dict(case=case, cache=cache, scale=1.0 / math.sqrt(d))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt)

    if op == "evict":
        pages = max(1, -(-case["budget"] // PAGE))
        dst = _pool(gen, B * pages, H_kv, d, False)
        dst.update(table=torch.randperm(B * pages, generator=gen, device=dev).int().view(B, pages),
                   len=torch.zeros((B, H_kv), dtype=torch.int32, device=dev),
                   next=torch.zeros(B, dtype=torch.int32, device=dev))
        s["dst"] = dst
        return s
    s["n_new"] = (1 + (rand(B) * T).int()).clamp_(max=T).int() if case["pad"] else None
    if op == "append":
        s["K"], s["V"] = normal(B, H_kv, T, d), normal(B, H_kv, T, d)
        first = torch.zeros(B, dtype=torch.int64, device=dev) + nxt
        s["len"], s["next"] = torch.empty_like(lens), torch.empty_like(cache["next"])
    else:
        s["Q"] = normal(B, H, T, d)
        first = nxt - (T if s["n_new"] is None else s["n_new"])
        s["O"] = torch.zeros_like(s["Q"])
        s["lse"] = torch.zeros((B, H, T), device=dev)
    where = (first[:, None] + torch.arange(T, device=dev)).clamp_(min=0)
    s["gid"] = torch.gather(of_token, 2, where[:, None].expand(B, A, T)).contiguous()
    return s


# ------------------------------------------------------------ plain forms ---

def _rows(x, table):
    """[n_pages, H_kv, PAGE, ...] -> [B, H_kv, slots, ...] through the table."""
    y = x[table.long()].transpose(1, 2)
    return y.reshape(y.shape[0], y.shape[1], -1, *y.shape[4:])


def _values(x, scale, table):
    y = x.view(torch.float8_e4m3fn)[table.long()].float() * scale[table.long()][..., None, None]
    y = y.transpose(1, 2)
    return y.reshape(y.shape[0], y.shape[1], -1, y.shape[-1])


def _quantise(x, e):
    """x [.., PAGE, d] at page exponents e [..] -> codes."""
    y = (x * _pow2(-e)[..., None, None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c, T = s["cache"], s["case"]["T"]
    B, H_kv = c["len"].shape
    dev = c["len"].device
    n_new = s["n_new"] if s["n_new"] is not None else torch.full((B,), T, dtype=torch.int32, device=dev)
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
        rows = torch.gather(x.float(), 2, tc.view(B, H_kv, -1, 1).expand(-1, -1, -1, x.shape[-1]))
        rows = rows.view(*t.shape, -1) * new[..., None]
        was = codes[where, head]
        e_old = torch.frexp(scale[where, head])[1] - 1
        need = _need_exp(rows.abs().amax(dim=(-1, -2)))
        e = torch.where(old.any(-1), torch.maximum(need, e_old), need)
        kept = was.view(torch.float8_e4m3fn).float() * scale[where, head][..., None, None]
        both = _quantise(torch.where(old[..., None], kept, rows), e)
        codes[where[used], head[used]] = torch.where((new | old)[..., None], both, was)[used]
        scale[where[used], head[used]] = _pow2(e)[used]

    one(s["K"], c["k"], c["k_scale"])
    one(s["V"], c["v"], c["v_scale"])
    at, h, r = where[..., None].expand_as(t)[new], head[..., None].expand_as(t)[new], (slot % PAGE)[new]
    c["pos"][at, h, r] = (c["next"].long()[:, None, None, None] + t)[new].int()
    ids = s["gid"].expand(B, H_kv, T)
    c["gid"][at, h, r] = torch.gather(ids, 2, tc.view(B, H_kv, -1)).view_as(t)[new].short()
    c["mass"][at, h, r] = 0.0
    s["len"].copy_(c["len"] + n_new[:, None])
    s["next"].copy_(c["next"] + n_new)


def _plain_attend(s):
    c, k = s["cache"], s["case"]
    B, H, T, d = s["Q"].shape
    H_kv, G = k["H_kv"], H // k["H_kv"]
    dev = s["Q"].device
    n_new = s["n_new"] if s["n_new"] is not None else torch.full((B,), T, dtype=torch.int32, device=dev)
    t = torch.arange(T, device=dev)
    i = (c["next"] - n_new)[:, None] + t                                                       # [B, T]
    pos, gid = _rows(c["pos"], c["table"]), _rows(c["gid"], c["table"])                        # [B, H_kv, S]
    slot = torch.arange(pos.shape[-1], device=dev)
    ahead = i[:, None, :, None] - pos[:, :, None, :]                                           # [B, H_kv, T, S]
    same = s["gid"].expand(B, H_kv, T)[..., None] == gid[:, :, None, :]
    keep = (ahead >= 0) & ((ahead < max(k["w"], 1)) | same) & (slot < c["len"][:, :, None, None])
    q = s["Q"].float().view(B, H_kv, G, T, d)
    score = torch.matmul(q.reshape(B, H_kv, G * T, d), _values(c["k"], c["k_scale"], c["table"]).transpose(2, 3))
    score = (score * s["scale"]).view(B, H_kv, G, T, -1).masked_fill(~keep[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    out = torch.matmul(p.view(B, H_kv, G * T, -1), _values(c["v"], c["v_scale"], c["table"]))
    there = t < n_new[:, None]                                                                 # [B, T]
    out = out.view(B, H, T, d).to(s["O"].dtype)
    s["O"].copy_(torch.where(there[:, None, :, None], out, s["O"]))
    lse = (top + torch.log(total)).view(B, H, T)
    s["lse"].copy_(torch.where(there[:, None], lse, s["lse"]))
    if k["accumulate"]:
        got = (p * there[:, None, None, :, None]).sum(dim=(2, 3))                              # [B, H_kv, S]
        got = got.view(B, H_kv, -1, PAGE).transpose(1, 2)
        c["mass"][c["table"].long()] += got


def _plain_evict(s):
    c, o, k = s["cache"], s["dst"], s["case"]
    B, H_kv = c["len"].shape
    dev, budget = c["len"].device, k["budget"]
    mass, pos, gid = (_rows(c[x], c["table"]) for x in ("mass", "pos", "gid"))
    S = mass.shape[-1]
    slot = torch.arange(S, device=dev)
    late = pos >= (c["next"].int()[:, None, None] - k["recent"])
    key = torch.where(late, math.inf, mass).masked_fill(slot >= c["len"][..., None], -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    n = torch.minimum(c["len"], torch.full_like(c["len"], budget))
    pages = o["table"].shape[1]
    rank = torch.arange(pages * PAGE, device=dev)
    picked = torch.where(rank[:order.shape[-1]] < n[..., None], order, S).sort(-1).values
    pick = torch.zeros((B, H_kv, pages * PAGE), dtype=torch.int64, device=dev)
    pick[..., :picked.shape[-1]] = picked.clamp(max=S - 1)
    valid = (rank < n[..., None]).view(B, H_kv, pages, PAGE)
    used = valid.any(-1)
    where = o["table"].long()[:, None].expand(B, H_kv, pages)
    head = torch.arange(H_kv, device=dev)[None, :, None].expand_as(where)

    def one(codes, scale, to, to_scale):
        x = torch.gather(_values(codes, scale, c["table"]), 2, pick[..., None].expand(-1, -1, -1, codes.shape[-1]))
        x = x.view(B, H_kv, pages, PAGE, -1) * valid[..., None]
        e = _need_exp(x.abs().amax(dim=(-1, -2)))
        was = to[where, head]
        to[where[used], head[used]] = torch.where(valid[..., None], _quantise(x, e), was)[used]
        to_scale[where[used], head[used]] = _pow2(e)[used]

    one(c["k"], c["k_scale"], o["k"], o["k_scale"])
    one(c["v"], c["v_scale"], o["v"], o["v_scale"])
    at, h = where[..., None].expand_as(valid)[valid], head[..., None].expand_as(valid)[valid]
    r = (rank % PAGE).view(pages, PAGE).expand_as(valid)[valid]
    o["pos"][at, h, r] = torch.gather(pos, 2, pick).view_as(valid)[valid]
    o["gid"][at, h, r] = torch.gather(gid, 2, pick).view_as(valid)[valid]
    o["mass"][at, h, r] = torch.gather(mass, 2, pick).view_as(valid)[valid]
    o["len"].copy_(n)
    o["next"].copy_(c["next"])


# -------------------------------------------------------------------- run ---

def _contents(c, **more):
    """A cache as the values it stands for: codes as e4m3 numbers, beside their pages' scales."""
    out = dict(k=c["k"].view(torch.float8_e4m3fn), v=c["v"].view(torch.float8_e4m3fn), k_scale=c["k_scale"],
               v_scale=c["v_scale"], pos=c["pos"], gid=c["gid"], mass=c["mass"])
    out.update(more)
    return out


def _handle(s):
    """What a program keeps between calls: problem description, cache handles and workspace."""
    from learned_group_sparse_focus_gb300 import focus as fz
    k = s["case"]
    p = fz.make_params(k["B"], k["H"], k["H_kv"], k["T"], k["d"], 64, 64, k["K"], k["A"], k["w"], scale=s["scale"],
                       dtype=k["dtype"])
    cache = fz.Cache(**s["cache"])
    dst = fz.Cache(**s["dst"]) if "dst" in s else None
    return fz, p, cache, dst, fz.alloc_workspace_cache(p, cache)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if "handle" not in s:
            s["handle"] = _handle(s)
        fz, p, cache, dst, ws = s["handle"]
        if op == "append":
            fz.focus_cache_append(p, s["K"], s["V"], s["gid"], cache, ws, n_new=s["n_new"], len_out=s["len"],
                                  next_out=s["next"])
        elif op == "attend":
            fz.focus_cache_attention_fwd(p, s["Q"], s["gid"], cache, s["O"], s["lse"], ws, n_new=s["n_new"],
                                         accumulate=s["case"]["accumulate"])
        else:
            fz.focus_cache_evict(p, s["case"]["budget"], s["case"]["recent"], cache, dst, ws)
    elif op == "append":
        _plain_append(s)
    elif op == "attend":
        _plain_attend(s)
    else:
        _plain_evict(s)
    if op == "append":
        return _contents(s["cache"], len=s["len"], next=s["next"])
    if op == "evict":
        return _contents(s["dst"], len=s["dst"]["len"], next=s["dst"]["next"])
    out = dict(O=s["O"], lse=s["lse"])
    if s["case"]["accumulate"]:
        out["mass"] = s["cache"]["mass"]
    return out


def work(case):
    B, H, H_kv, d, K, n, T = (case[x] for x in ("B", "H", "H_kv", "d", "K", "n", "T"))
    es, G = (2 if case["dtype"] == "bf16" else 4), H // H_kv
    if case["ragged"]:
        n = 0.625 * n
    if case["evicted"] and case["op"] != "evict":
        n = 0.875 * n
    new = (T + 1) / 2 if case["pad"] else T
    if case["op"] == "append":
        return {"bytes": B * H_kv * new * (2 * d * es + 2 * d + 4 + 2 + 4 + 4), "flops": 0}
    if case["op"] == "evict":
        kept = min(n, case["budget"])
        return {"bytes": B * H_kv * (4 * n + kept * 2 * (2 * d + 4 + 2 + 4) + 16 * kept / PAGE), "flops": 0}
    p = [1.0 / i ** (1.1 if case["groups"] == "zipf" else 0.0) for i in range(1, K + 1)]
    z = sum(p)
    one = sum((x / z) ** 2 for x in p)                                  # a far key shares one token's group
    some = sum(x / z * (1 - (1 - x / z) ** new) for x in p)             # ... or any of the tokens' groups
    near, far = min(n, max(case["w"], 1) + new), max(0.0, n - max(case["w"], 1) - new)
    kept, slots = near + far * some, B * H_kv
    bytes_ = slots * (2 * n + 8 * n / PAGE + 4 * near + kept * (2 * d + (8 if case["accumulate"] else 0)))
    return {"bytes": bytes_ + B * H * new * (2 * d * es + 4), "flops": 4 * d * B * H * new * (near + far * one)}


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


def _page_scales(rows):
    """Least power of two >= 2^MIN_EXP that brings each page's rows to at most 448: [.., PAGE, d] -> [..]."""
    a = rows.abs().amax(dim=(-1, -2))
    s = _two_to(torch.frexp(a.clamp(min=448.0 * 2.0 ** MIN_EXP) / 512.0)[1])     # 256 s <= a < 512 s
    return torch.where(a > 448.0 * s, 2.0 * s, s)


def _exact_slots(c, b, h):
    """The live slots of one head in order: (page, row) pairs."""
    j = torch.arange(int(c["len"][b, h]), device=c["len"].device)
    return c["table"][b].long()[j // PAGE], j % PAGE


def _exact_values(c, name, page, h, row):
    return _e4m3(c[name][page, h, row]) * c[name + "_scale"].double()[page, h][:, None]


def _exact_append(s):
    c, T = s["cache"], s["case"]["T"]
    out = {x: _e4m3(c[x]) for x in ("k", "v")}
    sc = {x: c[x + "_scale"].double().clone() for x in ("k", "v")}
    mass = c["mass"].double().clone()
    lens = c["len"].tolist()
    fresh = [T] * len(lens) if s["n_new"] is None else s["n_new"].tolist()
    table = c["table"].tolist()
    for b, of_head in enumerate(lens):
        for h, n in enumerate(of_head):
            for j in range(n // PAGE, (n + fresh[b] - 1) // PAGE + 1):
                g, lo, hi = table[b][j], max(n, j * PAGE), min(n + fresh[b], (j + 1) * PAGE)
                r = lo - j * PAGE
                mass[g, h, r:hi - j * PAGE] = 0.0
                for x, y in (("k", s["K"]), ("v", s["V"])):
                    rows = y[b, h, lo - n:hi - n].double()
                    scale = float(_page_scales(rows))
                    if r:
                        was = float(sc[x][g, h])
                        scale = max(scale, was)
                        out[x][g, h, :r] = _to_e4m3(out[x][g, h, :r] * (was / scale))
                    out[x][g, h, r:r + hi - lo] = _to_e4m3(rows / scale)
                    sc[x][g, h] = scale
    return dict(k=out["k"], v=out["v"], k_scale=sc["k"], v_scale=sc["v"], pos=None, gid=None, mass=mass, len=None,
                next=None)


def _exact_attend(s):
    c, k = s["cache"], s["case"]
    B, H, T, d = s["Q"].shape
    G = H // k["H_kv"]
    O, lse, mass = s["O"].double().clone(), s["lse"].double().clone(), c["mass"].double().clone()
    fresh = [T] * B if s["n_new"] is None else s["n_new"].tolist()
    for b in range(B):
        m = fresh[b]
        i = int(c["next"][b]) - m + torch.arange(m, device=O.device)
        for h in range(k["H_kv"]):
            page, row = _exact_slots(c, b, h)
            pos, gid = c["pos"][page, h, row], c["gid"][page, h, row]
            mine = s["gid"][b, h if k["A"] > 1 else 0, :m]
            far = i[:, None] - pos[None].long()
            keep = (far >= 0) & ((far < max(k["w"], 1)) | (mine[:, None] == gid[None]))       # [m, slots]
            any_ = keep.any(0).nonzero()[:, 0]
            page, row, keep = page[any_], row[any_], keep[:, any_]
            ks, vs = _exact_values(c, "k", page, h, row), _exact_values(c, "v", page, h, row)
            q = s["Q"][b, h * G:(h + 1) * G, :m].double()                                      # [G, m, d]
            z = torch.einsum("gtd,sd->gts", q, ks) * s["scale"]
            z = torch.where(keep[None], z, -math.inf)
            l = torch.logsumexp(z, -1)
            p = torch.where(keep[None], torch.exp(z - torch.where(torch.isfinite(l), l, 0.0)[..., None]), 0.0)
            O[b, h * G:(h + 1) * G, :m] = torch.einsum("gts,sd->gtd", p, vs)
            lse[b, h * G:(h + 1) * G, :m] = l
            mass[page, h, row] += p.sum((0, 1))
    out = dict(O=O, lse=lse)
    if k["accumulate"]:
        out["mass"] = mass
    return out


def _exact_evict(s):
    c, o, k = s["cache"], s["dst"], s["case"]
    out = {x: _e4m3(o[x]) for x in ("k", "v")}
    sc = {x: o[x + "_scale"].double().clone() for x in ("k", "v")}
    mass = o["mass"].double().clone()
    for b in range(c["len"].shape[0]):
        for h in range(k["H_kv"]):
            page, row = _exact_slots(c, b, h)
            if len(page) > k["budget"]:
                last = c["pos"][page, h, row] >= int(c["next"][b]) - k["recent"]
                old = (~last).nonzero()[:, 0]
                weight = c["mass"][page, h, row][old].double().cpu()
                best = sorted(range(len(old)), key=lambda x, w=weight.tolist(): (-w[x], x))
                best = best[:k["budget"] - int(last.sum())]
                stay = torch.cat([last.nonzero()[:, 0], old[torch.tensor(best, dtype=torch.int64, device=old.device)]])
                stay = stay.sort().values
                page, row = page[stay], row[stay]
            n, pages = len(page), -(-len(page) // PAGE)
            dst = o["table"][b].long()[:pages]
            for x in ("k", "v"):
                rows = torch.zeros((pages, PAGE, c[x].shape[-1]), dtype=torch.float64, device=page.device)
                rows.view(pages * PAGE, -1)[:n] = _exact_values(c, x, page, h, row)
                sc[x][dst, h] = _page_scales(rows)
                new = _to_e4m3(rows / sc[x][dst, h][:, None, None])
                slot = torch.arange(n, device=page.device)
                out[x][dst[slot // PAGE], h, slot % PAGE] = new.view(pages * PAGE, -1)[:n]
            mass[dst[slot // PAGE], h, slot % PAGE] = c["mass"][page, h, row].double()
    return dict(k=out["k"], v=out["v"], k_scale=sc["k"], v_scale=sc["v"], pos=None, gid=None, mass=mass, len=None,
                next=None)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](s)
