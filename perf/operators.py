"""Operators of a decode step around the MoE layer, as cases to be measured.

    tables   block tables and slot maps of a paged key-value cache, from request lengths
    append   new keys and values written into the cache at those slots
    attend   attention of one new token per request over the paged cache
    sample   the next token of each request from its logits and a given random number

``run`` computes a case in plain torch operations, or through the package's
entry points where ``own`` is true.  Shapes are those of the package's decode
workloads (hidden size 2048: 32 query heads of 128 on 4 key-value heads) and
generic ones; every value comes from the seed.
"""
import math

import torch

own = False

_KV = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_FLT_MAX = 3.4028234663852886e38


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of a full serving batch: a token each, contexts of all lengths
        dict(name="tables_decode", op="tables", B=256, page=16, ctx=8192, tokens=256, chunk=False),
        # a step that mixes chunks of prompts with decoding requests
        dict(name="tables_prompts", op="tables", B=300, page=16, ctx=4096, tokens=32768, chunk=True),
        # the keys and values of one layer in such a decode step, into an 8-bit cache
        dict(name="append_decode_e4m3", op="append", N=256, Hkv=4, D=128, page=16, kv="e4m3",
             slots=65536, major="token"),
        # the same for a step of long prompts, into a bf16 cache kept head by head
        dict(name="append_prompts_bf16", op="append", N=16384, Hkv=8, D=128, page=32, kv="bf16",
             slots=65536, major="head"),
        # a single short conversation: nothing but latency
        dict(name="attend_one_short_bf16", op="attend", B=1, Hq=32, Hkv=4, D=128, page=16,
             kv="bf16", longest=700, window=0, empty=0, major="token"),
        # an ordinary batch of mixed lengths, a few slots of the batch unused
        dict(name="attend_batch_bf16", op="attend", B=64, Hq=32, Hkv=4, D=128, page=16, kv="bf16",
             longest=4096, window=0, empty=3, major="token"),
        # one request with a very long document
        dict(name="attend_one_long_bf16", op="attend", B=1, Hq=32, Hkv=4, D=128, page=64,
             kv="bf16", longest=262161, window=0, empty=0, major="head"),
        # a large batch with an 8-bit cache
        dict(name="attend_batch_e4m3", op="attend", B=256, Hq=32, Hkv=4, D=128, page=16,
             kv="e4m3", longest=8192, window=0, empty=5, major="token"),
        # the f32 layer's small model: odd sizes, a page size that is no power of two, a window
        dict(name="attend_window_f32", op="attend", B=9, Hq=6, Hkv=2, D=80, page=5, kv="f32",
             longest=5000, window=1000, empty=1, major="token"),
        # one request's next token, with every restriction in force
        dict(name="sample_one_f32", op="sample", B=1, V=131072, dtype="f32", kind="all"),
        # an ordinary batch, odd vocabulary, each request with its own settings
        dict(name="sample_batch_bf16", op="sample", B=64, V=50257, dtype="bf16", kind="mixed"),
        # a large batch with top-p and with temperature alone
        dict(name="sample_large_f32", op="sample", B=512, V=131072, dtype="f32", kind="wide"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "attend", "sample", "sample"])
    if op == "tables":
        B, chunk = _log_int(rng, 1, 512), rng.random() < 0.5
        return dict(op=op, B=B, page=rng.choice([1, 5, 8, 16, 32, 64, 128]),
                    ctx=_log_int(rng, 16, 8192), chunk=chunk,
                    tokens=_log_int(rng, B, 32768) if chunk else B + rng.randrange(0, 9))
    if op == "append":
        return dict(op=op, N=_log_int(rng, 1, 16384), Hkv=rng.choice([1, 2, 3, 4, 8]),
                    D=rng.choice([64, 80, 96, 128, 192, 256]), page=rng.choice([1, 5, 8, 16, 32, 64]),
                    kv=rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"]), slots=32768,
                    major=rng.choice(["token", "head"]))
    if op == "attend":
        kv = rng.choice(["bf16", "bf16", "e4m3", "e4m3", "f32"])
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128, 128, 256])
        B = _log_int(rng, 1, 256)
        # at most half a gigabyte of keys and values, were every request the longest
        room = (1 << 28) // (B * Hkv * D * {"f32": 4, "bf16": 2, "e4m3": 1}[kv])
        longest = _log_int(rng, 1, max(1, min(262144, room)))
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 3, 4, 7, 8, 8, 16, 20]), Hkv=Hkv, D=D,
                    page=rng.choice([1, 5, 16, 16, 32, 64, 128]), kv=kv, longest=longest,
                    window=rng.choice([0, 0, 0, 100, 1024]), empty=rng.choice([0, 0, B // 8]),
                    major=rng.choice(["token", "head"]))
    B = _log_int(rng, 1, 512)
    return dict(op=op, B=B, V=_log_int(rng, 1000, min(262144, (1 << 26) // B)),
                dtype=rng.choice(["f32", "bf16"]),
                kind=rng.choice(["all", "mixed", "wide", "greedy", "topk"]))


# ------------------------------------------------------------------ their inputs
def _cache(g, pages, page, Hkv, D, dtype, major):
    """Keys and values [pages, page, Hkv, D], stored token by token or head by head."""
    kv = []
    for _ in range(2):
        if major == "head":
            t = torch.empty(pages, Hkv, page, D, dtype=_KV[dtype], device="cuda")
        else:
            t = torch.empty(pages, page, Hkv, D, dtype=_KV[dtype], device="cuda")
        for p in range(0, pages, max(1, (1 << 26) // (page * Hkv * D))):  # bounds the f32 copy
            e = min(pages, p + max(1, (1 << 26) // (page * Hkv * D)))
            x = torch.randn(t[p:e].shape, generator=g, device="cuda")
            t[p:e] = (x * 40 if dtype == "e4m3" else x).to(_KV[dtype])
        kv.append(t.transpose(1, 2) if major == "head" else t)
    return kv


def _lengths(g, n, longest):
    """Lengths 1 .. longest, half of them long and half spread over their logarithm; one is the longest."""
    a = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    b = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    flat = (a * longest).floor() + 1
    spread = torch.exp(a * math.log(longest + 1)).floor()
    lens = torch.where(b < 0.5, flat, spread).clamp(1, longest).to(torch.int32)
    lens[int(torch.randint(n, (1,), generator=g, device="cuda"))] = longest
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    c, op = dict(case), case["op"]
    s = {"op": op}

    def uniform(n):
        return torch.rand(n, generator=g, device="cuda")

    if op == "tables":
        B, page, tokens = c["B"], c["page"], c["tokens"]
        ctx = _lengths(g, B, c["ctx"]) - 1  # from 0: a request may be new
        if c["chunk"]:  # shares of the step's tokens; some requests get none
            share = torch.rand(B, generator=g, device="cuda", dtype=torch.float64) ** 3
            new = (share / share.sum() * tokens).floor().to(torch.int32)
        else:
            new = torch.ones(B, dtype=torch.int32, device="cuda")
        width = -(-(c["ctx"] + (tokens if c["chunk"] else 1)) // page)
        have = (ctx.long() + page - 1) // page
        pool = int(have.sum()) + int(((ctx.long() + new + page - 1) // page - have).sum()) + 100
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        col = torch.arange(width, device="cuda")
        first = torch.cumsum(have, 0) - have
        at = (first[:, None] + col[None, :]).clamp(max=pool - 1)
        table = torch.where(col[None, :] < have[:, None], ids[at], torch.full_like(ids[at], -1))
        free = torch.zeros(pool, dtype=torch.int32, device="cuda")
        n_free = pool - int(have.sum())
        free[:n_free] = ids[pool - n_free:]
        s.update(ctx=ctx, new=new, table=table.contiguous(), free=free, page=page, pool=pool,
                 n_free=torch.tensor([n_free], dtype=torch.int32, device="cuda"), tokens=tokens)
    elif op == "append":
        N, Hkv, D, page = c["N"], c["Hkv"], c["D"], c["page"]
        pages = max(-(-c["slots"] // page), -(-N // page))
        s["k_cache"], s["v_cache"] = _cache(g, pages, page, Hkv, D, c["kv"], c["major"])
        src = torch.float32 if c["kv"] == "f32" else torch.bfloat16
        # keys and values as a projection leaves them: rows of one product, side by side
        x = (torch.randn(N, 2 * Hkv * D, generator=g, device="cuda")).to(src)
        s["k"] = x[:, :Hkv * D].view(N, Hkv, D)
        s["v"] = x[:, Hkv * D:].view(N, Hkv, D)
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:N].to(torch.int32)
        if N > 8:
            slots[torch.randint(N, (N // 64 + 1,), generator=g, device="cuda")] = -1  # padding
        s["slots"] = slots
        if c["kv"] == "e4m3":
            s["k_scale"], s["v_scale"] = 0.005 + 0.01 * uniform(Hkv), 0.005 + 0.01 * uniform(Hkv)
    elif op == "attend":
        B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
        lens = _lengths(g, B, c["longest"])
        if c["empty"]:
            lens[torch.randperm(B, generator=g, device="cuda")[:c["empty"]]] = 0
        width = -(-c["longest"] // page)
        need = (lens.long() + page - 1) // page
        pages = int(need.sum()) + 3
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        col = torch.arange(width, device="cuda")
        at = ((torch.cumsum(need, 0) - need)[:, None] + col[None, :]).clamp(max=pages - 1)
        table = torch.where(col[None, :] < need[:, None], ids[at], torch.full_like(ids[at], -1))
        s["k_cache"], s["v_cache"] = _cache(g, pages, page, Hkv, D, c["kv"], c["major"])
        part = (lens % page) > 0  # what lies in a page after its last token may be anything
        rows = torch.nonzero(part).flatten()
        pg = table[rows, (lens[rows] // page).long()].long()
        for t in (s["k_cache"], s["v_cache"]):
            t[pg, (lens[rows] % page).long()] = torch.full((), float("nan"), device="cuda").to(t.dtype)
        src = torch.float32 if c["kv"] == "f32" else torch.bfloat16
        s["q"] = torch.randn(B, Hq, D, generator=g, device="cuda").to(src)
        if c["kv"] == "e4m3":
            s["k_scale"], s["v_scale"] = 0.02 + 0.01 * uniform(Hkv), 0.02 + 0.01 * uniform(Hkv)
        s.update(lens=lens, table=table.contiguous(), page=page, longest=c["longest"],
                 window=c["window"], scale=1.0 / math.sqrt(D))
    else:
        B, V, kind = c["B"], c["V"], c["kind"]
        # logits of a language model: a bulk, and a few likely tokens well above it
        x = 1.8 * torch.randn(B, V, generator=g, device="cuda")
        at = torch.randint(V, (B, 40), generator=g, device="cuda")
        top = 6.0 + 2.0 * torch.randn(B, 40, generator=g, device="cuda")
        x.scatter_reduce_(1, at, top, "amax")  # a token drawn twice: the same whatever comes first
        masked = torch.rand(B, generator=g, device="cuda") < 0.2  # rows under a grammar
        drop = torch.rand(1, V, generator=g, device="cuda") < 0.3
        x.masked_fill_(masked[:, None] & drop, float("-inf"))
        s["logits"] = x.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
        s["u"] = uniform(B)
        t = 0.6 + 0.7 * uniform(B)
        k = (1 + (uniform(B) ** 2 * min(100, V - 1)).floor()).to(torch.int32)
        p, m = 0.8 + 0.19 * uniform(B), 0.02 + 0.1 * uniform(B)
        off = uniform(B)
        zero = torch.zeros_like(k)
        if kind == "all":
            s.update(temperature=t, top_k=k, top_p=p, min_p=m)
        elif kind == "greedy":
            s.update(temperature=torch.zeros_like(t), top_k=None, top_p=None, min_p=None)
        elif kind == "topk":
            s.update(temperature=t, top_k=k, top_p=None, min_p=None)
        elif kind == "wide":
            s.update(temperature=t, top_k=None, min_p=None,
                     top_p=torch.where(off < 0.5, p, torch.ones_like(p)))
        else:
            s.update(temperature=torch.where(off < 0.15, torch.zeros_like(t), t),
                     top_k=torch.where(uniform(B) < 0.3, zero, k),
                     top_p=torch.where(uniform(B) < 0.3, torch.ones_like(p), p),
                     min_p=torch.where(uniform(B) < 0.5, torch.zeros_like(m), m))
    return s


# ------------------------------------------------------------------ their plain forms
def _tables_plain(s):
    page, pool, tokens, table = s["page"], s["pool"], s["tokens"], s["table"]
    ctx, new = s["ctx"].long().clamp(min=0), s["new"].long().clamp(min=0)
    B, width = table.shape
    ends = torch.cumsum(new, 0)
    starts = ends - new
    have = ((ctx + page - 1) // page).clamp(max=width)
    need = ((ctx + new + page - 1) // page).clamp(max=width)
    take = need - have
    base = torch.cumsum(take, 0) - take
    n_free = s["n_free"].long()
    # the new pages of each request, from the end of the list of free ones
    col = torch.arange(width, device=table.device)
    order = base[:, None] + col[None, :] - have[:, None]
    fresh = (col[None, :] >= have[:, None]) & (col[None, :] < need[:, None])
    got = s["free"][(n_free - 1 - order).clamp(0, s["free"].numel() - 1)]
    got = torch.where(order < n_free, got, torch.full_like(got, -1))
    table.copy_(torch.where(fresh, got, table))
    # the slot of each new token
    i = torch.arange(tokens, device=table.device)
    r = torch.searchsorted(ends, i, right=True).clamp(max=B - 1)
    real = i < ends[-1]
    pos = torch.where(real, ctx[r] + i - starts[r], torch.zeros_like(i))
    pg = torch.where(pos // page < width, table[r, (pos // page).clamp(max=width - 1)].long(),
                     torch.full_like(i, -1))
    real = real & (pg >= 0) & (pg < pool)
    slots = torch.where(real, pg * page + pos % page, torch.full_like(i, -1))
    begin = torch.cat([starts, ends[-1:]])
    return {"slots": slots.int(), "positions": pos.int(), "starts": begin.int(),
            "seq_lens": (ctx + new).int(), "n_free": (n_free - take.sum()).clamp(min=0).int(),
            "table": table}


def _append_plain(s):
    k_cache, v_cache, slots = s["k_cache"], s["v_cache"], s["slots"].long()
    page = k_cache.shape[1]
    keep = torch.nonzero(slots >= 0).flatten()
    at = slots[keep]
    for cache, x, scale in ((k_cache, s["k"], s.get("k_scale")), (v_cache, s["v"], s.get("v_scale"))):
        x = x[keep].float()
        if scale is not None:
            x = (x / scale[None, :, None]).clamp(-448.0, 448.0)
        cache[at // page, at % page] = x.to(cache.dtype)
    return {"k": k_cache, "v": v_cache}


def _attend_plain(s):
    q, lens, page, n = s["q"].float(), s["lens"].long(), s["page"], s["longest"]
    B, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    pos = torch.arange(n, device=q.device)
    live = pos[None, :] < lens[:, None]
    if s["window"]:
        live = live & (pos[None, :] >= lens[:, None] - s["window"])
    pages = torch.where(live, s["table"][:, pos // page], torch.zeros_like(s["table"][:, :1])).long()
    zero = torch.zeros((), device=q.device)
    K = torch.where(live[:, :, None, None], s["k_cache"][pages, pos % page].float(), zero)
    K = K.permute(0, 2, 3, 1)
    if "k_scale" in s:
        K = K * s["k_scale"][None, :, None, None]
    x = torch.matmul(q.view(B, Hkv, Hq // Hkv, D), K) * s["scale"]
    del K
    x = x.masked_fill(~live[:, None, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).view(B, Hq)
    V = torch.where(live[:, :, None, None], s["v_cache"][pages, pos % page].float(), zero)
    V = V.permute(0, 2, 1, 3)
    o = torch.matmul(p, V) / torch.where(total == 0, torch.ones_like(total), total)
    if "v_scale" in s:
        o = o * s["v_scale"][None, :, None, None]
    return {"out": o.view(B, Hq, D).to(s["q"].dtype), "lse": lse}


def _sample_plain(s):
    # 64 bits: a token is chosen by where a sum over the vocabulary passes a border
    x = s["logits"].double()
    B, V = x.shape
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x).clamp(max=_FLT_MAX)
    live = x > float("-inf")
    top = x.amax(-1, keepdim=True)
    t = s["temperature"].double()[:, None]
    d = torch.where(live, x - top, torch.full_like(x, float("-inf")))
    w = torch.where(live, torch.exp(d / torch.where(t > 0, t, torch.ones_like(t))), torch.zeros_like(x))
    x, order = torch.sort(x, dim=-1, descending=True, stable=True)  # ties: the lowest index first
    rank = torch.arange(V, device=x.device)[None, :]
    keep = x > float("-inf")
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((rank < k) | (k <= 0))
    w_sorted = torch.gather(w, 1, order)
    if s["min_p"] is not None:
        keep = keep & (w_sorted >= s["min_p"].double()[:, None].clamp(max=1.0))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        w_sorted = w_sorted * keep
        before = torch.cumsum(w_sorted, -1) - w_sorted
        keep = keep & ((before < p * w_sorted.sum(-1, keepdim=True)) | (rank == 0) | (p >= 1.0))
    keep = keep & ((t > 0) | (rank == 0))
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    mass = torch.where(kept, w, torch.zeros_like(w))
    sums = torch.cumsum(mass, -1)
    total = sums[:, -1:]
    ids = (sums <= s["u"].double()[:, None] * total).sum(-1, keepdim=True)
    last = (mass > 0).mul(rank).amax(-1, keepdim=True)
    ids = torch.minimum(ids, last)
    prob = torch.gather(mass, 1, ids) / total
    none = ~live.any(-1)
    return {"ids": torch.where(none, torch.full_like(ids[:, 0], -1), ids[:, 0]).int(),
            "probs": torch.where(none, torch.zeros_like(prob[:, 0]), prob[:, 0]).float()}


def run(state):
    s, op = state, state["op"]
    if own:
        import serving_moe_route_gb300 as moe

        if op == "tables":
            r = moe.kv_step(s["ctx"], s["new"], s["table"], s["free"], s["n_free"],
                            page_size=s["page"], num_pages=s["pool"], max_tokens=s["tokens"])
            return {"slots": r.slots, "positions": r.positions, "starts": r.starts,
                    "seq_lens": r.seq_lens, "n_free": r.n_free, "table": s["table"]}
        if op == "append":
            moe.kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
                          k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
            return {"k": s["k_cache"], "v": s["v_cache"]}
        if op == "attend":
            out, lse = moe.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                       scale=s["scale"], window=s["window"],
                                       k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                                       return_lse=True)
            return {"out": out, "lse": lse}
        ids, probs = moe.sample_tokens(s["logits"], s["u"], temperature=s["temperature"],
                                       top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return {"ids": ids, "probs": probs}
    if op == "tables":
        return _tables_plain(s)
    if op == "append":
        return _append_plain(s)
    if op == "attend":
        return _attend_plain(s)
    return _sample_plain(s)


# ------------------------------------------------------------------ what they cannot do without
def work(case):
    c, op = case, case["op"]
    if op == "tables":
        # lengths in, starts and lengths out; a slot and a position a token; a page id per page
        # that the tokens touch (at most one a token, or the pages of the chunk)
        pages = c["B"] + c["tokens"] // c["page"]
        return {"bytes": 16 * c["B"] + 8 * c["tokens"] + 8 * pages, "flops": 0}
    if op == "append":
        src, dst = (4, 4) if c["kv"] == "f32" else (2, 2 if c["kv"] == "bf16" else 1)
        return {"bytes": 2 * c["N"] * c["Hkv"] * c["D"] * (src + dst) + 4 * c["N"], "flops": 0}
    if op == "attend":
        # the lengths' mean: half are even over 1 .. longest, half even over the logarithm
        n = c["longest"]
        mean = 0.5 * (n + 1) / 2 + 0.5 * n / math.log(n + 1)
        if c["window"] and c["window"] < n:
            w = c["window"]
            mean = (0.5 * (w - w * w / (2 * n))
                    + 0.5 * (w + w * math.log((n + 1) / (w + 1))) / math.log(n + 1))
            n = w
        total = n + max(0, c["B"] - 1 - c["empty"]) * mean
        e = {"f32": 4, "bf16": 2, "e4m3": 1}[c["kv"]]
        q = 4 if c["kv"] == "f32" else 2
        return {"bytes": 2 * total * c["Hkv"] * c["D"] * e + 2 * c["B"] * c["Hq"] * c["D"] * q,
                "flops": 4 * total * c["Hq"] * c["D"]}
    e = 4 if c["dtype"] == "f32" else 2
    return {"bytes": c["B"] * (c["V"] * e + 28), "flops": c["B"] * c["V"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "tables":
        return None  # whole numbers
    if op == "append":
        out = []
        for cache, x, scale in ((s["k_cache"], s["k"], s.get("k_scale")),
                                (s["v_cache"], s["v"], s.get("v_scale"))):
            page, new = cache.shape[1], x.double()
            if scale is not None:
                new = new / scale.double()[:, None]
                new = torch.minimum(torch.maximum(new, torch.full_like(new, -448.0)),
                                    torch.full_like(new, 448.0))
            whole = cache.double()
            for j in range(0, new.shape[0], 4096):
                at = s["slots"][j:j + 4096].long()
                real = at > -1
                whole[at[real] // page, at[real] % page] = new[j:j + 4096][real]
            out.append(whole)
        return {"k": out[0], "v": out[1]}
    if op == "attend":
        q = s["q"].double()
        B, Hq, D = q.shape
        Hkv, page = s["k_cache"].shape[2], s["page"]
        out, lse = torch.zeros_like(q), torch.full((B, Hq), float("-inf"), dtype=q.dtype, device=q.device)
        for b, n in enumerate(s["lens"].tolist()):
            first = max(0, n - s["window"]) if s["window"] else 0
            if n == first:
                continue
            pg = s["table"][b, first // page:-(-n // page)].long()
            cut = slice(first - first // page * page, n - first // page * page)
            for h in range(Hkv):
                K = s["k_cache"][pg, :, h].reshape(-1, D)[cut].double()
                V = s["v_cache"][pg, :, h].reshape(-1, D)[cut].double()
                if "k_scale" in s:
                    K, V = K * s["k_scale"][h].double(), V * s["v_scale"][h].double()
                of = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                x = (q[b, of] @ K.T) * s["scale"]
                lse[b, of] = torch.logsumexp(x, -1)
                out[b, of] = torch.softmax(x, -1) @ V
        return {"out": out, "lse": lse}
    # one row at a time: the kept tokens by a loop over the restrictions, then their shares
    probs = []
    B = s["logits"].shape[0]
    for b in range(B):
        x = s["logits"][b].double().nan_to_num(float("-inf"), _FLT_MAX, float("-inf"))
        x, idx = torch.sort(x, descending=True, stable=True)
        T = float(s["temperature"][b])
        n = int((x > float("-inf")).sum())
        if n == 0:
            probs.append(0.0)
            continue
        if T <= 0:
            n = 1
            T = 1.0
        if s["top_k"] is not None and 0 < int(s["top_k"][b]) < n:
            n = int(s["top_k"][b])
        w = torch.exp((x[:n] - x[0]) / T)
        if s["min_p"] is not None:
            w = w[w >= min(1.0, float(s["min_p"][b]))]
        if s["top_p"] is not None and float(s["top_p"][b]) < 1.0:
            sums = torch.cumsum(w, 0)
            w = w[:1 + int((sums[:-1] < float(s["top_p"][b]) * sums[-1]).sum())]
        i, back = torch.sort(idx[:w.numel()])
        sums = torch.cumsum(w[back], 0)
        j = min(int((sums <= float(s["u"][b]) * sums[-1]).sum()), w.numel() - 1)
        probs.append(float(w[back][j] / sums[-1]))
    return {"ids": None, "probs": torch.tensor(probs, dtype=torch.float64, device="cuda")}
