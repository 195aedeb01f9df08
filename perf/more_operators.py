"""Operators of a decode step that checks drafted tokens, as cases to be measured.

    tree     attention of a tree of drafted tokens per request over the paged cache
    verify   masks and positions of such trees, the walk along the drawn tokens, and the
             accepted tokens' keys and values moved together
    fork     pages given back, and requests forked: shared pages, one copied
    adjust   penalties for repeated tokens, biases and grammar masks on logits

``run`` computes a case in plain torch operations, or through the package's
entry points where ``own`` is true.  Shapes are those of the package's decode
workloads (hidden size 2048: 32 query heads of 128 on 4 key-value heads) and
generic ones; every value comes from the seed.
"""
import math

import torch

own = False

_KV = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one short conversation with a chain of drafted tokens: nothing but latency
        dict(name="tree_one_short_bf16", op="tree", B=1, nodes=8, even=True, chain=True, Hq=32, Hkv=4,
             D=128, page=16, kv="bf16", ctx=700, window=0, idle=0, major="token"),
        # an ordinary batch, small trees of different sizes, a few rows of the batch idle
        dict(name="tree_batch_bf16", op="tree", B=64, nodes=16, even=False, chain=False, Hq=32, Hkv=4,
             D=128, page=16, kv="bf16", ctx=4096, window=0, idle=3, major="token"),
        # the same batch with full trees over longer contexts: products, not bytes
        dict(name="tree_wide_bf16", op="tree", B=64, nodes=64, even=True, chain=False, Hq=32, Hkv=4,
             D=128, page=16, kv="bf16", ctx=8192, window=0, idle=0, major="token"),
        # one request with a long document and a full tree
        dict(name="tree_one_long_bf16", op="tree", B=1, nodes=61, even=True, chain=False, Hq=32, Hkv=4,
             D=128, page=64, kv="bf16", ctx=131089, window=0, idle=0, major="head"),
        # a large batch with an 8-bit cache and a short chain each
        dict(name="tree_batch_e4m3", op="tree", B=128, nodes=8, even=True, chain=True, Hq=32, Hkv=4,
             D=128, page=16, kv="e4m3", ctx=8192, window=0, idle=5, major="token"),
        # the f32 layer's small model: odd sizes, a page size that is no power of two, a window
        dict(name="tree_window_f32", op="tree", B=5, nodes=13, even=False, chain=False, Hq=6, Hkv=2,
             D=80, page=5, kv="f32", ctx=3000, window=1000, idle=1, major="token"),
        # one conversation's chain: latency
        dict(name="verify_one", op="verify", B=1, nodes=8, even=True, ctx=700, Hkv=4, D=128, page=16,
             kv="bf16", major="token"),
        # a full batch of full trees, the cache kept head by head
        dict(name="verify_batch", op="verify", B=128, nodes=64, even=True, ctx=1024, Hkv=4, D=128,
             page=16, kv="bf16", major="head"),
        # four answers to one prompt
        dict(name="fork_one", op="fork", parents=1, children=4, ctx=900, Hkv=4, D=128, page=16,
             kv="bf16", major="token"),
        # beams: every prompt of a batch with eight of them, large pages
        dict(name="fork_batch", op="fork", parents=48, children=8, ctx=2048, Hkv=4, D=128, page=64,
             kv="bf16", major="token"),
        # the nodes of small trees, odd vocabulary, every restriction, part of the requests under a grammar
        dict(name="adjust_trees_bf16", op="adjust", R=16, per=4, V=50257, dtype="bf16", history=4096,
             bias=40, grammar=0.3, penalties=True),
        # a large batch, one token each, long histories
        dict(name="adjust_large_f32", op="adjust", R=512, per=1, V=131072, dtype="f32", history=8192,
             bias=100, grammar=0.1, penalties=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tree", "verify", "fork", "adjust", "adjust"])
    kv = rng.choice(["bf16", "bf16", "bf16", "e4m3", "e4m3", "f32"])
    major, page = rng.choice(["token", "head"]), rng.choice([1, 5, 8, 16, 16, 32, 64, 128])
    if op == "tree":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128, 128, 256])
        G = rng.choice([1, 3, 4, 7, 8, 8, 16])
        B = _log_int(rng, 1, 128)
        nodes = _log_int(rng, 1, min(128, (1 << 25) // (B * Hkv * G * D)))
        # at most half a gigabyte of keys and values, were every request the longest, and at
        # most the products of the listed cases (f32: a fortieth of them)
        room = (1 << 28) // (B * Hkv * D * {"f32": 4, "bf16": 2, "e4m3": 1}[kv])
        products = (1 << 30) // (B * nodes * Hkv * G * D) * (1 if kv == "f32" else 40)
        ctx = _log_int(rng, 1, max(1, min(131072, room, products)))
        return dict(op=op, B=B, nodes=nodes, even=rng.random() < 0.5, chain=rng.random() < 0.3,
                    Hq=Hkv * G, Hkv=Hkv, D=D, page=page, kv=kv, ctx=ctx,
                    window=rng.choice([0, 0, 0, 100, 1024]), idle=rng.choice([0, 0, B // 8]),
                    major=major)
    shape = dict(Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 80, 96, 128, 256]), page=page, kv=kv,
                 major=major)
    if op == "verify":
        B = _log_int(rng, 1, 128)
        return dict(op=op, B=B, nodes=_log_int(rng, 1, 128), even=rng.random() < 0.5,
                    ctx=_log_int(rng, 1, 1024 if B > 32 else 4096), **shape)
    if op == "fork":
        return dict(op=op, parents=_log_int(rng, 1, 48), children=rng.choice([1, 2, 3, 4, 5, 8]),
                    ctx=_log_int(rng, 1, 2048), **shape)
    per, R = rng.choice([1, 1, 1, 4, 7]), _log_int(rng, 1, 256)
    return dict(op=op, R=R, per=per, V=_log_int(rng, 1000, min(262144, (1 << 26) // (R * per))),
                dtype=rng.choice(["f32", "bf16"]), history=_log_int(rng, 1, 16384),
                bias=rng.choice([0, 0, 1, 40, 300]), grammar=rng.choice([0.0, 0.1, 0.5, 1.0]),
                penalties=rng.random() < 0.75)


# ------------------------------------------------------------------ their inputs
def _cache(g, pages, page, Hkv, D, dtype, major):
    """Keys and values [pages, page, Hkv, D], stored token by token or head by head."""
    kv = []
    for _ in range(2):
        shape = (pages, Hkv, page, D) if major == "head" else (pages, page, Hkv, D)
        t = torch.empty(shape, dtype=_KV[dtype], device="cuda")
        step = max(1, (1 << 26) // (page * Hkv * D))  # bounds the f32 copy
        for p in range(0, pages, step):
            x = torch.randn(t[p:p + step].shape, generator=g, device="cuda")
            t[p:p + step] = (x * 40 if dtype == "e4m3" else x).to(_KV[dtype])
        kv.append(t.transpose(1, 2) if major == "head" else t)
    return kv


def _lengths(n, longest):
    """n lengths 1 .. longest, half of them even and half spread over their logarithm; the last is
    the longest.  They are the same for every seed, which gives their order."""
    a = (torch.arange(n, device="cuda", dtype=torch.float64) + 0.5) / n
    spread = torch.exp(a * math.log(longest + 1)).floor()
    lens = torch.where(torch.arange(n, device="cuda") % 2 == 0, (a * longest).floor() + 1, spread)
    lens[-1] = longest
    return lens.clamp(1, longest).to(torch.int32)


def _table(g, need, width, spare):
    """A block table of rows with `need` pages each out of a shuffled pool, -1 behind them; the pool."""
    pages = int(need.sum()) + spare
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    at = ((torch.cumsum(need, 0) - need)[:, None] + col[None, :]).clamp(max=pages - 1)
    table = torch.where(col[None, :] < need[:, None], ids[at], torch.full_like(ids[at], -1))
    return table.contiguous(), ids


def _rows_of(new):
    """(starts, request of each row, index of each row in its request)"""
    starts = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)]).to(torch.int32)
    req = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new.long())
    return starts, req, torch.arange(len(req), device="cuda") - starts[req].long()


def _ancestors(parents, starts, req, index, width):
    """[N, width] truth values: which nodes of its request lie between a node and its root."""
    at = torch.arange(width, device=parents.device)
    anc = at[None, :] == index[:, None]
    up = torch.where(parents >= 0, starts[req].long() + parents, torch.arange(len(req), device=req.device))
    for _ in range(max(1, width.bit_length())):  # each round doubles the distance looked up
        anc = anc | anc[up]
        up = up[up]
    return anc


def _pack(bits):
    """[N, width] truth values as [N, words] of 64 bits."""
    n, width = bits.shape
    words = -(-width // 64)
    padded = torch.zeros(n, words * 64, dtype=torch.long, device=bits.device)
    padded[:, :width] = bits
    shifts = torch.arange(64, device=bits.device)
    return (padded.view(n, words, 64) << shifts).sum(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    c, op = dict(case), case["op"]
    s = {"op": op}

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def requests(B, nodes, idle=0):
        """Tokens in the cache and drafted ones of B requests, `idle` of them without any, in an
        order of the seed's"""
        ctx = _lengths(B, c["ctx"])
        new = torch.full((B,), nodes, dtype=torch.int32, device="cuda")
        if not c["even"]:
            new = (nodes - torch.arange(B, device="cuda") * 7 % nodes).to(torch.int32)
        ctx[:idle], new[:idle] = 0, 0
        order = torch.randperm(B, generator=g, device="cuda")
        return ctx[order], new[order]

    if op == "tree":
        B, Hq, Hkv, D, page, nodes = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], c["nodes"]
        ctx, new = requests(B, nodes, c["idle"])  # (rows of the batch that no request has)
        lens = ctx + new
        starts, req, index = _rows_of(new)
        if not c["chain"]:
            parents = (uniform(len(req)) * index).floor().long().clamp(max=nodes - 1)
            parents = torch.where(index > 0, torch.minimum(parents, index - 1), -torch.ones_like(index))
            s["masks"] = _pack(_ancestors(parents, starts, req, index, nodes))
        s["table"], ids = _table(g, (lens.long() + page - 1) // page, -(-(c["ctx"] + nodes) // page), 3)
        s["k_cache"], s["v_cache"] = _cache(g, len(ids), page, Hkv, D, c["kv"], c["major"])
        # what lies in a page after its last token may be anything
        rows = torch.nonzero((lens % page) > 0).flatten()
        pg = s["table"][rows, (lens[rows] // page).long()].long()
        for t in (s["k_cache"], s["v_cache"]):
            t[pg, (lens[rows] % page).long()] = torch.full((), float("nan"), device="cuda").to(t.dtype)
        src = torch.float32 if c["kv"] == "f32" else torch.bfloat16
        s["q"] = torch.randn(len(req), Hq, D, generator=g, device="cuda").to(src)
        if c["kv"] == "e4m3":
            s["k_scale"], s["v_scale"] = 0.02 + 0.01 * uniform(Hkv), 0.02 + 0.01 * uniform(Hkv)
        s.update(starts=starts, lens=lens, page=page, nodes=nodes, longest=c["ctx"] + nodes,
                 window=c["window"], scale=1.0 / math.sqrt(D))
    elif op == "verify":
        B, page, nodes = c["B"], c["page"], c["nodes"]
        ctx, new = requests(B, nodes)
        starts, req, index = _rows_of(new)
        N = len(req)
        # the accepted ones: node 0, and further nodes behind the place that they move to
        depth = 1 + (uniform(B) * uniform(B) * new).floor().long().clamp(max=16)
        depth = torch.minimum(depth, (new.long() + 1) // 2)
        key = uniform(B, nodes)
        at = torch.arange(nodes, device="cuda")[None, :]
        key = torch.where((at >= depth[:, None]) & (at < new[:, None]), key, torch.full_like(key, 2.0))
        rank = torch.argsort(torch.argsort(key, dim=1), dim=1)
        on = (rank < depth[:, None] - 1) | (at == 0)
        before = torch.where(on, at, -torch.ones_like(at)).cummax(1).values  # the last one up to here
        before = torch.cat([-torch.ones_like(before[:, :1]), before[:, :-1]], 1)
        parents = (uniform(B, nodes) * at).floor().long()
        parents = torch.where(on, before, torch.minimum(parents, at - 1))
        tokens = torch.randint(32000, (B, nodes), generator=g, device="cuda")
        tokens = tokens * 64 + torch.arange(nodes, device="cuda") % 64  # siblings differ
        draws = torch.randint(32000, (B, nodes), generator=g, device="cuda") * 64 + 2048064
        # at an accepted node the next one's token was drawn, at the last another one
        nxt = torch.where(on, at, torch.full_like(at, nodes)).flip(1).cummin(1).values.flip(1)
        nxt = torch.cat([nxt[:, 1:], torch.full_like(nxt[:, :1], nodes)], 1)
        follow = on & (nxt < new[:, None])
        draws = torch.where(follow, torch.gather(tokens, 1, nxt.clamp(max=nodes - 1)), draws)
        flat = at.expand(B, nodes) < new[:, None]
        s["parents"], s["tokens"], s["draws"] = (t[flat].to(torch.int32) for t in (parents, tokens, draws))
        lens = ctx + new
        s["table"], ids = _table(g, (lens.long() + page - 1) // page, -(-(c["ctx"] + nodes) // page), 3)
        s["k_cache"], s["v_cache"] = _cache(g, len(ids), page, c["Hkv"], c["D"], c["kv"], c["major"])
        s.update(starts=starts, ctx=ctx, lens=lens, page=page, nodes=nodes, N=N, max_path=min(nodes, 17))
    elif op == "fork":
        P, F, page = c["parents"], c["parents"] * c["children"], c["page"]
        rows = P + F
        src = torch.arange(F, device="cuda") // c["children"]
        dst = rows - 1 - torch.arange(F, device="cuda")
        ctx = torch.zeros(rows, dtype=torch.int32, device="cuda")
        ctx[:P] = _lengths(P, c["ctx"])[torch.randperm(P, generator=g, device="cuda")]
        ctx[dst] = ctx[src]
        full = ctx.long() // page
        part = ctx.long() % page
        # parents hold pages of their own, children (of the step before) a last page, if it is a part
        need = torch.where(torch.arange(rows, device="cuda") < P, (ctx.long() + page - 1) // page,
                           (part > 0).long())
        own_rows, ids = _table(g, need, -(-c["ctx"] // page), 40)
        table = own_rows.clone()
        col = torch.arange(table.shape[1], device="cuda")[None, :]
        theirs = torch.where(col == full[dst][:, None], own_rows[dst][:, :1], -torch.ones_like(col).int())
        theirs = torch.where((part[dst] > 0)[:, None], theirs, -torch.ones_like(theirs))
        table[dst] = torch.where(col < full[dst][:, None], own_rows[src], theirs)
        refs = torch.zeros(len(ids), dtype=torch.int32, device="cuda")
        shared = own_rows[src][col < full[src][:, None]].long()
        refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
        free = torch.full((len(ids),), -1, dtype=torch.int32, device="cuda")
        free[:40] = ids[-40:]
        s["k_cache"], s["v_cache"] = _cache(g, len(ids), page, c["Hkv"], c["D"], c["kv"], c["major"])
        keep = ctx.clone()
        keep[P:] = 0
        s.update(table=table, ctx=ctx, keep=keep, refs=refs, free=free, src=src.to(torch.int32),
                 dst=dst.to(torch.int32), page=page, pool=len(ids),
                 n_free=torch.full((1,), 40, dtype=torch.int32, device="cuda"))
    else:
        R, per, V, L = c["R"], c["per"], c["V"], c["history"]
        N = R * per
        x = 1.8 * torch.randn(N, V, generator=g, device="cuda")
        s["logits"] = (x + 4.0 * (uniform(N, V) < 0.001)).to(torch.float32 if c["dtype"] == "f32"
                                                             else torch.bfloat16)
        # tokens of a text: a few are frequent
        s["history"] = (V * uniform(R, L) ** 4).to(torch.int32).clamp(max=V - 1)
        s["history_lens"] = _lengths(R, L)[torch.randperm(R, generator=g, device="cuda")]
        s["prompt_lens"] = (uniform(R) * s["history_lens"]).to(torch.int32)
        s["rows"] = None
        if per > 1:
            s["rows"] = torch.arange(R, device="cuda").repeat_interleave(per).to(torch.int32)
        s["repetition"] = torch.where(uniform(R) < 0.3, torch.ones(R, device="cuda"), 1.0 + 0.3 * uniform(R))
        s["presence"], s["frequency"] = 0.5 * uniform(R), 0.3 * uniform(R)
        if not c["penalties"]:  # none asked for in this batch
            s["history"] = None
        s["bias_ids"] = s["bias"] = s["allowed"] = None
        if c["bias"]:
            ids = torch.argsort(uniform(R, min(V, 4096)), dim=1)[:, :c["bias"]] * max(1, V // 4096)
            some = uniform(R, 1) < 0.5  # a request without biases has a list of -1
            s["bias_ids"] = torch.where(some, ids, torch.full_like(ids, -1)).to(torch.int32).contiguous()
            s["bias"] = 10.0 * (uniform(*s["bias_ids"].shape) - 0.5)
        if c["grammar"]:
            bits = (uniform(N, -(-V // 32), 32) < 0.02).long()
            words = (bits << torch.arange(32, device="cuda")).sum(-1)
            free_rows = uniform(N, 1) >= c["grammar"]
            words = torch.where(free_rows, torch.full_like(words, 0xffffffff), words)
            s["allowed"] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return s


# ------------------------------------------------------------------ their plain forms
def _tree_plain(s):
    q, page, n, W = s["q"].float(), s["page"], s["longest"], s["nodes"]
    N, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    starts, lens = s["starts"].long(), s["lens"].long()
    new = starts[1:] - starts[:-1]
    ctx = lens - new
    B = len(new)
    at = torch.arange(W, device=q.device)
    real = at[None, :] < new[:, None]
    row = (starts[:-1, None] + at[None, :]).clamp(max=max(0, N - 1))
    # which drafted tokens each row attends [B, W, W], and how many
    if "masks" in s:
        word = s["masks"][row][:, :, at // 64]
        drafted = ((word >> (at % 64)) & 1).bool()
    else:
        drafted = (at[None, :] <= at[:, None]).expand(B, W, W)
    drafted = drafted & real[:, None, :] & real[:, :, None]
    pos = torch.arange(n, device=q.device)
    live = pos[None, :] < lens[:, None]
    see = (pos[None, :] < ctx[:, None])[:, None, :].expand(B, W, n)
    if s["window"]:
        first = ctx[:, None] - (s["window"] - drafted.sum(-1)).clamp(min=0)
        see = see & (pos >= first[:, :, None])
    back = pos[None, :] - ctx[:, None]
    inside = (back >= 0) & (back < new[:, None])
    own_part = torch.gather(drafted, 2, back.clamp(0, W - 1)[:, None, :].expand(B, W, n))
    see = see | (own_part & inside[:, None, :])
    pages = torch.where(live, s["table"][:, pos // page], torch.zeros_like(s["table"][:, :1])).long()
    zero = torch.zeros((), device=q.device)
    K = torch.where(live[:, :, None, None], s["k_cache"][pages, pos % page].float(), zero)
    K = K.permute(0, 2, 3, 1)
    if "k_scale" in s:
        K = K * s["k_scale"][None, :, None, None]
    G = Hq // Hkv
    qq = q[row].view(B, W, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * G, D)
    x = torch.matmul(qq, K).mul_(s["scale"]).view(B, Hkv, W, G, n)
    del K
    x.masked_fill_(~see[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    V = torch.where(live[:, :, None, None], s["v_cache"][pages, pos % page].float(), zero)
    V = V.permute(0, 2, 1, 3)
    o = torch.matmul(p.view(B, Hkv, W * G, n), V).view(B, Hkv, W, G, D)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    if "v_scale" in s:
        o = o * s["v_scale"][None, :, None, None, None]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, W, Hq, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, W, Hq)
    req, index = _positions(starts, N)
    return {"out": o[req, index].to(s["q"].dtype), "lse": lse[req, index]}


def _positions(starts, N):
    """Request and place in it of each of N rows."""
    i = torch.arange(N, device=starts.device)
    req = torch.searchsorted(starts[1:].contiguous(), i, right=True)
    return req, i - starts[req]


def _verify_plain(s):
    starts, N, W = s["starts"].long(), s["N"], s["nodes"]
    B = len(starts) - 1
    parents, tokens, draws = s["parents"].long(), s["tokens"], s["draws"]
    req, index = _positions(starts, N)
    new = starts[1:] - starts[:-1]
    anc = _ancestors(parents, starts, req, index, W)
    positions = (s["lens"].long() - new)[req] + anc.sum(-1) - 1
    # the walk
    path = torch.full((B, s["max_path"]), -1, dtype=torch.long, device=parents.device)
    cur = torch.where(new > 0, torch.zeros_like(new), -torch.ones_like(new))
    last = cur
    for step in range(s["max_path"]):
        path[:, step] = cur
        last = torch.where(cur >= 0, cur, last)
        want = draws[(starts[:-1] + cur.clamp(min=0)).clamp(max=N - 1)]
        hit = (cur[req] >= 0) & (parents == cur[req]) & (tokens == want[req]) & (index > 0)
        first = torch.full((B,), W, dtype=torch.long, device=parents.device)
        first.scatter_reduce_(0, req, torch.where(hit, index, torch.full_like(index, W)), "amin")
        cur = torch.where(first < W, first, -torch.ones_like(first))
    accepted = (path >= 0).sum(-1)
    nxt = draws[(starts[:-1] + last.clamp(min=0)).clamp(max=N - 1)]
    nxt = torch.where(last >= 0, nxt, -torch.ones_like(nxt))
    # the accepted tokens' keys and values, together
    page, ctx = s["page"], s["ctx"].long()
    b, j = torch.nonzero(path >= 0, as_tuple=True)
    a, to = ctx[b] + path[b, j], ctx[b] + j
    pa, pt = s["table"][b, a // page].long(), s["table"][b, to // page].long()
    for cache in (s["k_cache"], s["v_cache"]):
        cache[pt, to % page] = cache[pa, a % page]
    return {"masks": _pack(anc), "positions": positions.int(), "path": path.int(),
            "accepted": accepted.int(), "next": nxt.int(), "seq_lens": (ctx + accepted).int(),
            "k": s["k_cache"], "v": s["v_cache"]}


def _fork_plain(s):
    table, refs, free, n_free, page = s["table"], s["refs"], s["free"], s["n_free"], s["page"]
    ctx, keep = s["ctx"].long(), s["keep"].long()
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    # pages past what is kept: one holder fewer, and free where that was the last
    drop = (col >= ((keep + page - 1) // page)[:, None]) & (col < ((ctx + page - 1) // page)[:, None])
    pg = table[drop].long()
    refs.index_add_(0, pg, torch.full_like(pg, -1, dtype=torch.int32))
    gone = refs[pg] < 0
    first = torch.full((s["pool"],), pg.numel(), dtype=torch.long, device=pg.device)
    order = torch.arange(pg.numel(), device=pg.device)
    first.scatter_reduce_(0, pg, order, "amin")
    back = pg[gone & (first[pg] == order)]
    refs.clamp_(min=0)
    at = n_free.long() + torch.arange(back.numel(), device=pg.device)
    free[at] = back.int()
    n_free += back.numel()
    table.masked_fill_(drop, -1)
    # the forks
    src, dst = s["src"].long(), s["dst"].long()
    n = ctx[src]
    full, part = n // page, n % page
    take = (part > 0).long()
    rank = torch.cumsum(take, 0) - take
    fresh = free[(n_free.long() - 1 - rank).clamp(min=0)]
    rows = torch.where(col < full[:, None], table[src], -torch.ones_like(table[src]))
    rows = torch.where((col == full[:, None]) & (part > 0)[:, None], fresh[:, None], rows)
    shared = table[src][col < full[:, None]].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    a = table[src, full.clamp(max=table.shape[1] - 1)]
    none = torch.full_like(fresh, -1)
    a, to = torch.where(part > 0, a, none), torch.where(part > 0, fresh, none)
    table[dst] = rows
    s["ctx"][dst] = s["ctx"][src]
    n_free -= take.sum().int()
    # and the copied tokens
    f, t = torch.nonzero(torch.arange(page, device=pg.device)[None, :] < part[:, None], as_tuple=True)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[to[f].long(), t] = cache[a[f].long(), t]
    return {"src_pages": a, "dst_pages": to, "tokens": part.int(), "table": table, "refs": refs,
            "free": free, "n_free": n_free, "ctx": s["ctx"], "k": s["k_cache"], "v": s["v_cache"]}


def _adjust_plain(s):
    x = s["logits"].float()
    N, V = x.shape
    rows = torch.arange(N, device=x.device) if s["rows"] is None else s["rows"].long()
    if s["history"] is not None:
        h = s["history"].long()
        at = torch.arange(h.shape[1], device=x.device)[None, :]
        live = at < s["history_lens"][:, None]
        output = live & (at >= s["prompt_lens"][:, None])
        seen = torch.zeros(h.shape[0], V, dtype=torch.int32, device=x.device)
        seen.scatter_add_(1, h, live.int())
        count = torch.zeros_like(seen).scatter_add_(1, h, output.int())
        rep = s["repetition"][rows][:, None]
        x = torch.where(seen[rows] > 0, torch.where(x > 0, x / rep, x * rep), x)
        del seen
        count = count[rows]
        x = x - s["frequency"][rows][:, None] * count
        x = x - s["presence"][rows][:, None] * (count > 0)
    if s["bias_ids"] is not None:
        ids = s["bias_ids"][rows].long()
        real = ids >= 0
        x = x.scatter_add(1, ids.clamp(min=0), s["bias"][rows] * real)
    if s["allowed"] is not None:
        i = torch.arange(V, device=x.device)
        bit = (s["allowed"][:, i // 32] >> (i % 32).int()) & 1
        x = x.masked_fill(bit == 0, float("-inf"))
    return {"logits": x.to(s["logits"].dtype)}


def run(state):
    s, op = state, state["op"]
    if own:
        import serving_moe_route_gb300 as moe

        if op == "tree":
            out, lse = moe.attn_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["starts"],
                                     s["lens"], s.get("masks"), max_new=s["nodes"], scale=s["scale"],
                                     window=s["window"], k_scale=s.get("k_scale"),
                                     v_scale=s.get("v_scale"), return_lse=True)
            return {"out": out, "lse": lse}
        if op == "verify":
            t = moe.tree_masks(s["parents"], s["starts"], s["lens"], max_new=s["nodes"])
            a = moe.tree_accept(s["tokens"], s["draws"], s["parents"], s["starts"], s["ctx"],
                                max_path=s["max_path"])
            moe.kv_compact(a.path, a.accepted, s["ctx"], s["table"], s["k_cache"], s["v_cache"])
            return {"masks": t.masks, "positions": t.positions, "path": a.path,
                    "accepted": a.accepted, "next": a.next_ids, "seq_lens": a.seq_lens,
                    "k": s["k_cache"], "v": s["v_cache"]}
        if op == "fork":
            moe.kv_trim(s["keep"], s["ctx"], s["table"], s["free"], s["n_free"], page_size=s["page"],
                        num_pages=s["pool"], page_refs=s["refs"])
            f = moe.kv_fork(s["src"], s["dst"], s["ctx"], s["table"], s["refs"], s["free"], s["n_free"],
                            page_size=s["page"], num_pages=s["pool"])
            moe.kv_copy_pages(f.src_pages, f.dst_pages, s["k_cache"], s["v_cache"], tokens=f.tokens)
            return {"src_pages": f.src_pages, "dst_pages": f.dst_pages, "tokens": f.tokens,
                    "table": s["table"], "refs": s["refs"], "free": s["free"], "n_free": s["n_free"],
                    "ctx": s["ctx"], "k": s["k_cache"], "v": s["v_cache"]}
        past = {}
        if s["history"] is not None:
            past = dict(history=s["history"], history_lens=s["history_lens"],
                        prompt_lens=s["prompt_lens"], repetition=s["repetition"],
                        presence=s["presence"], frequency=s["frequency"])
        return {"logits": moe.adjust_logits(s["logits"], rows=s["rows"], bias_ids=s["bias_ids"],
                                            bias=s["bias"], allowed=s["allowed"], **past)}
    return {"tree": _tree_plain, "verify": _verify_plain, "fork": _fork_plain,
            "adjust": _adjust_plain}[op](s)


# ------------------------------------------------------------------ what they cannot do without
def _mean_length(n, w=0):
    """Mean of `_lengths`, and of their last w where w > 0."""
    if w and w < n:
        return (0.5 * (w - w * w / (2 * n))
                + 0.5 * (w + w * math.log((n + 1) / (w + 1))) / math.log(n + 1))
    return 0.5 * (n + 1) / 2 + 0.5 * n / math.log(n + 1)


def work(case):
    c, op = case, case["op"]
    if op == "tree":
        mean = _mean_length(c["ctx"], c["window"])
        longest = min(c["ctx"], c["window"]) if c["window"] else c["ctx"]
        total = longest + max(0, c["B"] - 1 - c["idle"]) * mean
        n = c["nodes"] if c["even"] else (c["nodes"] + 1) / 2
        rows = n * (c["B"] - c["idle"])
        e = {"f32": 4, "bf16": 2, "e4m3": 1}[c["kv"]]
        q = 4 if c["kv"] == "f32" else 2
        return {"bytes": 2 * (total + rows) * c["Hkv"] * c["D"] * e + 2 * rows * c["Hq"] * c["D"] * q,
                "flops": 4 * total * n * c["Hq"] * c["D"]}
    e = {"f32": 4, "bf16": 2, "e4m3": 1}[c.get("kv", "bf16")]
    if op == "verify":
        n = c["nodes"] if c["even"] else (c["nodes"] + 1) / 2
        moved = min(n / 4, 16)  # the mean of a product of two uniform numbers
        token = 2 * c["Hkv"] * c["D"] * e
        return {"bytes": c["B"] * (n * (12 + 4 + 8 * -(-c["nodes"] // 64)) + 80 + 2 * moved * token),
                "flops": 0}
    if op == "fork":
        F = c["parents"] * c["children"]
        pages = F * (_mean_length(c["ctx"]) / c["page"] + 1)
        copied = F * min(c["page"] - 1, _mean_length(c["ctx"])) / 2
        # of each page: its id in two rows, its holders read and written twice
        return {"bytes": 4 * c["Hkv"] * c["D"] * e * copied + 24 * pages, "flops": 0}
    e = 4 if c["dtype"] == "f32" else 2
    N = c["R"] * c["per"]
    past = 4 * c["R"] * _mean_length(c["history"]) if c["penalties"] else 0
    words = N * c["V"] / 8 if c["grammar"] else 0
    return {"bytes": 2 * N * c["V"] * e + past + words + 8 * c["R"] * c["bias"],
            "flops": 4 * N * c["V"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("verify", "fork"):
        return None  # whole numbers, and values that are moved
    if op == "tree":
        q = s["q"].double()
        N, Hq, D = q.shape
        Hkv, page, G = s["k_cache"].shape[2], s["page"], Hq // s["k_cache"].shape[2]
        out = torch.zeros_like(q)
        lse = torch.full((N, Hq), float("-inf"), dtype=q.dtype, device=q.device)
        starts, lens = s["starts"].tolist(), s["lens"].tolist()
        for b, length in enumerate(lens):
            lo, n = starts[b], starts[b + 1] - starts[b]
            if n == 0:
                continue
            ctx = length - n
            attend = torch.zeros(n, length, dtype=torch.bool, device=q.device)
            for i in range(n):
                if "masks" in s:
                    words = [w % (1 << 64) for w in s["masks"][lo + i].tolist()]
                    drafted = [j for j in range(n) if words[j // 64] >> (j % 64) & 1]
                else:
                    drafted = list(range(i + 1))
                first = max(0, ctx - max(0, s["window"] - len(drafted))) if s["window"] else 0
                attend[i, first:ctx] = True
                attend[i, [ctx + j for j in drafted]] = True
            pg = s["table"][b, :-(-length // page)].long()
            for h in range(Hkv):
                K = s["k_cache"][pg, :, h].reshape(-1, D)[:length].double()
                V = s["v_cache"][pg, :, h].reshape(-1, D)[:length].double()
                if "k_scale" in s:
                    K, V = K * s["k_scale"][h].double(), V * s["v_scale"][h].double()
                for i0 in range(0, n, 16):
                    i1 = min(n, i0 + 16)
                    x = (q[lo + i0:lo + i1, h * G:(h + 1) * G] @ K.T) * s["scale"]
                    x = x.masked_fill(~attend[i0:i1, None, :], float("-inf"))
                    lse[lo + i0:lo + i1, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                    out[lo + i0:lo + i1, h * G:(h + 1) * G] = torch.softmax(x, -1) @ V
        return {"out": out, "lse": lse}
    x = s["logits"].double()
    N, V = x.shape
    for b in range(N):
        r = b if s["rows"] is None else int(s["rows"][b])
        if s["history"] is not None:
            n, p = int(s["history_lens"][r]), int(s["prompt_lens"][r])
            past = s["history"][r, :n].long()
            seen = torch.unique(past)
            rep = float(s["repetition"][r])
            v = x[b, seen]
            x[b, seen] = torch.where(v > 0, v / rep, v * rep)
            said, times = torch.unique(past[p:], return_counts=True)
            x[b, said] -= float(s["frequency"][r]) * times + float(s["presence"][r])
        if s["bias_ids"] is not None:
            ids = s["bias_ids"][r].long()
            x[b, ids[ids >= 0]] += s["bias"][r][ids >= 0].double()
        if s["allowed"] is not None:
            words = s["allowed"][b].long() & 0xffffffff
            bits = (words[:, None] >> torch.arange(32, device=x.device)) & 1
            x[b, bits.flatten()[:V] == 0] = float("-inf")
    return {"logits": x}
