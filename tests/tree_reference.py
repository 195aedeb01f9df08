"""Plain numpy forms, in 64 bits, of the operators on drafted tokens, shared
pages and adjusted logits, written from the definitions in
``include/moe_route.h``: loops over requests, rows and tokens."""
import numpy as np

BAD_ID, DUP_ID, BAD_PAGE, NO_SPACE = 1, 2, 16, 32


def masks(parents, starts, lens, max_new, N):
    """(truth values [N, 64 * words], positions, error bits)"""
    words = -(-max_new // 64)
    out, pos, bits = np.zeros((N, 64 * words), bool), np.zeros(N, int), 0
    for r in range(len(lens)):
        lo, hi = starts[r], starts[r + 1]
        n = hi - lo
        if n > max_new:
            bits |= NO_SPACE
        for i in range(n):
            pos[lo + i] = max(0, lens[r] - n)
            if i >= max_new:
                continue
            p = parents[lo + i]
            if not -1 <= p < i:
                bits |= BAD_ID
                p = -1
            if p >= 0:
                out[lo + i] = out[lo + p]
            out[lo + i, i] = True
            pos[lo + i] += out[lo + i].sum() - 1
    return out, pos, bits


def packed(bits):
    """Truth values [N, 64 W] as int64 [N, W]."""
    n, width = bits.shape
    b = np.packbits(bits.reshape(n, width // 64, 64), axis=-1, bitorder="little")
    return b.view(np.int64).reshape(n, width // 64)


def accept(tokens, draws, parents, starts, ctx, max_path):
    """(path, accepted, next_ids, seq_lens)"""
    B = len(ctx)
    path, acc, nxt = np.full((B, max_path), -1), np.zeros(B, int), np.full(B, -1)
    for r in range(B):
        lo, n = starts[r], starts[r + 1] - starts[r]
        cur = 0 if n else None
        while cur is not None and acc[r] < max_path:
            path[r, acc[r]] = cur
            acc[r] += 1
            nxt[r] = draws[lo + cur]
            kids = [j for j in range(cur + 1, n)
                    if parents[lo + j] == cur and tokens[lo + j] == nxt[r] >= 0]
            cur = kids[0] if kids else None
    return path, acc, nxt, np.maximum(0, ctx) + acc


def attend(q, k, v, table, starts, lens, bits, max_new, scale, window=0, k_scale=None,
           v_scale=None):
    """q [N, Hq, D], k and v [pages, page, Hkv, D] as float64, bits [N, >= max_new]
    truth values or None.  Returns out, lse (rows of no request: NaN), and what
    error bounds need: sum_t p |v|, the largest sum_d |q k| * scale, how many
    tokens a row attends."""
    N, Hq, D = q.shape
    pages, page, Hkv, _ = k.shape
    G = Hq // Hkv
    out, lse = np.full((N, Hq, D), np.nan), np.full((N, Hq), np.nan)
    pv, dot, count = np.zeros((N, Hq, D)), np.zeros((N, Hq)), np.zeros((N, Hq))
    for r in range(len(lens)):
        lo, n = starts[r], starts[r + 1] - starts[r]
        ctx, length = max(0, lens[r] - n), min(max(0, lens[r]), table.shape[1] * page)
        for i in range(min(n, max_new)):
            drafted = [j for j in range(min(n, length - ctx))
                       if (j <= i if bits is None else j < bits.shape[1] and bits[lo + i, j])]
            if window:  # the last of them count, and of the context what is left
                drafted = drafted[-window:]
            first = max(0, ctx - (window - len(drafted))) if window else 0
            pos = np.array(list(range(first, min(ctx, length))) + [ctx + j for j in drafted], int)
            pg = table[r, pos // page].astype(np.int64)
            ok = (pg >= 0) & (pg < pages)
            pos, pg = pos[ok], pg[ok]
            out[lo + i], lse[lo + i], count[lo + i] = 0, -np.inf, len(pos)
            if not len(pos):
                continue
            for g in range(Hkv):
                K, V = k[pg, pos % page, g], v[pg, pos % page, g]
                if k_scale is not None:
                    K, V = K * float(k_scale[g]), V * float(v_scale[g])
                rows = slice(g * G, (g + 1) * G)
                s = q[lo + i, rows] @ K.T * scale
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                p = e / e.sum(-1, keepdims=True)
                out[lo + i, rows] = p @ V
                lse[lo + i, rows] = (m + np.log(e.sum(-1, keepdims=True)))[:, 0]
                pv[lo + i, rows] = p @ np.abs(V)
                dot[lo + i, rows] = (np.abs(q[lo + i, rows]) @ np.abs(K).T).max(-1) * abs(scale)
    return out, lse, pv, dot, count


def compact(path, accepted, ctx, table, cache, page):
    """(cache [pages, page, ...], error bits)"""
    pages, old, new, bits = cache.shape[0], cache, cache.copy(), 0

    def place(r, pos):
        if pos // page >= table.shape[1]:
            return None, NO_SPACE
        pg = table[r, pos // page]
        return ((pg, pos % page), 0) if 0 <= pg < pages else (None, BAD_PAGE)

    for r in range(len(ctx)):
        last = -1
        for j in range(min(max(0, accepted[r]), path.shape[1])):
            p = path[r, j]
            if p <= last:
                bits |= BAD_ID
                break
            last = p
            if p == j:
                continue
            (a, e1), (b, e2) = place(r, max(0, ctx[r]) + p), place(r, max(0, ctx[r]) + j)
            bits |= e1 | e2
            if a and b:
                new[b] = old[a]
    return new, bits


def fork(src, dst, ctx, table, refs, free, n_free, page, num_pages):
    """(pairs [F, 3], ctx, table, refs, n_free, error bits)"""
    ctx, table, refs = ctx.copy(), table.copy(), refs.copy()
    B, width = table.shape
    n_free = min(max(0, n_free), len(free))
    left, bits, pairs = n_free, 0, []
    first = {}
    for i, d in enumerate(dst):
        if 0 <= d < B:
            first.setdefault(int(d), i)
    old_ctx, old_table = ctx.copy(), table.copy()
    for i, (s, d) in enumerate(zip(src, dst)):
        pairs.append((-1, -1, 0))
        if not (0 <= s < B and 0 <= d < B):
            bits |= BAD_ID
            continue
        if first[int(d)] != i or int(s) in first:
            bits |= DUP_ID
            continue
        n = max(0, old_ctx[s])
        full, part = n // page, n % page
        if full + (part > 0) > width:
            bits |= NO_SPACE
            continue
        if part:
            a = old_table[s, full]
            if not 0 <= a < num_pages:  # no free page is taken for it
                bits |= BAD_PAGE
                continue
            left -= 1
            if left < 0:
                bits |= NO_SPACE
                continue
            b = free[left]
            if not 0 <= b < num_pages:
                bits |= BAD_PAGE
                continue
            table[d, full] = b
            pairs[-1] = (a, b, part)
        for c in range(full):
            pg = old_table[s, c]
            if 0 <= pg < num_pages:
                refs[pg] += 1
            else:
                pg, bits = -1, bits | BAD_PAGE
            table[d, c] = pg
        ctx[d] = n
    return np.array(pairs).reshape(-1, 3), ctx, table, refs, max(0, left), bits


def trim(keep, lens, table, free, n_free, page, num_pages, refs=None):
    """(table, free, n_free, refs, error bits)"""
    table, free = table.copy(), free.copy()
    refs = None if refs is None else refs.copy()
    width, bits = table.shape[1], 0
    n_free = min(max(0, n_free), len(free))
    entries = []
    for r in range(len(keep)):
        a, b = (min(width, -(-max(0, int(x)) // page)) for x in (keep[r], lens[r]))
        entries += [(r, c) for c in range(a, b)]
    pages = [int(table[e]) for e in entries]
    gone = []
    for pg in pages:
        if not 0 <= pg < num_pages:
            bits |= BAD_PAGE if pg != -1 else 0
        elif refs is None:
            gone.append(pg)
        else:
            refs[pg] -= 1
    if refs is not None:
        for pg in pages:
            if 0 <= pg < num_pages and refs[pg] < 0:
                gone.append(pg)
                refs[pg] = 0
    for pg in gone:
        if n_free < len(free):
            free[n_free] = pg
            n_free += 1
        else:
            bits |= NO_SPACE
    for e in entries:
        table[e] = -1
    return table, free, n_free, refs, bits


def adjust(x, rows=None, history=None, history_lens=None, prompt_lens=None, repetition=None,
           presence=None, frequency=None, bias_ids=None, bias=None, allowed=None, tokens=None,
           bits=None, starts=None):
    """x [N, V] float64, bits [N, >= nodes] truth values (``masks``); returns what the
    definition gives in 64 bits, and the sum of the magnitudes that were added up (for
    error bounds)."""
    x = x.copy()
    size = np.abs(x)
    N, V = x.shape
    for i in range(N):
        r = i if rows is None else int(rows[i])
        some = [a for a in (history, bias_ids) if a is not None]
        if some and 0 <= r < len(some[0]):
            if history is not None:
                h = history[r, :min(max(0, int(history_lens[r])), history.shape[1])]
                p = 0 if prompt_lens is None else min(max(0, int(prompt_lens[r])), len(h))
                if tokens is not None and starts[r] <= i < starts[r + 1]:
                    path = [j for j in range(1, min(starts[r + 1] - starts[r], bits.shape[1]))
                            if bits[i, j]]
                    h = np.concatenate([h, [tokens[starts[r] + j] for j in path]]).astype(int)
                for t in set(int(t) for t in h if 0 <= t < V):
                    if repetition is not None:
                        x[i, t] = (x[i, t] / repetition[r] if x[i, t] > 0 else x[i, t] * repetition[r])
                    c = int((h[p:] == t).sum())
                    f = 0.0 if frequency is None else frequency[r] * c
                    q = 0.0 if presence is None or c == 0 else presence[r]
                    size[i, t] = abs(x[i, t]) + abs(f) + abs(q)
                    x[i, t] -= f + q
            if bias_ids is not None:
                for t, b in dict((int(t), b) for t, b in zip(bias_ids[r], bias[r])).items():
                    if 0 <= t < V:
                        x[i, t] += b
                        size[i, t] += abs(b)
        if allowed is not None:
            bit = (allowed[i].astype(np.int64)[np.arange(V) // 32] >> (np.arange(V) % 32)) & 1
            x[i, bit == 0] = -np.inf
    return x, size
