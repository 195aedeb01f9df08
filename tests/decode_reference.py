"""Plain numpy forms of the decode-step operators in 64 bits, written from the
definitions in ``include/moe_route.h``: loops over requests and tokens, no
code of the product."""
import numpy as np
import torch

BAD_PAGE, NO_SPACE = 16, 32


def kv_step(ctx, new, table, free, n_free, page, num_pages, max_tokens):
    """(slots, positions, starts, seq_lens, n_free, table, error bits)"""
    ctx = [max(0, int(c)) for c in ctx]
    new = [max(0, int(n)) for n in new]
    table = table.copy()
    width = table.shape[1]
    n_free = min(max(0, int(n_free)), len(free))
    stack = list(free[:n_free])
    bits = 0
    slots, positions = [-1] * max_tokens, [0] * max_tokens
    starts, row = [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        starts.append(row)
        have, need = -(-c // page), -(-(c + n) // page)
        if need > width and n > 0:
            bits |= NO_SPACE
        fresh = {}
        for col in range(min(have, width), min(need, width)):
            if stack:
                got = int(stack.pop())
                if not 0 <= got < num_pages:
                    got, bits = -1, bits | BAD_PAGE
            else:
                got, bits = -1, bits | NO_SPACE
            fresh[col] = got
        for i in range(n):
            pos, at = c + i, row + i
            if at >= max_tokens:
                bits |= NO_SPACE
                break
            positions[at] = pos
            col = pos // page
            if col >= width:
                continue
            pg = fresh[col] if col in fresh else int(table[r, col])
            if col not in fresh and not 0 <= pg < num_pages:
                bits |= BAD_PAGE
                continue
            if pg >= 0:
                slots[at] = pg * page + pos % page
        for col, pg in fresh.items():
            table[r, col] = pg
        row += n
    starts.append(row)
    return (np.array(slots), np.array(positions), np.array(starts),
            np.array([c + n for c, n in zip(ctx, new)]), len(stack), table, bits)


def kv_release(done, table, free, n_free, num_pages):
    table, free = table.copy(), free.copy()
    bits = 0
    for r, d in enumerate(done):
        if not d:
            continue
        for pg in table[r]:
            if 0 <= pg < num_pages:
                if n_free < len(free):
                    free[n_free] = pg
                    n_free += 1
                else:
                    bits |= NO_SPACE
        table[r] = -1
    return table, free, n_free, bits


def attend(q, k, v, table, lens, scale, window=0, k_scale=None, v_scale=None):
    """q [B, Hq, D], k and v [pages, page, Hkv, D] as float64 arrays.  Returns
    out, lse, and per (b, h) what error bounds need: sum_t p |v| [B, Hq, D],
    the largest sum_d |q k| * scale, and the number of attended tokens."""
    B, Hq, D = q.shape
    pages, page, Hkv, _ = k.shape
    G = Hq // Hkv
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    pv, dot, count = np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, Hq))
    for b in range(B):
        n = min(max(0, int(lens[b])), table.shape[1] * page)
        first = max(0, n - window) if window else 0
        pos = np.arange(first, n)
        pg = table[b, pos // page].astype(np.int64)
        ok = (pg >= 0) & (pg < pages)
        pos, pg = pos[ok], pg[ok]
        if not len(pos):
            continue
        for h in range(Hq):
            g = h // G
            K, V = k[pg, pos % page, g], v[pg, pos % page, g]
            if k_scale is not None:
                K, V = K * float(k_scale[g]), V * float(v_scale[g])
            s = K @ q[b, h] * scale
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            out[b, h] = p @ V
            lse[b, h] = m + np.log(e.sum())
            pv[b, h] = p @ np.abs(V)
            dot[b, h] = (np.abs(K) @ np.abs(q[b, h])).max() * abs(scale)
            count[b, h] = len(pos)
    return out, lse, pv, dot, count


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, largest=np.inf):
    """ids and probs of every row (largest: what +inf counts as), how near a
    border the draw and the top-p cut came, and how far the sums they are
    compared with may be off: weights that are right to 2^-35 of themselves and
    to 2^-45 of the largest one, on both sides of the border.  Both as a share
    of the kept sum."""
    B, V = logits.shape
    ids, probs, near, off = np.full(B, -1), np.zeros(B), np.ones(B), np.zeros(B)
    for b in range(B):
        x = logits[b].astype(np.float64)
        x = np.where(np.isnan(x), -np.inf, np.minimum(x, largest))
        order = np.lexsort((np.arange(V), -x))
        order = order[x[order] > -np.inf]
        if not len(order):
            continue
        t = 1.0 if temperature is None else float(temperature[b])
        if not t > 0:
            ids[b], probs[b] = order[0], 1.0
            continue
        with np.errstate(over="ignore"):
            w = np.exp((x - x[order[0]]) / t)
        kept = order
        if top_k is not None and 0 < top_k[b] < len(kept):
            kept = kept[:top_k[b]]
        if min_p is not None and min_p[b] > 0:
            kept = kept[w[kept] >= min(1.0, float(min_p[b]))]
        if top_p is not None and top_p[b] < 1:
            before = np.concatenate([[0.0], np.cumsum(w[kept])[:-1]])
            border = float(top_p[b]) * w[kept].sum()
            inside = before < border
            inside[0] = True
            if len(kept) > 1:
                near[b] = np.abs(before[1:] - border).min() / w[kept].sum()
            kept = kept[inside]
        kept = np.sort(kept)
        sums = np.cumsum(w[kept])
        border = min(max(float(u[b]), 0.0), 1.0) * sums[-1]
        j = min(int((sums <= border).sum()), int(np.flatnonzero(w[kept])[-1]))
        near[b] = min(near[b], np.abs(sums - border).min() / sums[-1])
        ids[b], probs[b] = kept[j], w[kept[j]] / sums[-1]
        off[b] = 2 * (2.0 ** -35 + len(order) * 2.0 ** -45 / sums[-1])
    return ids, probs, near, off


def f64(t):
    """A tensor's values as float64 on the host."""
    return t.detach().float().cpu().double().numpy() if t.dtype != torch.float64 else t.cpu().numpy()
