"""The decoder of ``decode_loop.py`` with speculation, several answers to a prompt,
and penalties: drafted tokens are checked as a tree in one pass.

    python examples/speculative_loop.py

Drafts come from the request's own text (what followed the last tokens where they
occurred before), so nothing but the decoder is needed; a prompt goes through the
cache in chunks as a chain whose tokens are all accepted.  When a prompt is in the
cache, further answers fork from its row, each with a first token of its own: they
share its pages, and the last one is copied.  The host reads the accepted nodes once a
step, and what is drawn for such answers; nothing else leaves the GPU.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decode_loop import Decoder, moe  # noqa: E402


class TreeDecoder(Decoder):
    """Logits at every node of a tree per request."""

    def tree_logits(self, tokens, step, masks, block_table, max_new, err=None):
        x = self.embed[tokens]
        for b in self.blocks:
            qkv = (self.norm(x) @ b["qkv"].t()).view(len(x), self.Hq + 2 * self.Hkv, self.D)
            q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], dim=1)
            moe.kv_append(k, v, step.slots, b["k_cache"], b["v_cache"], err=err, **self.scales)
            # rows that pad the batch are no request's: attn_tree leaves them as they are
            a = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
            moe.attn_tree(q, b["k_cache"], b["v_cache"], block_table, step.starts, step.seq_lens,
                          masks, max_new=max_new, out=a, err=err, **self.scales)
            x = x + a.view(len(x), -1) @ b["out"].t()
            h = self.norm(x)
            x = x + b["moe"](h, (h @ b["router"].t()).contiguous())
        return (self.norm(x) @ self.head.t()).contiguous()


def draft(text, width, depth):
    """Up to `width` branches of up to `depth` tokens: what followed the latest
    other places of the text's last token, the longest of its ends first."""
    out = []
    for n in (3, 2, 1):
        end = text[-n:]
        for i in range(len(text) - n - 1, -1, -1):
            if len(out) == width:
                return out
            if text[i:i + n] == end and text[i + n:i + n + depth] not in out:
                out.append(text[i + n:i + n + depth])
    return out


def tree_of(root, branches, limit):
    """(tokens, parents) of a tree: node 0 and its branches, common beginnings once."""
    tokens, parents = [root], [-1]
    for branch in branches:
        at = 0
        for t in branch:
            kids = [j for j in range(at + 1, len(tokens)) if parents[j] == at and tokens[j] == t]
            if kids:
                at = kids[0]
            elif len(tokens) < limit:
                tokens.append(t)
                parents.append(at)
                at = len(tokens) - 1
            else:
                break
    return tokens, parents


def generate(model, prompts, new_tokens, *, samples=1, batch=4, max_new=8, max_pages=8, width=2,
             seed=0, repetition=None, frequency=None, banned=(), **sampling):
    """`samples` answers of `new_tokens` tokens to each prompt, on `batch` rows.
    `repetition`, `frequency`: penalties for repeated tokens, the prompt's among them;
    `banned`: tokens that are never drawn; `sampling`: numbers for temperature, top_k,
    top_p, min_p.  Returns the answers, the free pages at the end, and how many steps
    were taken."""
    for i, p in enumerate(prompts):
        if not p:
            raise ValueError(f"prompt {i} is empty")
    if samples > batch:
        raise ValueError("a prompt's answers need a row each")
    answers = [[[] for _ in range(samples)] for _ in prompts]
    if new_tokens < 1 or not prompts:
        return answers, model.num_pages, 0
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    pages = dict(page_size=model.page_size, num_pages=model.num_pages)
    table = torch.full((batch, max_pages), -1, **i32)
    free, refs = torch.arange(model.num_pages, **i32), torch.zeros(model.num_pages, **i32)
    n_free = torch.full((1,), model.num_pages, **i32)
    ctx, err = torch.zeros(batch, **i32), torch.zeros(1, **i32)
    rand = torch.Generator(device="cuda").manual_seed(seed)
    N = batch * max_new
    allowed = torch.full((N, -(-model.V // 32)), -1, **i32)
    for t in banned:
        allowed[:, t // 32] &= ~(1 << t % 32) if t % 32 < 31 else 0x7fffffff
    longest = max(map(len, prompts)) + new_tokens
    per_row = {name: torch.full((N,), v, **(i32 if name == "top_k" else f32))
               for name, v in sampling.items()}

    waiting = [(i, 0) for i in range(len(prompts))]
    rows, fed = [None] * batch, [0] * batch   # (prompt, answer) on a row; its tokens in the cache
    steps = 0
    while waiting or any(r is not None for r in rows):
        for i in range(batch):
            # a prompt begins when there are rows for all of its answers
            if rows[i] is None and waiting and sum(r is None for r in rows) >= samples \
                    and not any(r and fed[j] < len(prompts[r[0]]) for j, r in enumerate(rows)
                                if samples > 1):
                rows[i], fed[i] = waiting.pop(0), 0
        tokens, parents, forced, sizes, history = [], [], [], [], []
        for i, r in enumerate(rows):
            text = [] if r is None else prompts[r[0]] + answers[r[0]][r[1]]
            history.append(text + [-1] * (longest - len(text)))
            if r is None:
                t, p, known = [], [], []
            elif fed[i] < len(prompts[r[0]]) - 1:   # a chunk of the prompt: all of it is known
                t = prompts[r[0]][fed[i]:fed[i] + max_new]
                p = list(range(-1, len(t) - 1))
                known = prompts[r[0]][fed[i] + 1:fed[i] + 1 + len(t)]
                known += [-1] * (len(t) - len(known))
            else:
                left = new_tokens - len(answers[r[0]][r[1]])
                # (answers part at the first token: what forks has no drafts behind it)
                t, p = tree_of(text[-1], [] if samples > 1 and fed[i] < len(prompts[r[0]]) else
                               draft(text, width, min(left - 1, max_new - 1)), max_new)
                known = [-1] * len(t)
            tokens, parents, forced = tokens + t, parents + p, forced + known
            sizes.append(len(t))
        pad = N - len(tokens)
        tokens, parents, forced = (torch.tensor(x + [y] * pad, **i32) for x, y in
                                   ((tokens, 0), (parents, -1), (forced, -1)))
        row_of = torch.tensor([i for i, n in enumerate(sizes) for _ in range(n)] + [0] * pad, **i32)
        nodes = torch.tensor(sizes, **i32)
        step = moe.kv_step(ctx, nodes, table, free, n_free, max_tokens=N, n_free_out=n_free, err=err,
                           **pages)
        tree = moe.tree_masks(parents, step.starts, step.seq_lens, max_new=max_new, err=err)
        logits = model.tree_logits(tokens, step, tree.masks, table, max_new, err=err)
        past = {}
        if repetition or frequency:   # a drafted token's ancestors are text as well
            past = dict(history=torch.tensor(history, **i32), tokens=tokens, masks=tree.masks,
                        starts=step.starts, history_lens=torch.full((batch,), longest, **i32))
            past.update((name, torch.full((batch,), v, **f32)) for name, v in
                        (("repetition", repetition), ("frequency", frequency)) if v)
        logits = moe.adjust_logits(logits, rows=row_of, allowed=allowed, out=logits, err=err, **past)
        ids, _ = moe.sample_tokens(logits, torch.rand(N, generator=rand, device="cuda"), **per_row)
        draws = torch.where(forced >= 0, forced, ids)
        walk = moe.tree_accept(tokens, draws, parents, step.starts, ctx, max_path=max_new, err=err)
        for b in model.blocks:
            moe.kv_compact(walk.path, walk.accepted, ctx, table, b["k_cache"], b["v_cache"], err=err)
        steps += 1

        keep, forks, firsts = walk.seq_lens.clone(), [], []
        read = torch.cat([walk.path, walk.accepted[:, None], walk.next_ids[:, None]], 1).tolist()
        host = tokens.tolist()
        at = 0
        for i, r in enumerate(list(rows)):
            *path, accepted, last = read[i]
            lo, at = at, at + sizes[i]
            if r is None:
                continue
            prompt, text = prompts[r[0]], answers[r[0]][r[1]]
            fresh = [host[lo + j] for j in path[1:accepted]] + [last]
            before, fed[i] = fed[i], fed[i] + accepted
            if fed[i] < len(prompt):
                continue
            # (of a chunk of the prompt only what was drawn at its end is new)
            text += [last] if before < len(prompt) - 1 else fresh
            del text[new_tokens:]
            if before < len(prompt) and samples > 1:   # the prompt is in the cache: its other answers
                others = [j for j, x in enumerate(rows) if x is None][:samples - 1]
                for s, j in enumerate(others, 1):
                    rows[j], fed[j] = (r[0], s), fed[i]
                    firsts.append((lo + path[accepted - 1], answers[r[0]][s]))
                    forks.append((i, j))
        if firsts:   # drawn from the logits at the prompt's end
            ids, _ = moe.sample_tokens(logits[[row for row, _ in firsts]],
                                       torch.rand(len(firsts), generator=rand, device="cuda"),
                                       **{k: v[:len(firsts)] for k, v in per_row.items()})
            for (_, text), token in zip(firsts, ids.tolist()):
                text.append(token)
        done = [i for i, r in enumerate(rows) if r and len(answers[r[0]][r[1]]) == new_tokens]
        if forks:
            moe.kv_trim(keep, step.seq_lens, table, free, n_free, page_refs=refs, err=err, **pages)
            ctx = keep.clone()
            f = moe.kv_fork(*(torch.tensor(x, **i32) for x in zip(*forks)), ctx, table, refs, free,
                            n_free, err=err, **pages)
            for b in model.blocks:
                moe.kv_copy_pages(f.src_pages, f.dst_pages, b["k_cache"], b["v_cache"],
                                  tokens=f.tokens, err=err)
            keep, lens = ctx.clone(), ctx
        else:
            lens = step.seq_lens
        keep[done] = 0
        moe.kv_trim(keep, lens, table, free, n_free, page_refs=refs, err=err, **pages)
        ctx = keep
        for i in done:
            rows[i] = None
    rc, bits = moe.check_word(err)
    if rc:
        raise moe.MoeError(rc, f"speculative loop: error bits {bits:#x}")
    return answers, int(n_free), steps


if __name__ == "__main__":
    model = TreeDecoder()
    prompts = [[1, 2, 3, 1, 2, 3, 1, 2], list(range(10, 40)), [7] * 9, [100, 200], [9, 8]]
    answers, left, steps = generate(model, prompts, 12, samples=2, temperature=0.8, top_k=50,
                                    repetition=1.2)
    for p, two in zip(prompts, answers):
        for a in two:
            print(f"{len(p):3d} prompt tokens -> {a}")
    print(f"{steps} steps, {left} of {model.num_pages} pages free")
