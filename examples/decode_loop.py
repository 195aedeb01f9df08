"""A small decoder that serves requests with this package: block tables, paged
cache, attention, the MoE layer and sampling in one loop.

    python examples/decode_loop.py

Weights are random and there is no tokenizer: the point is how the calls fit
together.  Prompts go through the cache token by token like everything else,
requests finish at different times, their pages go back to the pool and
waiting requests take their rows.  The host reads the drawn tokens once a step,
as a server does that has to send them on; nothing else leaves the GPU.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_moe_route_gb300 as moe  # noqa: E402

_TORCH = {moe.F32: torch.float32, moe.BF16: torch.bfloat16}


class Decoder:
    """`layers` blocks of attention and MoE over one paged cache per layer."""

    def __init__(self, *, layers=2, H=256, I=128, E=8, k=2, Hq=8, Hkv=2, D=64, V=1000,
                 dtype=moe.BF16, kv_dtype=None, num_pages=64, page_size=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = _TORCH[dtype]
        self.k, self.Hq, self.Hkv, self.D, self.V = k, Hq, Hkv, D, V
        self.num_pages, self.page_size = num_pages, page_size

        def w(*shape):
            std = shape[-1] ** -0.5
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(self.dtype)

        self.embed = torch.randn(V, H, generator=g, device="cuda").to(self.dtype)
        self.head = w(V, H)
        kv = kv_dtype or self.dtype
        self.scales = {}
        if kv == torch.float8_e4m3fn:  # keys and values of unit size: 448 steps to 16
            one = torch.full((Hkv,), 16.0 / 448.0, device="cuda")
            self.scales = dict(k_scale=one, v_scale=one)
        self.blocks = []
        for _ in range(layers):
            self.blocks.append(dict(
                qkv=w((Hq + 2 * Hkv) * D, H), out=w(H, Hq * D), router=w(E, H),
                moe=moe.MoELayer(w(E, 2 * I, H), w(E, H, I), k=k, dtype=dtype),
                k_cache=torch.zeros(num_pages, page_size, Hkv, D, device="cuda").to(kv),
                v_cache=torch.zeros(num_pages, page_size, Hkv, D, device="cuda").to(kv)))

    @staticmethod
    def norm(x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def logits(self, tokens, step, block_table, err=None):
        """Logits of one new token per request (a row with slot -1 is idle)."""
        x = self.embed[tokens]
        for b in self.blocks:
            qkv = (self.norm(x) @ b["qkv"].t()).view(len(x), self.Hq + 2 * self.Hkv, self.D)
            q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], dim=1)
            moe.kv_append(k, v, step.slots, b["k_cache"], b["v_cache"], err=err, **self.scales)
            a = moe.attn_decode(q, b["k_cache"], b["v_cache"], block_table, step.seq_lens, err=err,
                                **self.scales)
            x = x + a.view(len(x), -1) @ b["out"].t()
            h = self.norm(x)
            x = x + b["moe"](h, (h @ b["router"].t()).contiguous())
        return (self.norm(x) @ self.head.t()).contiguous()


def generate(model, prompts, new_tokens, *, batch=4, max_pages=8, seed=0, **sampling):
    """Serve `prompts` (lists of token ids) on `batch` rows; returns the drawn
    tokens of each.  `sampling`: numbers for temperature, top_k, top_p, min_p."""
    for i, p in enumerate(prompts):
        if not p:
            raise ValueError(f"prompt {i} is empty")
    if new_tokens < 1 or not prompts:
        return [[] for _ in prompts], model.num_pages
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((batch, max_pages), -1, **i32)
    free = torch.arange(model.num_pages, **i32)
    n_free = torch.full((1,), model.num_pages, **i32)
    ctx, err = torch.zeros(batch, **i32), torch.zeros(1, **i32)
    rand = torch.Generator(device="cuda").manual_seed(seed)
    f32 = dict(dtype=torch.float32, device="cuda")
    per_row = {name: torch.full((batch,), v, **(i32 if name == "top_k" else f32))
               for name, v in sampling.items()}

    waiting = list(range(len(prompts)))
    answers = [[] for _ in prompts]
    rows, fed = [None] * batch, [0] * batch      # request on a row, tokens fed to it
    while waiting or any(r is not None for r in rows):
        for i in range(batch):
            if rows[i] is None and waiting:
                rows[i], fed[i] = waiting.pop(0), 0
        tokens = [0 if r is None else (prompts[r] + answers[r])[fed[i]] for i, r in enumerate(rows)]
        active = torch.tensor([int(r is not None) for r in rows], **i32)
        # an idle row keeps its place in the batch: its position is padded away
        step = moe.kv_step(ctx, active, table, free, n_free, page_size=model.page_size,
                           num_pages=model.num_pages, max_tokens=batch, n_free_out=n_free, err=err)
        # token rows are packed by request: spread them over the batch's rows
        slots = torch.where(active > 0, step.slots[step.starts[:-1].clamp(max=batch - 1).long()],
                            torch.full_like(ctx, -1))
        logits = model.logits(torch.tensor(tokens, device="cuda"), step._replace(slots=slots), table,
                              err=err)
        u = torch.rand(batch, generator=rand, device="cuda")
        ids, _ = moe.sample_tokens(logits, u, **per_row)
        ctx = step.seq_lens.clone()
        done = [0] * batch
        for i, t in enumerate(ids.tolist()):
            r = rows[i]
            if r is None:
                continue
            fed[i] += 1
            if fed[i] >= len(prompts[r]):
                answers[r].append(t)
            if len(answers[r]) == new_tokens:
                rows[i], done[i] = None, 1
        if any(done):
            d = torch.tensor(done, **i32)
            moe.kv_release(d, table, free, n_free, num_pages=model.num_pages, err=err)
            ctx = torch.where(d > 0, torch.zeros_like(ctx), ctx)
    rc, bits = moe.check_word(err)
    if rc:
        raise moe.MoeError(rc, f"decode loop: error bits {bits:#x}")
    return answers, int(n_free)


if __name__ == "__main__":
    model = Decoder()
    prompts = [[1, 2, 3], list(range(10, 40)), [7], [100, 200], [5] * 20, [9, 8]]
    answers, left = generate(model, prompts, 12, temperature=0.8, top_k=50, top_p=0.95)
    for p, a in zip(prompts, answers):
        print(f"{len(p):3d} prompt tokens -> {a}")
    print(f"{left} of {model.num_pages} pages free")
