"""The example's decode loop on the GPU: the operators together, against the
same model computed densely in 64 bits from its weights (no cache, no pages)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import serving_moe_route_gb300 as moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def loop():
    spec = importlib.util.spec_from_file_location(
        "decode_loop", os.path.join(ROOT, "examples", "decode_loop.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _dense_logits(model, tokens):
    """Logits after every token of one request, in 64 bits."""
    def norm(x):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)

    def w(t):
        return t.detach().double().cpu().numpy()

    x = w(model.embed)[tokens]
    n, D, G = len(tokens), model.D, model.Hq // model.Hkv
    for b in model.blocks:
        qkv = (norm(x) @ w(b["qkv"]).T).reshape(n, -1, D)
        q, k, v = np.split(qkv, [model.Hq, model.Hq + model.Hkv], axis=1)
        a = np.zeros((n, model.Hq, D))
        for h in range(model.Hq):
            s = q[:, h] @ k[:, h // G].T * D ** -0.5
            s[np.triu_indices(n, 1)] = -np.inf
            p = np.exp(s - s.max(-1, keepdims=True))
            a[:, h] = p / p.sum(-1, keepdims=True) @ v[:, h // G]
        x = x + a.reshape(n, -1) @ w(b["out"]).T
        h_ = norm(x)
        r = h_ @ w(b["router"]).T
        w13, w2 = w(b["moe"].w13), w(b["moe"].w2)
        y = np.zeros_like(x)
        for t in range(n):
            top = np.argsort(-r[t], kind="stable")[:model.k]
            e = np.exp(r[t, top] - r[t, top].max())
            for j, weight in zip(top, e / e.sum()):
                gate, up = np.split(w13[j] @ h_[t], 2)
                y[t] += weight * (w2[j] @ (gate / (1 + np.exp(-gate)) * up))
        x = x + y
    return norm(x) @ w(model.head).T


def test_greedy_tokens_follow_the_dense_model(loop):
    model = loop.Decoder(dtype=moe.F32, num_pages=40, page_size=5)
    prompts = [[1, 2, 3], list(range(10, 31)), [7], [100, 200], [5] * 12, [9, 8]]
    answers, left = loop.generate(model, prompts, 6, batch=3, temperature=0.0)
    assert left == model.num_pages          # every page came back
    for p, a in zip(prompts, answers):
        logits = _dense_logits(model, p + a)[len(p) - 1:-1]
        for row, token in zip(logits, a):
            # products of TF32 operands (2^-11 each) behind every logit: the
            # drawn token's may lie that much, times a few layers, below the best
            assert row[token] >= row.max() - 0.02 * np.abs(row).max()


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn])
def test_sampling_stays_within_top_k(loop, kv):
    model = loop.Decoder(kv_dtype=kv, num_pages=40)
    prompts = [[3] * n for n in (1, 30, 5, 17, 2)]
    answers, left = loop.generate(model, prompts, 8, batch=4, temperature=0.7, top_k=5, top_p=0.9)
    again, _ = loop.generate(model, prompts, 8, batch=4, temperature=0.7, top_k=5, top_p=0.9)
    assert left == model.num_pages and answers == again
    assert all(len(a) == 8 and all(0 <= t < model.V for t in a) for a in answers)


def test_a_pool_that_runs_out_is_reported(loop):
    model = loop.Decoder(num_pages=1)
    with pytest.raises(moe.MoeError):
        loop.generate(model, [[1] * 20], 4, batch=1, temperature=0.0)
