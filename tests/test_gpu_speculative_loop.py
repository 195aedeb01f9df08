"""The example's speculative loop on the GPU: the calls on drafted tokens, shared
pages and adjusted logits together, against the same model computed densely in 64
bits (no cache, no pages, one token after the other)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import serving_moe_route_gb300 as moe
from test_gpu_decode_loop import _dense_logits

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROMPTS = [[1, 2, 3, 1, 2, 3, 1], list(range(10, 31)), [7], [100, 200], [5] * 12, [9, 8, 9, 8, 9]]


@pytest.fixture(scope="module")
def loop():
    spec = importlib.util.spec_from_file_location(
        "speculative_loop", os.path.join(ROOT, "examples", "speculative_loop.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _follows(model, prompt, answer, repetition=None, banned=()):
    """Every token of a greedy answer is the best there is, as far as the kernels'
    products of TF32 operands can tell (the decode loop's bound)."""
    logits = _dense_logits(model, prompt + answer)[len(prompt) - 1:-1]
    for i, (row, token) in enumerate(zip(logits, answer)):
        near = 0.02 * np.abs(row).max()
        if repetition:
            for t in set(prompt + answer[:i]):
                row[t] = row[t] / repetition if row[t] > 0 else row[t] * repetition
        row[list(banned)] = -np.inf
        assert row[token] >= row.max() - near


@pytest.mark.parametrize("max_new,page,width", [(1, 5, 1), (8, 5, 2), (16, 16, 3)])
def test_greedy_tokens_follow_the_dense_model(loop, max_new, page, width):
    model = loop.TreeDecoder(dtype=moe.F32, num_pages=60, page_size=page)
    answers, left, steps = loop.generate(model, PROMPTS, 9, batch=3, max_new=max_new, width=width,
                                         max_pages=16, temperature=0.0)
    assert left == model.num_pages               # every page came back
    for p, (a,) in zip(PROMPTS, answers):
        assert len(a) == 9
        _follows(model, p, a)


def test_drafts_are_accepted_where_the_text_repeats(loop):
    # a model that repeats itself: its greedy text is the best draft, fed as a prompt
    model = loop.TreeDecoder(dtype=moe.F32, num_pages=60, page_size=5)
    prompt = [3, 4]
    (plain,), _, slow = loop.generate(model, [prompt], 20, max_new=1, max_pages=16, temperature=0.0)
    (fast,), _, steps = loop.generate(model, [prompt], 20, max_new=8, max_pages=16, temperature=0.0)
    _follows(model, prompt, plain[0])
    _follows(model, prompt, fast[0])
    assert slow == len(prompt) + 19 and steps <= slow


def test_answers_fork_from_one_prompt(loop):
    # greedily all are the same one; the pages that they share come back
    model = loop.TreeDecoder(dtype=moe.F32, num_pages=80, page_size=5)
    answers, left, _ = loop.generate(model, PROMPTS, 7, samples=3, batch=6, max_new=8, max_pages=16,
                                     temperature=0.0)
    assert left == model.num_pages
    for p, three in zip(PROMPTS, answers):
        for a in three:
            _follows(model, p, a)


def test_penalties_and_banned_tokens(loop):
    # one node a request: a drafted token's own ancestors are not in its history
    model = loop.TreeDecoder(dtype=moe.F32, num_pages=60, page_size=5)
    banned = (31, 32, 999)
    answers, left, _ = loop.generate(model, PROMPTS, 8, batch=4, max_new=1, max_pages=16,
                                     temperature=0.0, repetition=1.5, banned=banned)
    for p, (a,) in zip(PROMPTS, answers):
        _follows(model, p, a, repetition=1.5, banned=banned)


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn])
def test_sampling_runs_and_repeats(loop, kv):
    model = loop.TreeDecoder(kv_dtype=kv, num_pages=60)
    kw = dict(samples=2, batch=4, temperature=0.7, top_k=5, top_p=0.9, repetition=1.1, banned=(4,))
    answers, left, _ = loop.generate(model, PROMPTS, 8, **kw)
    again, _, _ = loop.generate(model, PROMPTS, 8, **kw)
    assert left == model.num_pages and answers == again
    assert all(len(a) == 8 and all(0 <= t < model.V and t != 4 for t in a)
               for two in answers for a in two)


def test_a_pool_that_runs_out_is_reported(loop):
    model = loop.TreeDecoder(num_pages=1)
    with pytest.raises(moe.MoeError):
        loop.generate(model, [[1] * 20], 4, batch=1, temperature=0.0)


def test_trees_and_drafts_on_the_host(loop):
    assert loop.draft([1, 2, 3, 1, 2], 2, 3) == [[3, 1, 2]]
    assert loop.draft([5], 3, 3) == []
    tokens, parents = loop.tree_of(9, [[1, 2], [1, 3], [4]], 5)
    assert tokens == [9, 1, 2, 3, 4] and parents == [-1, 0, 1, 1, 0]
    assert loop.tree_of(9, [[1, 2, 3]], 2) == ([9, 1], [-1, 0])
    with pytest.raises(ValueError, match="empty"):
        loop.generate(None, [[]], 3)


def _right_drafts(prompts, answers):
    """Drafts that know the answers: a wrong sibling first, so that accepted nodes' keys
    and values have to move, and then the answer's next tokens."""
    def draft(text, width, depth):
        for p, (a,) in zip(prompts, answers):
            known = p + a
            if known[:len(text)] == text and depth > 0:
                right = known[len(text):len(text) + depth]
                return [[(right[0] + 1) % 1000], right] if right else []
        return []
    return draft


def test_tokens_on_a_nodes_path_are_penalised(loop, monkeypatch):
    # long paths are accepted, and every token is the best after the penalties of the text
    # before it, the step's own drafted tokens included
    model = loop.TreeDecoder(dtype=moe.F32, num_pages=60, page_size=5)
    prompts = [[1, 2, 3], [7], [5] * 4]
    kw = dict(batch=3, max_pages=16, temperature=0.0, repetition=1.2, frequency=0.6)
    plain, _, slow = loop.generate(model, prompts, 20, max_new=1, **kw)
    monkeypatch.setattr(loop, "draft", _right_drafts(prompts, plain))
    fast, left, steps = loop.generate(model, prompts, 20, max_new=8, **kw)
    assert left == model.num_pages and steps < slow
    for p, (a,) in zip(prompts, fast):
        logits = _dense_logits(model, p + a)[len(p) - 1:-1]
        for i, (row, token) in enumerate(zip(logits, a)):
            near = 0.02 * np.abs(row).max()
            text = p + a[:i]
            for t in set(text):
                row[t] = (row[t] / 1.2 if row[t] > 0 else row[t] * 1.2) - 0.6 * text.count(t)
            assert row[token] >= row.max() - near
    assert fast == plain and steps <= 1 + -(-19 // 7)


def test_right_drafts_are_accepted_and_their_vectors_move(loop, monkeypatch):
    model = loop.TreeDecoder(dtype=moe.F32, num_pages=60, page_size=5)
    prompts = [[3, 4], [9]]
    kw = dict(batch=2, max_pages=16, temperature=0.0)
    plain, _, slow = loop.generate(model, prompts, 20, max_new=1, **kw)
    monkeypatch.setattr(loop, "draft", _right_drafts(prompts, plain))
    walks, accept = [], moe.tree_accept
    monkeypatch.setattr(moe, "tree_accept", lambda *a, **k: walks.append(accept(*a, **k)) or walks[-1])
    fast, left, steps = loop.generate(model, prompts, 20, max_new=8, **kw)
    # seven tokens a step: the root, the wrong sibling, six of the answer, and the one drawn
    assert slow == 21 and steps <= 1 + -(-19 // 7) and left == model.num_pages
    moved = [int((w.path[r, :n] != torch.arange(n, device="cuda")).sum())
             for w in walks for r, n in enumerate(w.accepted.tolist())]
    assert max(moved) == 6
    for p, (a,) in zip(prompts, fast):
        assert len(a) == 20
        _follows(model, p, a)


@pytest.mark.parametrize("max_new", [1, 3, 8])
def test_answers_to_a_prompt_part_at_their_first_token(loop, max_new):
    model = loop.TreeDecoder(num_pages=80)
    answers, left, _ = loop.generate(model, PROMPTS, 5, samples=4, batch=8, max_new=max_new,
                                     temperature=5.0)
    assert left == model.num_pages
    for four in answers:
        assert all(len(a) == 5 for a in four)
        assert len({a[0] for a in four}) > 1             # of a thousand nearly as likely ones
    one, _, _ = loop.generate(model, PROMPTS, 1, samples=4, batch=4, max_new=max_new, temperature=5.0)
    assert all(len(a) == 1 for four in one for a in four)
