"""Every step of the example's decode loop: attention against the keys and
values that were appended, kept densely, and the drawn tokens against the
definition of sampling, for a cache of each type the loop's bf16 model has."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import decode_reference as R
import serving_moe_route_gb300 as moe
from test_gpu_decode import _check

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def loop():
    spec = importlib.util.spec_from_file_location(
        "decode_loop_steps", os.path.join(ROOT, "examples", "decode_loop.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn])
def test_every_step_is_what_its_definitions_say(loop, kv, monkeypatch):
    history, attended, drawn = {}, [], []
    append, attend, sample = moe.kv_append, moe.attn_decode, moe.sample_tokens

    def kv_append(k, v, slots, k_cache, v_cache, **kw):
        append(k, v, slots, k_cache, v_cache, **kw)
        rows = history.setdefault(k_cache.data_ptr(), [[] for _ in range(len(k))])
        for b, s in enumerate(slots.tolist()):
            if s >= 0:
                rows[b].append((k[b].clone(), v[b].clone()))

    def attn_decode(q, k_cache, v_cache, block_table, seq_lens, **kw):
        out = attend(q, k_cache, v_cache, block_table, seq_lens, **kw)
        rows, lens = history[k_cache.data_ptr()], seq_lens.tolist()
        dense = torch.zeros(2, len(lens), max(1, *lens), *k_cache.shape[2:],
                            device="cuda")
        for b, n in enumerate(lens):  # a row's last tokens are its present request's
            for t, kv_ in enumerate(rows[b][len(rows[b]) - n:]):
                dense[:, b, t] = torch.stack(kv_).float()
        if "k_scale" in kw:
            dense[0] /= kw["k_scale"][:, None]
            dense[1] /= kw["v_scale"][:, None]
        k, v = dense.clamp(-448, 448).to(k_cache.dtype)
        scales = {x: kw[x] for x in ("k_scale", "v_scale") if x in kw}
        attended.append((q, k, v, seq_lens, out, scales))
        return out

    def sample_tokens(logits, u, **kw):
        ids, probs = sample(logits, u, **kw)
        drawn.append((logits, u, kw, ids))
        return ids, probs

    monkeypatch.setattr(moe, "kv_append", kv_append)
    monkeypatch.setattr(moe, "attn_decode", attn_decode)
    monkeypatch.setattr(moe, "sample_tokens", sample_tokens)
    model = loop.Decoder(kv_dtype=kv, num_pages=40)
    prompts = [[3] * n for n in (1, 30, 5, 17, 2)]
    answers, _ = loop.generate(model, prompts, 8, batch=3, temperature=0.7, top_k=5, top_p=0.9)
    assert len(history) == 2 and len(attended) == 2 * len(drawn)
    assert sum(len(rows[b]) for rows in history.values() for b in range(3)) == \
        2 * sum(len(p) + 7 for p in prompts)
    for q, k, v, lens, out, scales in attended:
        table = torch.arange(len(lens), dtype=torch.int32, device="cuda")[:, None]
        _check(q, k, v, table, lens, out, None, **scales)
    given, checked = [], 0
    for logits, u, kw, ids in drawn:
        x, got = R.f64(logits), ids.cpu().numpy()
        host = {n: t.cpu().numpy() for n, t in kw.items()}
        want, _, near, off = R.sample(x, u.cpu().numpy(), **host)
        far = near > off
        checked += int(far.sum())
        np.testing.assert_array_equal(got[far], want[far])
        rank = (x > np.take_along_axis(x, got[:, None], 1)).sum(1)
        assert (rank < 5).all()
        given.extend(got.tolist())
    assert checked > 0.9 * len(given)
    assert all(t in given for a in answers for t in a)


def test_settings_may_be_whole_numbers(loop):
    model = loop.Decoder(num_pages=12)
    a, _ = loop.generate(model, [[1, 2], [4]], 3, batch=2, temperature=0, top_p=1, min_p=0, top_k=5)
    b, _ = loop.generate(model, [[1, 2], [4]], 3, batch=2, temperature=0.0)
    assert a == b and [len(x) for x in a] == [3, 3]
