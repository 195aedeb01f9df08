"""The decode-step calls and autograd: tensors written in place say so, and
outputs are cut off from the inputs' graph."""
import pytest
import torch

import serving_moe_route_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _state():
    both = torch.zeros(2, 6, 4, 1, 64, device=DEV)
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    return both, both[0], both[1], table, torch.arange(6, dtype=torch.int32, device=DEV), _i32(6)


def test_what_is_written_has_a_new_version():
    both, kc, vc, table, free, n_free = _state()
    seen = {}

    def changed(*tensors):
        now = [t._version > seen.get(id(t), 0) for t in tensors]
        seen.update((id(t), t._version) for t in (both, table, free, n_free, out))
        return now

    out = torch.empty(2, 2, 64, device=DEV)
    changed()
    step = moe.kv_step(_i32(0, 0), _i32(1, 1), table, free, n_free, page_size=4, num_pages=6,
                       max_tokens=2, n_free_out=n_free)
    assert changed(both, table, free, n_free, out) == [False, True, False, True, False]
    again = moe.kv_step(_i32(0, 0), _i32(1, 1), table, free, n_free, page_size=4, num_pages=6,
                        max_tokens=2)
    assert again.n_free is not n_free
    assert changed(both, table, free, n_free, out) == [False, True, False, False, False]
    k = torch.randn(2, 1, 64, device=DEV)
    moe.kv_append(k, k, step.slots, kc, vc)      # views: their base has the version
    assert changed(both, table, free, n_free, out) == [True, False, False, False, False]
    q = torch.randn(2, 2, 64, device=DEV)
    moe.attn_decode(q, kc, vc, table, step.seq_lens)
    moe.sample_tokens(q[0], torch.rand(2, device=DEV))
    assert changed(both, table, free, n_free, out) == [False] * 5
    moe.attn_decode(q, kc, vc, table, step.seq_lens, out=out)
    assert changed(both, table, free, n_free, out) == [False] * 4 + [True]
    moe.kv_release(_i32(1, 0), table, free, n_free, num_pages=6)
    assert changed(both, table, free, n_free, out) == [False, True, True, True, False]


def test_backward_through_an_overwritten_cache_is_refused():
    both, kc, vc, table, free, n_free = _state()
    w = torch.ones(64, device=DEV, requires_grad=True)
    loss = (kc * w).sum()                          # saves the cache
    moe.kv_append(torch.ones(1, 1, 64, device=DEV), torch.ones(1, 1, 64, device=DEV), _i32(0), kc, vc)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_are_cut_off_and_inference_mode_works():
    both, kc, vc, table, free, n_free = _state()
    q = torch.randn(2, 2, 64, device=DEV, requires_grad=True)
    out = moe.attn_decode(q, kc, vc, table, _i32(0, 0))
    assert not out.requires_grad
    with torch.inference_mode():
        both, kc, vc, table, free, n_free = _state()
        step = moe.kv_step(_i32(0, 0), _i32(1, 1), table, free, n_free, page_size=4, num_pages=6,
                           max_tokens=2, n_free_out=n_free)
        k = torch.randn(2, 1, 64, device=DEV)
        moe.kv_append(k, k, step.slots, kc, vc)
        out = moe.attn_decode(k, kc, vc, table, step.seq_lens)
        torch.testing.assert_close(out, k)          # one token: its value
        moe.kv_release(_i32(1, 1), table, free, n_free, num_pages=6)
    assert int(n_free) == 6
