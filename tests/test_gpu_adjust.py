"""Adjusted logits on the GPU against the definition in 64 bits
(``tree_reference``).  Up to four roundings to f32 (the division or product, the
two subtractions, the addition; the product of frequency and count is contracted
or rounded: a fifth) of at most the sum of the magnitudes, and the output's:
5 x 2^-24 of that sum, and 2^-8 of a bf16 output."""
import numpy as np
import pytest
import torch

import decode_reference as D64
import serving_moe_route_gb300 as moe
import tree_reference as R
from test_gpu_decode import _i32, _word

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _f32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.float32, device=DEV)


def _settings(seed, N, V, R_=None, L=50, n_bias=0, penalties=True, grammar=False, prompt=True):
    rng = np.random.default_rng(seed)
    s = {}
    if R_:
        s["rows"] = rng.integers(0, R_, N)
    R_ = R_ or N
    if penalties:
        s["history"] = (V * rng.random((R_, L)) ** 3).astype(int)
        s["history"][rng.random((R_, L)) < 0.1] = -1
        s["history"][rng.random((R_, L)) < 0.05] = V     # neither is a token
        s["history_lens"] = rng.integers(0, L + 1, R_)
        if prompt:
            s["prompt_lens"] = rng.integers(-1, L, R_)
        for name, lo in (("repetition", 1.0), ("presence", -0.3), ("frequency", 0.0)):
            s[name] = (lo + rng.random(R_)).astype(np.float32)
    if n_bias:
        s["bias_ids"] = rng.integers(-1, V + 1, (R_, n_bias))
        s["bias"] = (10 * rng.standard_normal((R_, n_bias))).astype(np.float32)
    if grammar:
        s["allowed"] = rng.integers(-2 ** 31, 2 ** 31, (N, -(-V // 32)))
    return s


def _gpu(s):
    return {k: _f32(v) if k in ("repetition", "presence", "frequency", "bias") else _i32(v)
            for k, v in s.items()}


def _check(x, s, got, out_dtype):
    want, size = R.adjust(D64.f64(x), **s)
    got = D64.f64(got)
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want))
    f = np.isfinite(want)
    tol = 5 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(want) if out_dtype == torch.bfloat16 else 0)
    assert (np.abs(got[f] - want[f]) <= tol[f] * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,kw", [
    (1, 1, {}), (3, 7, dict(n_bias=3, grammar=True)), (2, 255, dict(L=1)), (5, 1000, dict(n_bias=40)),
    (4, 50257, dict(L=3000, n_bias=300, grammar=True)), (6, 4099, dict(R_=2, grammar=True)),
    (3, 33000, dict(penalties=False, grammar=True)), (3, 8193, dict(penalties=False, n_bias=9)),
    (2, 262144, dict(L=500, n_bias=5, grammar=True)), (4, 131, dict(penalties=False)),
    (9, 32000, dict(L=9000, prompt=False))])
def test_adjust(dtype, N, V, kw):
    x = torch.randn(N, V, device=DEV).mul_(3).to(DT[dtype])
    s = _settings(V, N, V, **kw)
    before = x.clone()
    err = _word()
    out = moe.adjust_logits(x, err=err, **_gpu(s))
    assert torch.equal(x, before) and moe.check_word(err) == (0, 0)
    _check(x, s, out, out.dtype)
    same = moe.adjust_logits(x, out=x, **_gpu(s))        # in place
    assert same is x and torch.equal(x, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off_in,off_out", [(0, 0), (1, 0), (0, 3), (3, 3), (5, 2)])
def test_rows_of_any_alignment(dtype, off_in, off_out):
    N, V = 5, 2011
    s = _settings(1, N, V, n_bias=20, grammar=True)
    room = torch.randn(N, V + 13, device=DEV).to(DT[dtype])
    to = torch.full((N, V + 30), 7.0, device=DEV).to(DT[dtype])
    x, out = room[:, off_in:off_in + V], to[:, off_out:off_out + V]
    allowed = torch.zeros(N, 70, dtype=torch.int32, device=DEV)
    allowed[:, :63] = _i32(s["allowed"])
    g = dict(_gpu(s), allowed=allowed)
    moe.adjust_logits(x, out=out, **g)
    _check(x, s, out, out.dtype)
    assert (to[:, :off_out] == 7).all() and (to[:, off_out + V:] == 7).all()


def test_each_part_alone_and_none():
    N, V = 4, 3001
    x = torch.randn(N, V, device=DEV)
    s = _settings(2, N, V, n_bias=7, grammar=True)
    past = ("history", "history_lens")
    for names in (past, (*past, "prompt_lens", "repetition"), (*past, "presence"),
                  (*past, "frequency", "prompt_lens"), ("bias_ids", "bias"), ("allowed",),
                  (*past, "repetition", "bias_ids", "bias"), ()):
        part = {k: s[k] for k in names}
        _check(x, part, moe.adjust_logits(x, **_gpu(part)), torch.float32)


def test_values_that_are_not_numbers():
    V = 100
    x = torch.zeros(2, V, device=DEV)
    x[:, 0], x[:, 1], x[:, 2] = float("nan"), float("inf"), -float("inf")
    words = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    words[1, 0] = ~7                                     # tokens 0, 1, 2 are not allowed
    out = moe.adjust_logits(x, history=_i32([[0, 1, 2, 3]] * 2), history_lens=_i32([4, 4]),
                            repetition=_f32([1.5, 1.5]), presence=_f32([1.0, 1.0]), allowed=words)
    assert out[0, 0].isnan() and out[0, 1] == float("inf") and out[0, 2] == -float("inf")
    assert (out[:, 3] == -1).all() and (out[1, :3] == -float("inf")).all()


def test_the_last_of_equal_biases_counts():
    V, n = 40, 1000
    ids = np.full((1, n), -1)
    ids[0, ::3] = 7
    ids[0, 1::3] = 6                                     # the other half of 7's word
    bias = np.arange(n, dtype=np.float32)[None]
    out = moe.adjust_logits(torch.zeros(1, V, device=DEV), bias_ids=_i32(ids), bias=_f32(bias))
    assert out[0, 7] == 999 and out[0, 6] == 997 and out[0, 5] == 0 and out[0, 8] == 0


def test_rows_of_no_request():
    N, V = 4, 500
    x = torch.randn(N, V, device=DEV)
    s = _settings(3, N, V, R_=2, n_bias=3, grammar=True)
    s["rows"] = np.array([1, -1, 2, 0])                  # the second and third are of none
    err = _word()
    out = moe.adjust_logits(x, err=err, **_gpu(s))
    assert moe.check_word(err) == (-5, R.BAD_ID)
    _check(x, s, out, torch.float32)


def test_counts_far_past_16_bits():
    V, L = 9, 200000
    h = torch.full((1, L), 4, dtype=torch.int32, device=DEV)
    h[0, 100] = 5
    out = moe.adjust_logits(torch.zeros(1, V, device=DEV), history=h, history_lens=_i32([10 ** 9]),
                            prompt_lens=_i32([50]), frequency=_f32([0.5]))
    assert out[0, 4] == -0.5 * (L - 51) and out[0, 5] == -0.5 and not out[0, :4].any()


def test_a_captured_call_and_another_stream():
    N, V = 6, 5000
    x = torch.randn(N, V, device=DEV).to(torch.bfloat16)
    s = _gpu(_settings(4, N, V, n_bias=5, grammar=True))
    want = moe.adjust_logits(x, **s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = moe.adjust_logits(x, stream=side, **s)
    side.synchronize()
    assert torch.equal(other, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = moe.adjust_logits(x, **s)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)


def _trees(rng, sizes, pad, V, words):
    """Random trees' tokens (of a few words, so that paths repeat them), what their nodes
    attend, and where requests begin."""
    starts = np.concatenate([[0], np.cumsum(sizes)]).astype(int)
    parents = np.concatenate([[-1] + [rng.integers(max(0, j - 3), j) for j in range(1, n)]
                              for n in sizes if n] + [np.zeros(pad, int)]).astype(int)
    N = sum(sizes) + pad
    bits = R.masks(parents, starts, sizes, 64 * words, N)[0]
    return dict(tokens=rng.integers(0, min(V, 40), N), bits=bits, starts=starts)


def _tree_args(t):
    return dict(tokens=_i32(t["tokens"]), starts=_i32(t["starts"]),
                masks=torch.as_tensor(R.packed(t["bits"]), device=DEV))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,pad,V,L,words,n_bias", [
    ([1], 0, 5, 3, 1, 0), ([7, 0, 4], 2, 1000, 30, 1, 5), ([64, 3, 20], 0, 50257, 2000, 1, 0),
    ([256, 1], 3, 9001, 100, 4, 9), ([100, 130], 0, 300, 10, 2, 0)])
def test_tokens_on_a_nodes_path_are_text(dtype, sizes, pad, V, L, words, n_bias):
    rng = np.random.default_rng(V)
    t = _trees(rng, sizes, pad, V, words)
    N = sum(sizes) + pad
    s = _settings(V, N, V, R_=len(sizes), L=L, n_bias=n_bias, grammar=True)
    s["rows"] = np.array([r for r, n in enumerate(sizes) for _ in range(n)] + [0] * pad)
    t["tokens"][rng.random(N) < 0.05] = -1               # not a token
    s["tokens"] = t["tokens"]
    x = torch.randn(N, V, device=DEV).mul_(3).to(DT[dtype])
    g = _gpu({k: v for k, v in s.items() if k != "tokens"})
    err = _word()
    out = moe.adjust_logits(x, err=err, **g, **_tree_args(t))
    assert moe.check_word(err) == (0, 0)
    _check(x, dict(s, bits=t["bits"], starts=t["starts"]), out, out.dtype)
    # the same bits as with a history a row that ends with the path
    longer = np.full((N, L + 64 * words), -1)
    lens, of = np.zeros(N, int), s["rows"]
    for i in range(N):
        n, lo = int(s["history_lens"][of[i]]), t["starts"][of[i]]
        path = [t["tokens"][lo + j] for j in range(1, 64 * words) if i < sum(sizes) and t["bits"][i, j]]
        longer[i, :n] = s["history"][of[i], :n]
        longer[i, n:n + len(path)] = path
        lens[i] = n + len(path)
    each = {k: v[of] for k, v in s.items() if k in ("prompt_lens", "repetition", "presence", "frequency",
                                                   "bias_ids", "bias")}
    # (a path is never the prompt's)
    each["prompt_lens"] = np.minimum(each["prompt_lens"], s["history_lens"][of])
    want = moe.adjust_logits(x, **_gpu(dict(each, history=longer, history_lens=lens,
                                            allowed=s["allowed"])))
    assert torch.equal(out, want)


def test_drafted_tokens_without_a_text_before_them():
    x = torch.zeros(3, 9, device=DEV)
    bits = np.zeros((3, 64), bool)
    bits[0, 0], bits[1, :2], bits[2, [0, 1, 2]] = True, True, True
    t = dict(tokens=np.array([4, 5, 5]), bits=bits, starts=np.array([0, 3]))
    kw = dict(rows=_i32([0, 0, 0]), history_lens=_i32([0]), frequency=_f32([2.0]), presence=_f32([0.5]))
    for history in (torch.zeros(1, 0, dtype=torch.int32, device=DEV), _i32([[7]])):
        out = moe.adjust_logits(x, history=history, **kw, **_tree_args(t))
        want = torch.zeros(3, 9)
        want[1, 5], want[2, 5] = -2.5, -4.5
        assert torch.equal(out.cpu(), want)


def test_starts_that_do_not_rise_add_nothing_outside():
    # what rows get is not said, but nothing outside the arrays is looked at
    x = torch.zeros(6, 50, device=DEV)
    t = dict(tokens=np.zeros(6, int), bits=np.ones((6, 256), bool), starts=np.zeros(3, int))
    for starts in ([5, 2, 9], [-4, 100, 3], [0, 4, 2 ** 31 - 1], [4, 4, 4], [3, -2 ** 31, 2 ** 31 - 1]):
        t["starts"] = np.array(starts)
        out = moe.adjust_logits(x, rows=_i32([0, 0, 1, 1, 0, 1]), history=_i32([[1], [1]]),
                                history_lens=_i32([1, 1]), frequency=_f32([1.0, 1.0]), **_tree_args(t))
        assert (out[:, 1] == -1).all() and (out[:, 2:] == 0).all()


def test_refusals_of_drafted_tokens():
    x = torch.zeros(3, 9, device=DEV)
    t = _tree_args(dict(tokens=np.zeros(3, int), bits=np.ones((3, 64), bool), starts=np.array([0, 3])))
    past = dict(rows=_i32([0, 0, 0]), history=_i32([[1]]), history_lens=_i32([1]))
    for kw, what in ((dict(t, tokens=None), "together"), (dict(t, masks=None), "together"),
                     (dict(t, starts=None), "together"), (dict(t, starts=_i32([0, 1, 3])), "starts"),
                     (dict(t, tokens=_i32([0, 0])), "tokens"), (dict(t, masks=t["masks"][:2]), "masks"),
                     (dict(t, masks=t["masks"].int()), "masks"),
                     (dict(t, masks=t["masks"].repeat(1, 5)), "masks")):
        with pytest.raises(ValueError, match=what):
            moe.adjust_logits(x, **past, **kw)
    with pytest.raises(ValueError, match="history"):
        moe.adjust_logits(x, rows=past["rows"], **t)
