"""Trees of drafted tokens on the GPU against plain forms in 64 bits
(``tree_reference``): masks, attention, the walk along the drawn tokens.

Tolerances of attention count roundings as ``test_gpu_decode`` does.  With ds
the error of a logit, an attended weight is off by 2 ds, n 2^-24 for the sum
over n tokens, 2^-20 for the exponential, rescaling and the additions of the
second product, and w for its own rounding (2^-8 to bf16, 2^-11 to f16, none for
an f32 cache) of sum p |v|; the output's rounding (2^-8, 2^-24) comes on top.
ds is at most 2^-23 of sum |q k| for every one of the D products and additions;
the weights' sum takes the weights before they are rounded."""
import numpy as np
import pytest
import torch

import decode_reference as D64
import serving_moe_route_gb300 as moe
import tree_reference as R
from test_gpu_decode import _empty_cache, _i32, _pool, _word

pytestmark = pytest.mark.gpu
DEV = "cuda"
KV = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
WEIGHT = {"f32": 0.0, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}


def _tree(rng, n, kind="random"):
    if kind == "chain":
        return np.arange(n) - 1
    if kind == "star":
        return np.where(np.arange(n) > 0, 0, -1)
    return np.array([-1] + [rng.integers(0, j) for j in range(1, n)])[:n]


def _starts(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(int)


def _case(seed, ctx, sizes, Hq, Hkv, D, page, kv, major="token", pad=0, max_new=None, kind="random"):
    """A cache whose unused slots hold NaN, masks of random trees, q."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = [c + n for c, n in zip(ctx, sizes)]
    width = max(1, max(-(-n // page) for n in lens)) + 1
    table, _, pool = _pool(rng, lens, page, width, 2)
    kc, vc = _empty_cache(pool, page, Hkv, D, kv, major, fill=float("nan"))
    for b, n in enumerate(lens):
        pos = torch.arange(max(0, n), device=DEV)
        pg = torch.as_tensor(table[b], device=DEV)[pos // page].long()
        for c in (kc, vc):
            x = torch.randn(len(pos), Hkv, D, generator=g, device=DEV)
            c[pg, pos % page] = (x * 30 if kv == "e4m3" else x).to(KV[kv])
    N = sum(sizes) + pad
    q = torch.randn(N, Hq, D, generator=g, device=DEV).to(
        torch.float32 if kv == "f32" else torch.bfloat16)
    sc = {}
    if kv == "e4m3":
        sc = dict(k_scale=torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.02,
                  v_scale=torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.02)
    max_new = max_new or max(1, max(sizes))
    starts = _starts(sizes)
    parents = np.concatenate([_tree(rng, n, kind) for n in sizes] + [np.zeros(pad, int)]).astype(int)
    bits = R.masks(parents, starts, lens, max_new, N)[0]
    return dict(q=q, kc=kc, vc=vc, table=_i32(table), starts=_i32(starts), lens=_i32(lens), bits=bits,
                masks=torch.as_tensor(R.packed(bits), device=DEV), max_new=max_new, sc=sc, kv=kv)


def _attend(c, masks=True, **kw):
    return moe.attn_tree(c["q"], c["kc"], c["vc"], c["table"], c["starts"], c["lens"],
                         c["masks"] if masks else None, max_new=c["max_new"], return_lse=True,
                         **c["sc"], **kw)


def _bounds(c, masks=True, scale=None, window=0, kc=None, vc=None, q=None):
    """(out, lse, tolerances of both) in 64 bits"""
    q, kc, vc = (c[n] if t is None else t for n, t in (("q", q), ("kc", kc), ("vc", vc)))
    D = q.shape[2]
    s = {k: v.cpu().numpy() for k, v in c["sc"].items()}
    want, lse, pv, dot, n = R.attend(
        D64.f64(q), D64.f64(kc), D64.f64(vc), c["table"].cpu().numpy(), c["starts"].cpu().numpy(),
        c["lens"].cpu().numpy(), c["bits"] if masks else None, c["max_new"],
        D ** -0.5 if scale is None else scale, window, **s)
    ds = dot * D * 2.0 ** -23
    share = 2 * ds + n * 2.0 ** -24 + WEIGHT[c["kv"]] + 2.0 ** -20
    tol = (2.0 ** -24 if c["kv"] == "f32" else 2.0 ** -8) * np.abs(want) + share[..., None] * pv + 1e-37
    return want, lse, tol, ds + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)


def _check(c, got, lse, rows=None, **kw):
    want, want_lse, tol, lse_tol = _bounds(c, **kw)
    mine = ~np.isnan(want_lse[:, 0]) if rows is None else rows
    err = np.abs(D64.f64(got) - want)[mine]
    assert (err <= tol[mine]).all(), f"{np.nanmax(err / tol[mine]):.3g} of the tolerance"
    lse, want_lse, lse_tol = D64.f64(lse)[mine], want_lse[mine], lse_tol[mine]
    assert np.array_equal(np.isinf(lse), np.isinf(want_lse))
    f = np.isfinite(want_lse)
    assert (np.abs(lse[f] - want_lse[f]) <= lse_tol[f]).all()


# ------------------------------------------------------------------ masks and walks
@pytest.mark.parametrize("sizes,max_new,pad", [
    ([1], 1, 0), ([8], 8, 3), ([0, 5, 64, 1, 0, 33], 64, 7), ([65, 128, 3], 128, 0),
    ([256, 200, 0], 256, 1), ([7] * 300, 9, 0), ([70, 10], 64, 2)])
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
def test_masks(sizes, max_new, pad, kind):
    rng = np.random.default_rng(len(sizes))
    starts = _starts(sizes)
    N = sum(sizes) + pad
    parents = np.concatenate([_tree(rng, n, kind) for n in sizes] + [np.full(pad, 99)]).astype(int)
    lens = np.array(sizes) + rng.integers(0, 50, len(sizes))
    err = _word()
    got = moe.tree_masks(_i32(parents), _i32(starts), _i32(lens), max_new=max_new, err=err)
    bits, pos, flags = R.masks(parents, starts, lens, max_new, N)
    np.testing.assert_array_equal(got.masks.cpu().numpy(), R.packed(bits))
    np.testing.assert_array_equal(got.positions.cpu().numpy(), pos)
    assert moe.check_word(err)[1] == flags


def test_masks_of_bad_parents():
    parents = np.array([0, 0, 7, -2, 3, 1, -1, -1, 1])      # of trees of 6 and 3 nodes
    starts, lens = np.array([0, 6, 9]), np.array([6, 2])    # the second has fewer tokens than nodes
    err = _word()
    got = moe.tree_masks(_i32(parents), _i32(starts), _i32(lens), max_new=6, err=err)
    bits, pos, flags = R.masks(parents, starts, lens, 6, 9)
    np.testing.assert_array_equal(got.masks.cpu().numpy(), R.packed(bits))
    np.testing.assert_array_equal(got.positions.cpu().numpy(), pos)
    assert moe.check_word(err)[1] == flags == R.BAD_ID


def test_masks_of_starts_that_do_not_rise():
    # what rows get is not said, but nothing is written outside
    for starts in ([5, 2, 9], [-4, 100, 3], [0, 4, 2 ** 31 - 1], [4, 4, 4]):
        got = moe.tree_masks(_i32(np.zeros(6)), _i32(starts), _i32([3, 3]), max_new=4)
        assert got.masks.shape == (6, 1)
        moe.tree_accept(*(_i32(np.zeros(6)) for _ in range(3)), _i32(starts), _i32([1, 1]), max_path=4)
    torch.cuda.synchronize()


@pytest.mark.parametrize("sizes,max_path", [
    ([1], 1), ([8], 8), ([0, 5, 64, 1, 33], 20), ([256, 200, 0, 130], 256), ([30] * 200, 3)])
@pytest.mark.parametrize("words", [1, 3, 50])
def test_accept(sizes, max_path, words):
    # few words: long walks, and siblings of the same token
    rng = np.random.default_rng(words)
    starts, N = _starts(sizes), sum(sizes)
    parents = np.concatenate([_tree(rng, n, "chain" if i % 3 == 0 else "random")
                              for i, n in enumerate(sizes)]).astype(int)
    tokens, draws = rng.integers(0, words, N), rng.integers(-1 if words > 1 else 0, words, N)
    ctx = rng.integers(-2, 90, len(sizes))
    got = moe.tree_accept(_i32(tokens), _i32(draws), _i32(parents), _i32(starts), _i32(ctx),
                          max_path=max_path)
    want = R.accept(tokens, draws, parents, starts, ctx, max_path)
    for a, b, name in zip(got, want, got._fields):
        np.testing.assert_array_equal(a.cpu().numpy(), b, err_msg=name)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("ctx,sizes,Hq,Hkv,page,major", [
    ([0], [1], 1, 1, 16, "token"),
    ([2, 0, 17, 0, 15, 63, 127, 128, 129, 260], [3, 5, 0, 0, 16, 1, 2, 130, 64, 7], 4, 2, 5, "head"),
    ([700, 3, 1500], [9, 33, 12], 24, 3, 16, "fused"), ([40, 333], [2, 31], 40, 2, 1, "token"),
    ([5000], [61], 7, 1, 64, "token"), ([900, 20], [17, 250], 2, 2, 16, "head")])
def test_attend_shapes(kv, D, ctx, sizes, Hq, Hkv, page, major):
    c = _case(D + len(ctx), ctx, sizes, Hq, Hkv, D, page, kv, major)
    out, lse = _attend(c)
    _check(c, out, lse)
    again = _attend(c)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])  # parts join in one order


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_a_chain_needs_no_masks(kv):
    c = _case(2, [30, 0, 500], [5, 70, 128], 8, 2, 64, 16, kv, kind="chain")
    plain = _attend(c, masks=False)
    masked = _attend(c)
    assert torch.equal(plain[0], masked[0]) and torch.equal(plain[1], masked[1])
    _check(c, *plain, masks=False)


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_one_token_each_is_decode(kv):
    # bounds of both are those of the same definition
    c = _case(3, [0, 9, 100, 1200], [1, 1, 1, 1], 16, 4, 128, 16, kv)
    out, lse = _attend(c)
    one, one_lse = moe.attn_decode(c["q"], c["kc"], c["vc"], c["table"], c["lens"], return_lse=True)
    _, _, tol, lse_tol = _bounds(c)
    assert (np.abs(D64.f64(out) - D64.f64(one)) <= 2 * tol).all()
    assert (np.abs(D64.f64(lse) - D64.f64(one_lse)) <= 2 * lse_tol).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 5000])
@pytest.mark.parametrize("kind", ["random", "chain"])
def test_window_and_scale(kv, window, kind):
    c = _case(4, [0, 90, 0, 101, 600], [5, 1, 0, 20, 64], 8, 2, 128, 7, kv, kind=kind)
    for scale in (0.31, -0.2):
        out, lse = _attend(c, scale=scale, window=window)
        _check(c, out, lse, scale=scale, window=window)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_masks_of_any_bits(kv):
    # rows that attend nothing, only others, nodes behind them, bits past the tree
    c = _case(5, [0, 0, 40, 130], [4, 1, 100, 9], 6, 2, 64, 16, kv, max_new=128)
    rng = np.random.default_rng(1)
    c["bits"] = rng.random(c["bits"].shape) < 0.3
    c["bits"][:2] = False
    c["bits"][4] = False
    c["masks"] = torch.as_tensor(R.packed(c["bits"]), device=DEV)
    out, lse = _attend(c)
    _check(c, out, lse)
    assert (out[[0, 1, 4]] == 0).all() and (lse[[0, 1, 4]] == -float("inf")).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_requests(kv):
    # more units than CTAs, and more requests than threads of a CTA
    rng = np.random.default_rng(6)
    ctx, sizes = rng.integers(0, 60, 700).tolist(), rng.integers(0, 6, 700).tolist()
    c = _case(6, ctx, sizes, 2, 1, 64, 16, kv)
    _check(c, *_attend(c))


def test_no_requests_and_no_rows():
    c = _case(7, [10, 20], [2, 3], 2, 1, 64, 16, "bf16")
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    zero = _i32([0, 0, 0])
    out, lse = moe.attn_tree(none, c["kc"], c["vc"], c["table"], zero, c["lens"], max_new=4,
                             return_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out = torch.full_like(c["q"], 3.0)
    moe.attn_tree(c["q"], c["kc"], c["vc"], c["table"][:0], zero[:1], c["lens"][:0], max_new=4, out=out)
    moe.attn_tree(c["q"], c["kc"], c["vc"], c["table"], zero, c["lens"], max_new=4, out=out)
    assert (out == 3).all()                            # rows of no request are left alone


def test_strides_padding_rows_and_workspace():
    c = _case(8, [70, 10, 0, 33], [4, 0, 20, 1], 8, 2, 64, 16, "bf16", pad=5)
    N = len(c["q"])
    qkv = torch.randn(N, 12, 64, device=DEV).to(torch.bfloat16)
    qkv[:, :8] = c["q"]
    table = torch.full((4, c["table"].shape[1] + 5), -3, dtype=torch.int32, device=DEV)
    table[:, :-5] = c["table"]
    room = torch.full((N, 8, 128), 5.0, device=DEV).to(torch.bfloat16)
    ws = torch.empty(moe.attn_tree_workspace(torch.bfloat16, 64) + 100, dtype=torch.uint8, device=DEV)
    ws.fill_(255)                                       # needs no initialisation
    out, lse = moe.attn_tree(qkv[:, :8], c["kc"], c["vc"], table[:, :-5], c["starts"], c["lens"],
                             c["masks"], max_new=20, out=room[:, :, :64], workspace=ws,
                             return_lse=True)
    assert out.data_ptr() == room.data_ptr()
    _check(c, out, lse)
    assert (room[:, :, 64:] == 5).all() and (room[25:] == 5).all()
    with pytest.raises(moe.MoeError, match="orkspace"):
        _attend(c, workspace=ws[:256])


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_bad_pages_are_left_out(kv):
    c = _case(9, [200, 90, 31], [20, 7, 3], 4, 2, 128, 16, kv)
    t = c["table"]
    t[0, 3], t[1, 0], t[1, 5], t[0, 13] = -1, c["kc"].shape[0], 2 ** 31 - 1, -9
    t[2, :] = -2                                        # nothing left: empty rows
    err = _word()
    out, lse = _attend(c, err=err)
    assert moe.check_word(err) == (-5, R.BAD_PAGE)
    _check(c, out, lse)
    assert (out[27:] == 0).all() and torch.isinf(lse[27:]).all()


def test_lengths_and_rows_past_their_limits():
    c = _case(10, [30, 20], [6, 5], 2, 1, 64, 16, "bf16", kind="chain")
    c["table"] = c["table"][:, :2].contiguous()         # the first request's end is cut off
    err = _word()
    _check(c, *_attend(c, err=err))
    assert moe.check_word(err) == (-5, R.NO_SPACE)
    c = _case(11, [30, 20], [6, 5], 2, 1, 64, 16, "bf16", max_new=5)
    out = torch.full_like(c["q"], 9.0)
    got, lse = _attend(c, err=err, out=out)
    assert moe.check_word(err) == (-5, R.NO_SPACE)
    assert (out[5] == 9).all()                          # the sixth row is left out
    _check(c, got, lse)
    c["lens"][1] = 3                                    # fewer tokens than rows
    _check(c, *_attend(c))
    c["lens"][1] = -7
    _check(c, *_attend(c))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_large_logits_and_q_range(kv):
    c = _case(12, [300, 40, 9], [8, 3, 2], 4, 2, 64, 16, kv)
    q = c["q"]
    q[0] *= 200
    q[8, 1] = 0
    q[9, 2] *= 1e-30
    q[11, 0] *= 1e-38
    _check(c, *_attend(c))


def _poke(c, cache, r, pos, head, elem, value):
    page = cache.shape[1]
    cache[int(c["table"][r, pos // page]), pos % page, head, elem] = torch.tensor(
        value, device=DEV).to(cache.dtype)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_attended_has_no_part(kv, D, value):
    # a drafted token that its siblings do not attend, and context that has left
    # the window of some rows only, for a large tree and a small one
    if kv == "e4m3" and value == float("inf"):
        value = float("nan")
    for sizes, Hq in (([20, 6], 16), ([60, 3], 12), ([5, 2], 4)):
        c = _case(13, [50, 300], sizes, Hq, 2, D, 16, kv, kind="star")
        for window in (0, 40):
            clean = _attend(c, window=window)
            for r, pos in ((0, 50 + 2), (1, 300 + 1)) + (((0, 50 - 40 + 1),) if window else ()):
                lo = 0 if r == 0 else sizes[0]
                n, ctx = sizes[r], (50, 300)[r]
                reached = torch.zeros(len(c["q"]), Hq, dtype=torch.bool, device=DEV)
                for i in range(n):
                    own = 1 if i == 0 else 2            # a star: itself and node 0
                    at = (pos < ctx and pos >= ctx - max(0, window - own)) or pos - ctx in (0, i)
                    reached[lo + i, Hq // 2:] = at
                for which in ("kc", "vc"):
                    d = dict(c, **{which: c[which].clone()})
                    _poke(d, d[which], r, pos, 1, 5, value)
                    out, lse = _attend(d, window=window)
                    assert torch.equal(out[~reached], clean[0][~reached])
                    assert torch.equal(lse[~reached], clean[1][~reached])
                    if which == "vc":
                        assert not out[..., 5][reached].isfinite().any()
                        assert torch.equal(lse, clean[1])
                        out[..., 5][reached] = clean[0][..., 5][reached]
                        assert torch.equal(out, clean[0])
                    elif value != value:
                        assert out[reached].isnan().all() and lse[reached].isnan().all()


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 256])
def test_logits_that_are_all_minus_infinity(kv, D):
    c = _case(14, [0, 300, 6000], [4, 3, 2], 2, 1, D, 16, kv)
    c["q"][:, :, 2] = 0.5
    for r, n in ((0, 4), (1, 303), (2, 6002)):
        for pos in range(n):
            if r != 2 or pos > 9:
                _poke(c, c["kc"], r, pos, 0, 2, -float("inf"))
    out, lse = _attend(c)
    assert out[:7].isnan().all() and (lse[:7] == -float("inf")).all()
    assert out[7:].isfinite().all() and lse[7:].isfinite().all()
    short = dict(c, lens=_i32([4, 303, 12]), table=c["table"].clone())
    short["masks"] = c["masks"].clone()
    short["masks"][7:] = 0                               # ten context tokens, no drafted ones
    few, few_lse = _attend(short)
    torch.testing.assert_close(out[7:], few[7:], rtol=2.0 ** -6, atol=2.0 ** -9)
    torch.testing.assert_close(lse[7:], few_lse[7:], rtol=2.0 ** -20, atol=2.0 ** -19)


def test_far_offsets_and_a_long_split():
    # one long request over every CTA; its pages lie beyond 2^32 bytes
    D, page, ctx, n = 128, 64, 70001, 5
    pages = (5 << 30) // (page * D * 2)
    both = torch.empty(2, pages, page, 1, D, dtype=torch.bfloat16, device=DEV)
    used = -(-(ctx + n) // page)
    ids = torch.arange(pages - used, pages, device=DEV).flip(0)
    g = torch.Generator(device=DEV).manual_seed(1)
    for t in both:
        t[ids] = torch.randn(used, page, 1, D, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(n, 4, D, generator=g, device=DEV).to(torch.bfloat16)
    out, lse = moe.attn_tree(q, both[0], both[1], ids.int()[None], _i32([0, n]), _i32([ctx + n]),
                             max_new=n, return_lse=True)
    c = dict(q=q, kc=both[0][ids], vc=both[1][ids], table=_i32(np.arange(used)[None]),
             starts=_i32([0, n]), lens=_i32([ctx + n]), max_new=n, sc={}, kv="bf16")
    _check(c, out, lse, masks=False)


def test_two_streams_two_graphs_and_one_call_are_the_same():
    a = _case(15, [900, 5, 64], [20, 64, 3], 16, 2, 128, 16, "bf16")
    b = _case(16, [10, 2000], [33, 8], 16, 2, 128, 16, "bf16")
    want = _attend(a), _attend(b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s in zip((a, b), streams):
            got.append(_attend(c, stream=s))             # workspaces of their own
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = _attend(c)
        graphs.append((g, res))
    for _ in range(3):
        for i in (0, 1, 1, 0):
            for t in graphs[i][1]:
                t.fill_(-1)
            graphs[i][0].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(graphs[i][1], want[i]))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_of_an_8_bit_cache_that_are_odd(D):
    # negative ones turn logits and values round, 0 makes weights alike, NaN is NaN
    c = _case(17, [100, 3], [9, 2], 4, 2, D, 16, "e4m3")
    for k, v in ((-0.03, 0.02), (0.0, -0.5), (1e-42, 1.0)):
        c["sc"] = dict(k_scale=torch.tensor([0.02, k], device=DEV),
                       v_scale=torch.tensor([0.03, v], device=DEV))
        _check(c, *_attend(c))
    c["sc"]["k_scale"][1] = float("nan")
    out, lse = _attend(c)
    assert out[:, 2:].isnan().all() and out[:, :2].isfinite().all()
    c["sc"] = dict(k_scale=torch.tensor([0.02, 0.02], device=DEV),
                   v_scale=torch.tensor([0.03, float("nan")], device=DEV))
    out, lse = _attend(c)
    assert out[:, 2:].isnan().all() and out[:, :2].isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_a_scale_of_zero(kv):
    c = _case(18, [70, 0], [5, 3], 4, 2, 64, 16, kv)
    out, lse = _attend(c, scale=0.0)
    _check(c, out, lse, scale=0.0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("page", [1, 5, 8, 24, 48, 96, 256])
def test_pages_of_any_size(kv, D, page):
    c = _case(page, [200, 7, 130], [20, 3, 1], 6, 2, D, page, kv, "head" if page % 2 else "token")
    _check(c, *_attend(c))
    _check(c, *_attend(c, window=50), window=50)


def test_a_cache_that_overlaps_may_be_read():
    # all kv heads on one memory: no box fits, the copies do
    c = _case(19, [90], [6], 8, 1, 64, 16, "bf16")
    one = _attend(c)
    c["kc"], c["vc"] = (t.expand(-1, -1, 4, -1) for t in (c["kc"], c["vc"]))
    four = _attend(c)
    torch.testing.assert_close(four[0], one[0], rtol=2.0 ** -7, atol=2.0 ** -9)
    torch.testing.assert_close(four[1], one[1], rtol=2.0 ** -20, atol=2.0 ** -19)


def test_outputs_are_cut_off_and_out_has_a_new_version():
    c = _case(20, [9], [3], 2, 1, 64, 16, "f32")
    c["q"].requires_grad_(True)
    out, lse = _attend(c)
    assert not out.requires_grad and not lse.requires_grad
    to = torch.empty_like(out)
    before = to._version
    _attend(c, out=to)
    assert to._version > before and torch.equal(to, out)
    with torch.inference_mode():
        _attend(c, out=torch.empty(3, 2, 64, device=DEV))


def test_refusals_of_the_wrapper():
    c = _case(21, [9, 4], [3, 2], 4, 2, 64, 16, "bf16")

    def call(**kw):
        d = dict(c, **kw)
        return moe.attn_tree(d["q"], d["kc"], d["vc"], d["table"], d["starts"], d["lens"], d["masks"],
                             max_new=d["max_new"])

    for kw, what in ((dict(max_new=0), "max_new"), (dict(max_new=257), "max_new"),
                     (dict(masks=c["masks"].int()), "masks"), (dict(masks=c["masks"][:2]), "masks"),
                     (dict(max_new=65), "masks"), (dict(starts=c["starts"][:0]), "starts"),
                     (dict(lens=c["lens"][:1]), "seq_lens"), (dict(q=c["q"].float()), "q"),
                     (dict(q=c["q"][:, :3]), "multiple"), (dict(table=c["table"][:1]), "block_table")):
        with pytest.raises(ValueError, match=what):
            call(**kw)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("window", [1, 4, 40, 64, 100])
def test_a_chain_longer_than_the_window_is_decode_token_by_token(kv, window):
    c = _case(23, [3, 0, 200, 31], [6, 40, 170, 1], 4, 2, 64, 16, kv, kind="chain")
    starts, lens = c["starts"].tolist(), c["lens"].tolist()
    of = [r for r in range(4) for _ in range(starts[r + 1] - starts[r])]
    upto = [lens[r] - starts[r + 1] + i + 1 for i, r in enumerate(of)]
    one, one_lse = moe.attn_decode(c["q"], c["kc"], c["vc"], c["table"][of], _i32(upto), window=window,
                                   return_lse=True, **c["sc"])
    for masks in (False, True):
        out, lse = _attend(c, masks=masks, window=window)
        _, _, tol, lse_tol = _bounds(c, masks=masks, window=window)
        assert (np.abs(D64.f64(out) - D64.f64(one)) <= 2 * tol).all()
        assert (np.abs(D64.f64(lse) - D64.f64(one_lse)) <= 2 * lse_tol).all()
        _check(c, out, lse, masks=masks, window=window)


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 3, 65, 130])
def test_of_more_new_tokens_than_the_window_the_last_count(kv, window):
    # masks of any bits over four words; a table that cuts the last request's nodes off
    c = _case(24, [0, 90, 20], [250, 4, 200], 2, 1, 64, 16, kv, max_new=256)
    c["bits"] = np.random.default_rng(2).random(c["bits"].shape) < 0.6
    c["bits"][[3, 251]] = False
    c["masks"] = torch.as_tensor(R.packed(c["bits"]), device=DEV)
    _check(c, *_attend(c, window=window), window=window)
    c["table"] = c["table"][:, :9].contiguous()
    _check(c, *_attend(c, window=window), window=window)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("page", [1, 4, 8, 16, 64])
@pytest.mark.parametrize("window", [1, 30, 64, 200])
def test_pages_behind_the_window_may_be_gone(kv, page, window):
    # a server gives pages back once every token to come has left them behind
    c = _case(25, [500, 130, 700, 9], [5, 20, 1, 3], 4, 2, 64, page, kv)
    lens, starts = c["lens"].tolist(), c["starts"].tolist()
    first = [max(0, lens[r] - starts[r + 1] + starts[r] + 1 - window) for r in range(4)]
    whole = _attend(c, window=window)
    gone = c["table"].clone()
    for r in range(4):
        gone[r, :first[r] // page] = torch.tensor([-1, c["kc"].shape[0], -9], device=DEV).repeat(
            gone.shape[1])[:first[r] // page]
    err = _word()
    cut = _attend(dict(c, table=gone), window=window, err=err)
    assert moe.check_word(err) == (0, 0)
    assert torch.equal(cut[0], whole[0]) and torch.equal(cut[1], whole[1])
    one = _attend(dict(c, table=gone), masks=False, window=window, err=err)
    assert moe.check_word(err) == (0, 0) and one[0].isfinite().all()
    for r in range(4):                                   # the page of the first token is needed
        less = gone.clone()
        less[r, first[r] // page] = -1
        _attend(dict(c, table=less), window=window, err=err)
        assert moe.check_word(err) == (-5, R.BAD_PAGE)


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 8])
def test_what_lies_behind_the_window_goes_by_the_rows_masks(kv, page):
    # the row with the fewest new tokens reaches farthest back
    window, ctx = 16, 64
    for least in (0, 1, 3):
        c = _case(26, [ctx], [7], 2, 1, 64, page, kv)
        c["bits"][:] = False
        for i, n in enumerate([3, 4, 5, least, 6, 3, 4]):
            c["bits"][i, :n] = True
        c["masks"] = torch.as_tensor(R.packed(c["bits"]), device=DEV)
        first, err = ctx - window + least, _word()
        for at, bits in ((first // page, R.BAD_PAGE), (first // page - 1, 0)):
            gone = c["table"].clone()
            gone[0, :at + 1] = -1
            _attend(dict(c, table=gone), window=window, err=err)
            assert moe.check_word(err)[1] == bits


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_row_that_attends_nothing_under_a_nan_scale(D):
    c = _case(27, [0, 0, 40], [200, 3, 5], 4, 2, D, 16, "e4m3", max_new=256)
    rng = np.random.default_rng(3)
    c["bits"] = rng.random(c["bits"].shape) < 0.2
    none = [0, 7, 64, 130, 199, 201]
    c["bits"][none] = False
    c["masks"] = torch.as_tensor(R.packed(c["bits"]), device=DEV)
    starts = c["starts"].tolist()
    few = [i for r, ctx in enumerate((0, 0, 40)) for i in range(starts[r], starts[r + 1])
           if ctx == 0 and not c["bits"][i, :starts[r + 1] - starts[r]].any()]
    assert set(none) <= set(few)
    c["sc"]["k_scale"][1] = float("nan")
    out, lse = _attend(c)
    assert (out[few] == 0).all() and (lse[few] == -float("inf")).all()
    some = torch.ones(len(out), dtype=torch.bool, device=DEV)
    some[few] = False
    assert out[some][:, 2:].isnan().all() and out[:, :2].isfinite().all()


def test_lengths_at_the_ends_of_32_bits():
    starts, lens = _i32([0, 3, 5, 8]), _i32([-2 ** 31, 1, 2 ** 31 - 1])
    parents, tokens = _i32([-1, 0, 1, -1, 0, -1, 0, 1]), _i32([1] * 8)
    got = moe.tree_masks(parents, starts, lens, max_new=3)
    assert got.positions.tolist() == [0, 1, 2, 0, 1, 2 ** 31 - 4, 2 ** 31 - 3, 2 ** 31 - 2]
    walk = moe.tree_accept(tokens, tokens, parents, starts, lens, max_path=3)
    assert walk.accepted.tolist() == [3, 2, 3]
    assert walk.seq_lens.tolist() == [3, 3, 2 ** 31 - 1]
