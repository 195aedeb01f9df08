"""Block tables, cache append and paged decode attention on the GPU against
plain forms in 64 bits (``decode_reference``).

Tolerances count roundings, eps/2 = 2^-8 (bf16), 2^-11 (f16), 2^-24 (fp32)
relative to the rounded value.  An attended weight is off by
  2 ds      the logits' error ds on it and on the sum: every one of the D
            products and additions of a logit at most 2^-23 of sum |q k|
            (tensor cores cut their sums); fp32 operands are pairs of 11-bit
            halves, 3 x 2^-22 a product more
  n 2^-24   the sum over n tokens
  w         the weight's own rounding for the second product: pairs of bf16
            2^-16, f16 2^-11, pairs of tf32 2^-22
  2^-20     exponential, rescaling and the additions of the second product
of sum p |v|, and the output's rounding comes on top."""
import math

import numpy as np
import pytest
import torch

import decode_reference as R
import serving_moe_route_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
KV = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ tables
def _run_step(ctx, new, table, free, n_free, page, pool, tokens, in_place=False, stride=None):
    err = _word()
    if stride:
        wide = torch.full((table.shape[0], stride), -7, dtype=torch.int32, device=DEV)
        t = wide[:, :table.shape[1]]
        t.copy_(_i32(table))
    else:
        t = _i32(table)
    n = _i32([n_free])
    got = moe.kv_step(_i32(ctx), _i32(new), t, _i32(free), n, page_size=page, num_pages=pool,
                      max_tokens=tokens, n_free_out=n if in_place else None, err=err)
    _, bits = moe.check_word(err)
    want = R.kv_step(ctx, new, table, free, n_free, page, pool, tokens)
    for name, a, b in zip(("slots", "positions", "starts", "seq_lens"), got[:4], want[:4]):
        np.testing.assert_array_equal(a.cpu().numpy(), b, err_msg=name)
    assert int(got.n_free) == want[4]
    if in_place:
        assert int(n) == want[4]
    else:
        assert int(n) == n_free
    np.testing.assert_array_equal(t.cpu().numpy(), want[5])
    assert bits == want[6]
    if stride:
        assert (wide[:, table.shape[1]:] == -7).all()


def _pool(rng, ctx, page, width, spare):
    have = [min(width, -(-max(0, c) // page)) for c in ctx]
    pool = sum(have) + spare
    ids = rng.permutation(pool)
    table = np.full((len(ctx), width), -1)
    at = 0
    for r, h in enumerate(have):
        table[r, :h] = ids[at:at + h]
        at += h
    return table, ids[at:], pool


@pytest.mark.parametrize("B,page,longest,chunk,tokens", [
    (1, 16, 40, 1, 1), (1, 1, 5, 3, 8), (7, 5, 60, 9, 70), (64, 16, 500, 1, 64),
    (64, 16, 500, 1, 80), (300, 16, 200, 40, 9000), (1025, 8, 60, 3, 2500),
    (2500, 128, 900, 2, 4000), (33, 7, 100, 700, 20000)])
def test_step_sizes(B, page, longest, chunk, tokens):
    rng = np.random.default_rng(B + page)
    ctx = rng.integers(0, longest, B)
    new = rng.integers(0, chunk + 1, B) if chunk > 1 else np.ones(B, int)
    while new.sum() > tokens:
        new[rng.integers(B)] = 0
    width = -(-(longest + chunk) // page) + 1
    spare = int(sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))) + 3
    table, free, pool = _pool(rng, ctx, page, width, spare)
    _run_step(ctx, new, table, free, len(free), page, pool, tokens, in_place=B % 2 == 1,
              stride=width + 3 if B % 3 == 0 else None)


def test_step_shortage_negative_lengths_and_bad_ids():
    rng = np.random.default_rng(0)
    ctx, new = np.array([3, 8, 0, -4, 31, 6]), np.array([2, 1, 9, 2, 5, -3])
    table, free, pool = _pool(rng, ctx, 4, 9, 2)       # 2 pages for 2 + 1 + 3 + 1 + 1
    _run_step(ctx, new, table, free, len(free), 4, pool, 16)       # no pages left
    _run_step(ctx, new, table, free, len(free), 4, pool, 10)       # too few rows as well
    table, free, pool = _pool(rng, ctx, 4, 8, 20)
    _run_step(ctx, new, table, free, len(free), 4, pool, 40)       # row 4 outgrows the table
    free = free.copy()
    free[-1], free[-3] = pool, -9                                  # ids outside the cache
    table[0, 0] = pool + 1
    _run_step(ctx, new, table, free, len(free), 4, pool, 40)
    _run_step(ctx, new, table, free, len(free) + 50, 4, pool, 40)  # n_free past the list
    _run_step(ctx, new, table, free, -5, 4, pool, 40)


def test_step_no_requests_and_no_rows():
    empty = np.zeros(0, int)
    _run_step(empty, empty, np.zeros((0, 4), int), np.arange(3), 3, 16, 10, 5)
    _run_step([5], [1], np.array([[0, 1]]), np.arange(2, 4), 2, 4, 4, 0)


@pytest.mark.parametrize("B,width", [(1, 1), (5, 33), (64, 100), (1500, 7)])
def test_release(B, width):
    rng = np.random.default_rng(B)
    table, free, pool = _pool(rng, rng.integers(0, width + 1, B), 1, width, 11)
    done = rng.integers(0, 2, B)
    done[0] = 3
    for cap in (pool, len(free) + 2):  # the second is too short for what comes back
        lst = np.zeros(cap, int)
        lst[:len(free)] = free
        want = R.kv_release(done, table, lst, len(free), pool)
        t, f, n, err = _i32(table), _i32(lst), _i32([len(free)]), _word()
        moe.kv_release(_i32(done), t, f, n, num_pages=pool, err=err)
        _, bits = moe.check_word(err)
        np.testing.assert_array_equal(t.cpu().numpy(), want[0])
        np.testing.assert_array_equal(f.cpu().numpy(), want[1])
        assert int(n) == want[2] and bits == want[3]


# ------------------------------------------------------------------ append
def _empty_cache(pages, page, Hkv, D, kv, major, fill=0.0):
    shape = (pages, Hkv, page, D) if major == "head" else (pages, page, Hkv, D)
    out = [torch.full(shape, fill, device=DEV).to(KV[kv]) for _ in range(2)]
    if major == "fused":  # keys and values side by side in one tensor
        both = torch.full((pages, page, 2, Hkv, D), fill, device=DEV).to(KV[kv])
        return both[:, :, 0], both[:, :, 1]
    return [t.transpose(1, 2) for t in out] if major == "head" else out


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("N,Hkv,D,page,major,src", [
    (1, 1, 64, 16, "token", "plain"), (5, 3, 80, 5, "head", "side"), (300, 4, 128, 16, "fused", "side"),
    (33, 2, 256, 1, "token", "odd"), (17, 1, 16, 7, "head", "odd"), (2000, 8, 128, 32, "head", "plain")])
def test_append(kv, N, Hkv, D, page, major, src):
    g = torch.Generator(device=DEV).manual_seed(N)
    pages = -(-N // page) + 3
    kc, vc = _empty_cache(pages, page, Hkv, D, kv, major, fill=2.0)
    dt = torch.float32 if kv == "f32" else torch.bfloat16
    off = 1 if src == "odd" else 0  # one element past alignment
    x = (torch.randn(N, 2 * Hkv * D + off, generator=g, device=DEV) * 3).to(dt)
    x[0, off] = float("nan")
    x[0, off + 1] = float("inf")
    x[0, off + 2] = -1e6
    if src == "plain":
        k, v = x[:, :Hkv * D].reshape(N, Hkv, D), x[:, Hkv * D:].reshape(N, Hkv, D)
    else:
        k = x[:, off:off + Hkv * D].view(N, Hkv, D)
        v = x[:, off + Hkv * D:].view(N, Hkv, D)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:N].int()
    if N > 4:
        slots[1], slots[3], slots[4] = -1, pages * page, -5  # skipped; the last two are errors
    scales = {}
    if kv == "e4m3":
        scales = dict(k_scale=torch.rand(Hkv, device=DEV) * 0.01 + 0.01,
                      v_scale=torch.rand(Hkv, device=DEV) * 0.1 + 0.1)
    want = []
    for c, t, s in ((kc, k, scales.get("k_scale")), (vc, v, scales.get("v_scale"))):
        w = c.float().cpu().clone()
        y = t.float().cpu()
        if s is not None:
            y = (y / s.cpu()[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        for i, sl in enumerate(slots.tolist()):
            if 0 <= sl < pages * page:
                w[sl // page, sl % page] = y[i]
        want.append(w)
    err = _word()
    moe.kv_append(k, v, slots, kc, vc, err=err, **scales)
    _, bits = moe.check_word(err)
    for c, w in zip((kc, vc), want):
        assert torch.equal(torch.nan_to_num(c.float().cpu(), nan=7e5), torch.nan_to_num(w, nan=7e5))
    assert bits == (R.BAD_PAGE if N > 4 else 0)


def test_append_nothing():
    kc, vc = _empty_cache(2, 4, 1, 64, "bf16", "token")
    k = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    moe.kv_append(k, k, _i32([]), kc, vc)


# ------------------------------------------------------------------ attention
def _check(q, kc, vc, table, lens, got, lse, *, scale=None, window=0, k_scale=None, v_scale=None):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    s = {} if k_scale is None else dict(k_scale=k_scale.cpu().numpy(), v_scale=v_scale.cpu().numpy())
    want, want_lse, pv, dot, n = R.attend(R.f64(q), R.f64(kc), R.f64(vc), table.cpu().numpy(),
                                          lens.cpu().numpy(), scale, window, **s)
    f32 = kc.dtype == torch.float32
    ds = dot * (D * 2.0 ** -23 + (3 * 2.0 ** -22 if f32 else 0.0))
    w = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -16}.get(kc.dtype, 2.0 ** -11)
    share = 2 * ds + n * 2.0 ** -24 + w + 2.0 ** -20
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(want) + share[..., None] * pv + 1e-37
    err = np.abs(R.f64(got) - want)
    assert (err <= tol).all(), f"{(err / tol).max():.3g} of the tolerance"
    if lse is not None:
        lse = R.f64(lse)
        assert np.array_equal(np.isinf(lse), np.isinf(want_lse))
        f = np.isfinite(want_lse)
        tol = ds + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse)
        assert (np.abs(lse[f] - want_lse[f]) <= tol[f]).all()


def _case(seed, B, Hq, Hkv, D, page, kv, lens, major="token", spare=2):
    """A cache whose unused slots hold NaN, and a table with junk past each request's pages."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-n // page) for n in lens)) + 1
    table, _, pool = _pool(rng, lens, page, width, spare)
    kc, vc = _empty_cache(pool, page, Hkv, D, kv, major, fill=float("nan"))
    for b, n in enumerate(lens):
        pos = torch.arange(max(0, n), device=DEV)
        pg = torch.as_tensor(table[b], device=DEV)[pos // page].long()
        for c in (kc, vc):
            x = torch.randn(len(pos), Hkv, D, generator=g, device=DEV)
            c[pg, pos % page] = (x * 30 if kv == "e4m3" else x).to(KV[kv])
    q = torch.randn(B, Hq, D, generator=g, device=DEV).to(
        torch.float32 if kv == "f32" else torch.bfloat16)
    sc = {}
    if kv == "e4m3":
        sc = dict(k_scale=torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.02,
                  v_scale=torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.02)
    return q, kc, vc, _i32(table), _i32(lens), sc


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("lens,Hq,Hkv,page,major", [
    ([1], 1, 1, 16, "token"), ([2, 0, 17, 16, 15, 63, 64, 65, 129], 4, 2, 5, "head"),
    ([700, 3, 1500], 24, 3, 16, "fused"), ([40, 333], 40, 2, 1, "token"),
    ([5000], 7, 1, 64, "token")])
def test_attend_shapes(kv, D, lens, Hq, Hkv, page, major):
    q, kc, vc, table, n, sc = _case(D + len(lens), len(lens), Hq, Hkv, D, page, kv, lens, major)
    out, lse = moe.attn_decode(q, kc, vc, table, n, return_lse=True, **sc)
    _check(q, kc, vc, table, n, out, lse, **sc)
    again = moe.attn_decode(q, kc, vc, table, n, **sc)
    assert torch.equal(out, again)  # the parts join in one order


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
def test_attend_window_and_scale(kv, window):
    lens = [1, 90, 0, 101, 100, 99, 2222]
    q, kc, vc, table, n, sc = _case(3, len(lens), 8, 2, 128, 7, kv, lens)
    out, lse = moe.attn_decode(q, kc, vc, table, n, scale=0.31, window=window, return_lse=True, **sc)
    _check(q, kc, vc, table, n, out, lse, scale=0.31, window=window, **sc)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_many_requests(kv):
    # more units than CTAs, and more requests than threads of a CTA
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 60, 700).tolist()
    q, kc, vc, table, n, sc = _case(4, 700, 2, 1, 64, 16, kv, lens)
    out, lse = moe.attn_decode(q, kc, vc, table, n, return_lse=True, **sc)
    _check(q, kc, vc, table, n, out, lse, **sc)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_attend_large_logits_and_q_range(kv):
    # weights of one token only; rows of q of very different size, one zero,
    # one whose values are near the type's smallest
    lens = [300, 40, 9]
    q, kc, vc, table, n, sc = _case(6, 3, 4, 2, 64, 16, kv, lens)
    q[0] *= 200
    q[1, 1] = 0
    q[1, 2] *= 1e-30
    q[2, 0] *= 1e-38
    out, lse = moe.attn_decode(q, kc, vc, table, n, return_lse=True, **sc)
    _check(q, kc, vc, table, n, out, lse, **sc)


def test_attend_strided_q_out_and_table():
    lens = [70, 10, 0, 33]
    q, kc, vc, table, n, _ = _case(7, 4, 8, 2, 64, 16, "bf16", lens)
    qkv = torch.randn(4, 12, 64, device=DEV).to(torch.bfloat16)
    qkv[:, :8] = q
    wide = torch.full((4, table.shape[1] + 5), -3, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    room = torch.full((4, 8, 128), 5.0, device=DEV).to(torch.bfloat16)
    out = moe.attn_decode(qkv[:, :8], kc, vc, wide[:, :table.shape[1]], n, out=room[:, :, :64])
    assert out.data_ptr() == room.data_ptr()
    _check(q, kc, vc, table, n, out, None)
    assert (room[:, :, 64:] == 5).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_attend_bad_pages_are_left_out(kv):
    lens = [200, 90, 31]
    q, kc, vc, table, n, sc = _case(8, 3, 4, 2, 128, 16, kv, lens)
    table[0, 3], table[1, 0], table[1, 5] = -1, kc.shape[0], 2 ** 31 - 1
    table[2, :] = -2  # nothing left: an empty row
    err = _word()
    out, lse = moe.attn_decode(q, kc, vc, table, n, return_lse=True, err=err, **sc)
    assert moe.check_word(err) == (-5, R.BAD_PAGE)
    _check(q, kc, vc, table, n, out, lse, **sc)
    assert (out[2] == 0).all() and torch.isinf(lse[2]).all()


def test_attend_length_past_the_table_is_cut():
    q, kc, vc, table, n, _ = _case(9, 2, 2, 1, 64, 16, "bf16", [32, 20])
    table = table[:, :2].contiguous()
    n[0] = 1000
    err = _word()
    out, lse = moe.attn_decode(q, kc, vc, table, n, return_lse=True, err=err)
    assert moe.check_word(err) == (-5, R.NO_SPACE)
    _check(q, kc, vc, table, n, out, lse)


def test_attend_long_split_and_far_offsets():
    # one long request over every CTA; its pages lie beyond 2^32 bytes
    D, page, n = 128, 64, 70001
    pages = (5 << 30) // (page * D * 2)
    both = torch.empty(2, pages, page, 1, D, dtype=torch.bfloat16, device=DEV)
    kc, vc = both[0], both[1]
    g = torch.Generator(device=DEV).manual_seed(1)
    used = -(-n // page)
    ids = torch.arange(pages - used, pages, device=DEV).flip(0)
    for c in (kc, vc):
        c[ids] = torch.randn(used, page, 1, D, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(1, 8, D, generator=g, device=DEV).to(torch.bfloat16)
    lens = _i32([n])
    out, lse = moe.attn_decode(q, kc, vc, ids.int()[None], lens, return_lse=True)
    first = pages - used
    _check(q, kc[first:], vc[first:], (ids - first).int()[None], lens, out, lse)


def test_attend_side_stream_and_graph():
    q, kc, vc, table, n, _ = _case(10, 3, 8, 2, 128, 16, "bf16", [500, 20, 130])
    want = moe.attn_decode(q, kc, vc, table, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.empty(moe.attn_workspace(kc.dtype, 128), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    side.wait_stream(torch.cuda.current_stream())
    moe.attn_decode(q, kc, vc, table, n, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.attn_decode(q, kc, vc, table, n, out=out, workspace=ws)
    n2 = torch.tensor([77, 500, 0], dtype=torch.int32, device=DEV)
    n2 = torch.minimum(n2, n)  # other lengths, read at replay
    n.copy_(n2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    _check(q, kc, vc, table, n, out, None)
    assert math.isfinite(float(out.float().sum()))


def test_wrappers_refuse_what_does_not_fit():
    q, kc, vc, table, n, _ = _case(11, 2, 4, 2, 64, 16, "bf16", [20, 3])
    e4 = kc.float().to(torch.float8_e4m3fn)
    sc = torch.ones(2, device=DEV)
    for why, args, kw in [
            ("one type", (q, kc, e4, table, n), {}),
            ("must be torch.bfloat16", (q.float(), kc, vc, table, n), {}),
            ("shape", (q[:, :, :32], kc, vc, table, n), {}),
            ("multiple of kv_heads", (q[:, :3], kc, vc, table, n), {}),
            ("block_table", (q, kc, vc, table.long(), n), {}),
            ("block_table", (q, kc, vc, table[:1], n), {}),
            ("seq_lens", (q, kc, vc, table, n.long()), {}),
            ("needs k_scale", (q, e4, e4, table, n), {}),
            ("only used by", (q, kc, vc, table, n), dict(k_scale=sc, v_scale=sc)),
            ("k_scale", (q, e4, e4, table, n), dict(k_scale=sc[:1], v_scale=sc)),
            ("float32, bfloat16 or", (q.half(), kc.half(), vc.half(), table, n), {}),
            ("contiguous", (q.transpose(1, 2).contiguous().transpose(1, 2), kc, vc, table, n), {}),
            ("out must", (q, kc, vc, table, n), dict(out=torch.empty(2, 4, 64, device=DEV)))]:
        with pytest.raises(ValueError, match=why):
            moe.attn_decode(*args, **kw)
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.attn_decode(q, kc, vc, table, n,
                        workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    for why, args in [("shape", (k[:1], k, n, kc, vc)), ("must be", (k.float(), k, n, kc, vc)),
                      ("slots", (k, k, n.long(), kc, vc)),
                      ("same strides", (k, k, n, kc, vc.transpose(0, 1)))]:
        with pytest.raises(ValueError, match=why):
            moe.kv_append(*args)
    with pytest.raises(ValueError, match="max_tokens"):
        moe.kv_step(n, n, table, n, n[:1], page_size=16, num_pages=4, max_tokens=-1)
    with pytest.raises(ValueError, match="overlap"):
        moe.kv_step(n, n, table[:1].expand(2, -1), n, n[:1], page_size=16, num_pages=4, max_tokens=1)


def test_a_whole_step_in_a_graph():
    # tables, append, attention and sampling of one step, captured once and
    # replayed while lengths and tables grow on the device
    B, Hq, Hkv, D, page, V = 5, 8, 2, 64, 4, 300
    g = torch.Generator(device=DEV).manual_seed(0)
    pool, width = 40, 6
    kc, vc = _empty_cache(pool, page, Hkv, D, "bf16", "token")
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    free, n_free = torch.arange(pool, dtype=torch.int32, device=DEV), _i32([pool])
    ctx, new, err = _i32([0] * B), _i32([1, 1, 0, 1, 1]), _word()
    qkv = torch.empty(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    logits = torch.empty(B, V, device=DEV)
    u = torch.empty(B, device=DEV)

    def step():
        s = moe.kv_step(ctx, new, table, free, n_free, page_size=page, num_pages=pool,
                        max_tokens=B, n_free_out=n_free, err=err)
        moe.kv_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], s.slots, kc, vc, err=err)
        out = moe.attn_decode(qkv[:, :Hq], kc, vc, table, s.seq_lens, err=err)
        ids, _ = moe.sample_tokens(logits, u)
        ctx.copy_(s.seq_lens)
        return out, ids

    def inputs(i):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=DEV))
        logits.copy_(torch.randn(B, V, generator=g, device=DEV) * 3)
        u.copy_(torch.rand(B, generator=g, device=DEV))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the first calls load what a capture may not
        inputs(0)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, ids = step()
    # the capture ran nothing: one step is behind, ten more follow
    for i in range(10):
        inputs(i + 1)
        q = qkv[:, :Hq].clone()
        graph.replay()
        torch.cuda.synchronize()
        assert ctx.tolist() == [i + 2, i + 2, 0, i + 2, i + 2]
        _check(q, kc, vc, table, ctx, out, None)
        want, _ = moe.sample_tokens(logits, u)
        assert torch.equal(ids, want)
    assert moe.check_word(err) == (0, 0)
    used = table[table >= 0].tolist()
    assert len(set(used)) == len(used) == pool - int(n_free) == 4 * 3


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,Hq,Hkv", [
    ([60000, 300, 0, 9000], 32, 2),   # parts by the hundred, a few and none, in one call
    ([30011], 20, 1),                 # two units of 16 and of 4 rows on one cached head
    ([900] * 40, 5, 1)])              # a cut about every unit
def test_attend_joins_few_and_many_parts(kv, D, lens, Hq, Hkv):
    q, kc, vc, table, lens, sc = _case(5, len(lens), Hq, Hkv, D, 16, kv, lens)
    out, lse = moe.attn_decode(q, kc, vc, table, lens, return_lse=True, **sc)
    _check(q, kc, vc, table, lens, out, lse, **sc)
    again = moe.attn_decode(q, kc, vc, table, lens, **sc)
    assert torch.equal(out, again)
