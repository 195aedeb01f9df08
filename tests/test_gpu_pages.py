"""Pages that are forked, copied, moved together and given back, on the GPU
against plain loops (``tree_reference``): whole numbers and bytes, all equal."""
import numpy as np
import pytest
import torch

import serving_moe_route_gb300 as moe
import tree_reference as R
from test_gpu_decode import _empty_cache, _i32, _pool, _word

pytestmark = pytest.mark.gpu
DEV = "cuda"
KV = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _fork(src, dst, ctx, table, refs, free, n_free, page, pool):
    c, t, r, n, err = _i32(ctx), _i32(table), _i32(refs), _i32([n_free]), _word()
    got = moe.kv_fork(_i32(src), _i32(dst), c, t, r, _i32(free), n, page_size=page, num_pages=pool,
                      err=err)
    want = R.fork(src, dst, ctx, table, refs, free, n_free, page, pool)
    for j, name in enumerate(got._fields):
        np.testing.assert_array_equal(got[j].cpu().numpy(), want[0][:, j], err_msg=name)
    for name, a, b in (("ctx", c, want[1]), ("table", t, want[2]), ("refs", r, want[3])):
        np.testing.assert_array_equal(a.cpu().numpy(), b, err_msg=name)
    assert int(n) == want[4] and moe.check_word(err)[1] == want[5]
    return want


def _trim(keep, lens, table, free, n_free, page, pool, refs=None):
    t, f, n, err = _i32(table), _i32(free), _i32([n_free]), _word()
    r = None if refs is None else _i32(refs)
    moe.kv_trim(_i32(keep), _i32(lens), t, f, n, page_size=page, num_pages=pool, page_refs=r, err=err)
    want = R.trim(keep, lens, table, free, n_free, page, pool, refs)
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    np.testing.assert_array_equal(f.cpu().numpy(), want[1])
    assert int(n) == want[2] and moe.check_word(err)[1] == want[4]
    if refs is not None:
        np.testing.assert_array_equal(r.cpu().numpy(), want[3])
    return want


@pytest.mark.parametrize("parents,children,longest,page", [
    (1, 1, 1, 1), (1, 4, 900, 16), (5, 3, 60, 5), (40, 8, 700, 16), (300, 5, 200, 7), (3, 2000, 90, 8)])
def test_fork_and_give_back(parents, children, longest, page):
    rng = np.random.default_rng(parents)
    B, F = parents + parents * children, parents * children
    ctx = np.zeros(B, int)
    ctx[:parents] = rng.integers(0, longest + 1, parents)
    table, free, pool = _pool(rng, ctx, page, -(-longest // page) + 1, F + 3)
    src, dst = np.arange(F) % parents, parents + rng.permutation(F)
    pairs, ctx, table, refs, n_free, bits = _fork(src, dst, ctx, table, np.zeros(pool, int), free,
                                                  len(free), page, pool)
    assert bits == 0
    lst = np.full(pool, -1)
    lst[:len(free)] = free
    # some rows give all back, some a few pages, the parents among them
    keep = np.where(rng.random(B) < 0.5, 0, ctx - rng.integers(0, 3 * page, B))
    table, lst, n_free, refs, bits = _trim(keep, ctx, table, lst, n_free, page, pool, refs)
    assert bits == 0
    left = np.maximum(0, np.minimum(keep, ctx))
    table, lst, n_free, refs, bits = _trim(np.zeros(B, int), left, table, lst, n_free, page, pool, refs)
    assert bits == 0 and n_free == pool and (refs == 0).all()
    assert sorted(lst) == list(range(pool)) and (table == -1).all()


def test_fork_refusals():
    rng = np.random.default_rng(1)
    ctx = np.array([20, 7, 8, 0, 0, 0, 0, 0, 33])
    table, free, pool = _pool(rng, ctx, 4, 9, 2)
    refs = np.zeros(pool, int)
    args = (ctx, table, refs, free, len(free), 4, pool)
    _fork([0, 0, 2], [3, 3, 4], *args)                   # the second is refused: a row twice
    _fork([0, 1, 1], [1, 3, 4], *args)                   # a source that is written, and its forks
    _fork([0, 2], [0, 2], *args)                         # onto itself
    _fork([-1, 9, 0, 2, 2], [3, 4, -5, 9, 5], *args)     # outside the table
    _fork([1, 8, 1, 2], [3, 4, 5, 6], *args)             # three partial pages, two free
    _fork([1, 2], [3, 4], ctx, table, refs, free, -3, 4, pool)
    _fork([1, 2], [3, 4], ctx, table, refs, free, 100, 4, pool)
    long = ctx.copy()
    long[1], long[2] = 37, 36                            # one more than the row, just the row
    _fork([1, 2, 0], [3, 4, 5], long, table, refs, free, len(free), 4, pool)
    bad = table.copy()
    bad[0, 2], bad[1, 1] = pool, -7                      # a shared page, a partial one
    _fork([0, 1, 8], [3, 4, 5], ctx, bad, refs, free, len(free), 4, pool)
    worse = free.copy()
    worse[-1] = pool + 5
    _fork([1, 8], [3, 4], ctx, table, refs, worse, len(worse), 4, pool)
    _fork([], [], *args)


def test_bad_source_page_takes_no_free_page():
    ctx, table = np.array([6, 6, 0, 0]), np.full((4, 3), -1)
    table[0, :2], table[1, :2] = (0, 9), (1, 2)          # pages of 4, a pool of 9
    pairs, *_, n_free, bits = _fork([0, 1], [2, 3], ctx, table, np.zeros(9, int), np.array([7, 8]), 2,
                                    4, 9)
    assert bits == R.BAD_PAGE and n_free == 1
    np.testing.assert_array_equal(pairs, [(-1, -1, 0), (2, 8, 2)])


def test_row_cut_inside_a_shared_page_goes_on_as_a_fork():
    ctx, table = np.array([10, 0, 0]), np.full((3, 3), -1)
    table[0] = 0, 1, 2                                   # pages of 4, a pool of 6
    lst = np.array([3, 4, 5, -1, -1, -1])
    _, ctx, table, refs, n_free, _ = _fork([0], [1], ctx, table, np.zeros(6, int), lst, 3, 4, 6)
    keep = np.array([10, 6, 0])                          # page 1 is shared: row 1 may not go on in it
    table, lst, n_free, refs, _ = _trim(keep, ctx, table, lst, n_free, 4, 6, refs)
    pairs, ctx, table, refs, n_free, bits = _fork([1], [2], keep, table, refs, lst, n_free, 4, 6)
    assert bits == 0 and pairs[0][0] == 1 and pairs[0][2] == 2
    table, lst, n_free, refs, _ = _trim(np.array([10, 0, 6]), ctx, table, lst, n_free, 4, 6, refs)
    np.testing.assert_array_equal(refs, [1, 0, 0, 0, 0, 0])
    np.testing.assert_array_equal(table, [[0, 1, 2], [-1, -1, -1], [0, pairs[0][1], -1]])


@pytest.mark.parametrize("shared", [False, True])
def test_trim_shortage_and_bad_entries(shared):
    rng = np.random.default_rng(2)
    lens = np.array([20, 0, -4, 33, 9])
    table, free, pool = _pool(rng, lens, 4, 9, 3)
    refs = np.zeros(pool, int) if shared else None
    for cap in (pool, len(free) + 2):                    # the second is too short
        lst = np.zeros(cap, int)
        lst[:len(free)] = free
        _trim([8, 3, 2, -5, 50], lens, table, lst, len(free), 4, pool, refs)
        bad = table.copy()
        bad[0, 3], bad[3, 0], bad[3, 8], bad[4, 1] = pool, -2, -1, 2 ** 31 - 1
        _trim([1, 0, 0, 0, 0], lens, bad, lst, len(free), 4, pool, refs)
        _trim([0] * 5, [1000] * 5, table, lst, len(free), 4, pool, refs)  # rows that end early
        _trim([0] * 5, lens, table, lst, cap + 7, 4, pool, refs)
        _trim([0] * 5, lens, table, lst, -7, 4, pool, refs)
    _trim([], [], table[:0], np.zeros(3, int), 1, 4, pool)


def test_trim_a_page_in_every_row():
    # one page held by thousands of rows, and by one that keeps it
    B, pool = 3000, 10
    table = np.tile([4, -1, 7], (B, 1))
    table[:, 1] = np.arange(B) % 4
    refs = np.zeros(pool, int)
    for pg, n in zip(*np.unique(table, return_counts=True)):
        refs[pg] = n - 1
    keep = np.zeros(B, int)
    keep[B // 2] = 1
    got = _trim(keep, np.full(B, 3), table, np.full(pool, -1), 0, 1, pool, refs)
    assert got[3][4] == 0 and sorted(got[1][:got[2]]) == [0, 1, 2, 3, 7]


def test_trim_reads_rows_of_a_wider_table():
    rng = np.random.default_rng(3)
    lens = np.array([20, 17])
    table, free, pool = _pool(rng, lens, 4, 6, 3)
    wide = torch.full((2, 11), -7, dtype=torch.int32, device=DEV)
    wide[:, :6] = _i32(table)
    f, n = _i32(np.concatenate([free, np.zeros(20, int)])), _i32([len(free)])
    moe.kv_trim(_i32([5, 0]), _i32(lens), wide[:, :6], f, n, page_size=4, num_pages=pool)
    want = R.trim([5, 0], lens, table, f.cpu().numpy(), len(free), 4, pool)
    np.testing.assert_array_equal(wide[:, :6].cpu().numpy(), want[0])
    assert (wide[:, 6:] == -7).all() and int(n) == want[2]


def _filled(pages, page, Hkv, D, kv, major):
    """Caches whose every byte is random, NaNs of all kinds among them, and bytes of both"""
    caches = _empty_cache(pages, page, Hkv, D, kv, major)
    for c in caches:
        bits = torch.randint(256, (pages, page, Hkv, D * c.element_size()), device=DEV)
        c.copy_(bits.to(torch.uint8).view(c.dtype))
    return caches


def _bytes(c):
    return c.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,D,page,major", [
    (1, 64, 16, "token"), (3, 80, 5, "head"), (4, 128, 16, "fused"), (2, 256, 1, "token"),
    (1, 16, 7, "head"), (8, 128, 128, "head")])
def test_copy_pages(kv, Hkv, D, page, major):
    pages = 24
    rng = np.random.default_rng(D)
    src, dst = rng.integers(0, 12, 10), 12 + rng.permutation(12)[:10]
    src[3], dst[4], src[5], dst[6] = -1, -1, pages, -2
    dst[7] = src[7]
    if page > 1:
        src[8] = dst[8] = 3
    tokens = rng.integers(-1, page + 2, 10)
    for given in (tokens, None):
        caches = _filled(pages, page, Hkv, D, kv, major)
        want = [_bytes(c) for c in caches]
        for w in want:
            for i in range(10):
                if 0 <= src[i] < pages and 0 <= dst[i] < pages:
                    n = page if given is None else min(max(0, given[i]), page)
                    w[dst[i], :n] = w[src[i], :n]
        err = _word()
        moe.kv_copy_pages(_i32(src), _i32(dst), *caches, err=err,
                          tokens=None if given is None else _i32(given))
        assert moe.check_word(err)[1] == R.BAD_PAGE
        for c, w in zip(caches, want):
            np.testing.assert_array_equal(_bytes(c), w)


def test_copy_many_small_pages():
    caches = _filled(140000, 1, 1, 16, "bf16", "token")
    want = [_bytes(c) for c in caches]
    src = np.arange(70000)
    moe.kv_copy_pages(_i32(src), _i32(src + 70000), *caches)
    for c, w in zip(caches, want):
        w[70000:] = w[:70000]
        np.testing.assert_array_equal(_bytes(c), w)


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("nodes,Hkv,D,page,major", [
    (1, 1, 64, 16, "token"), (8, 3, 80, 5, "head"), (64, 4, 128, 16, "fused"), (256, 2, 256, 1, "token"),
    (200, 1, 16, 7, "head")])
def test_compact(kv, nodes, Hkv, D, page, major):
    rng = np.random.default_rng(nodes)
    B = 9
    ctx = rng.integers(-1, 40, B)
    table, _, pool = _pool(rng, ctx + nodes + 1, page, -(-(41 + nodes) // page), 2)
    accepted = rng.integers(0, nodes + 2, B)
    accepted[0] = nodes
    path = np.full((B, nodes), -1)
    for r in range(B):
        n = min(nodes, accepted[r])
        path[r, :n] = np.sort(rng.permutation(nodes)[:n])
    if nodes > 6:
        accepted[1:5] = 5
        path[1, :5] = [0, 2, 1, 5, 6]                    # does not rise
        path[2, :5] = [0, 1, 1, 5, 6]
        path[3, :5] = [-3, 1, 2, 3, 4]
        path[4, :5] = [0, 2, 3, 5, 2 ** 31 - 1]          # past the table
        table[5, (max(0, ctx[5]) + 1) // page] = pool + 3
    caches = _filled(pool, page, Hkv, D, kv, major)
    want = [R.compact(path, accepted, ctx, table, _bytes(c), page) for c in caches]
    err = _word()
    moe.kv_compact(_i32(path), _i32(accepted), _i32(ctx), _i32(table), *caches, err=err)
    assert moe.check_word(err)[1] == want[0][1]
    for c, (w, _) in zip(caches, want):
        np.testing.assert_array_equal(_bytes(c), w)


def test_nothing_to_move():
    caches = _filled(4, 4, 1, 64, "bf16", "token")
    before = [_bytes(c) for c in caches]
    none = _i32([])
    moe.kv_copy_pages(none, none, *caches)
    moe.kv_compact(none.view(0, 3), none, none, none.view(0, 2), *caches)
    moe.kv_compact(_i32([[0, 1, 2]]), _i32([3]), _i32([5]), _i32([[0, 1]]), *caches)  # all in place
    moe.kv_compact(_i32([[1, 2, 3]]), _i32([0]), _i32([1]), _i32([[0, 1]]), *caches)  # none accepted
    for c, w in zip(caches, before):
        np.testing.assert_array_equal(_bytes(c), w)


def test_versions_and_a_captured_step():
    # what is written in place says so; the calls can be captured and replayed
    kc, vc = _filled(12, 4, 1, 64, "bf16", "token")
    table = _i32([[0, 1, -1], [-1, -1, -1]])
    ctx, refs, free, n_free = _i32([6, 0]), _i32([0] * 12), _i32([2, 3] + [0] * 10), _i32([2])
    state = (kc, vc, table, ctx, refs, free, n_free)

    def changed(before):
        return [t._version > v for t, v in zip(state, before)]

    def versions():
        return [t._version for t in state]

    now = versions()
    f = moe.kv_fork(_i32([0]), _i32([1]), ctx, table, refs, free, n_free, page_size=4, num_pages=12)
    assert changed(now) == [False, False, True, True, True, False, True]
    now = versions()
    moe.kv_copy_pages(*f[:2], kc, vc, tokens=f.tokens)
    assert changed(now) == [True, True] + [False] * 5
    now = versions()
    moe.kv_compact(_i32([[0, 2], [0, 1]]), _i32([2, 0]), ctx, table, kc, vc)
    assert changed(now) == [True, True] + [False] * 5
    now = versions()
    moe.kv_trim(_i32([6, 0]), ctx, table, free, n_free, page_size=4, num_pages=12, page_refs=refs)
    assert changed(now) == [False, False, True, False, True, True, True]
    assert table.tolist() == [[0, 1, -1], [-1, -1, -1]] and int(n_free) == 2 and not refs.any()
    src, dst, keep = _i32([0]), _i32([1]), _i32([6, 0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f = moe.kv_fork(src, dst, ctx, table, refs, free, n_free, page_size=4, num_pages=12)
        moe.kv_copy_pages(*f[:2], kc, vc, tokens=f.tokens)
        moe.kv_trim(keep, ctx, table, free, n_free, page_size=4, num_pages=12, page_refs=refs)
    for _ in range(3):
        g.replay()
    assert f.src_pages.tolist() == [1] and f.dst_pages.tolist() == [3] and f.tokens.tolist() == [2]
    assert int(n_free) == 2 and not refs.any() and free[:2].tolist() == [2, 3]
    assert torch.equal(kc[3, :2].view(torch.int16), kc[1, :2].view(torch.int16))


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,width,page", [(1, 1025, 1), (64, 40, 16), (600, 220, 3), (8192, 9, 2)])
def test_trim_of_large_tables(B, width, page, shared):
    # more entries than one CTA takes, and (600 x 220) than its threads hold
    rng = np.random.default_rng(B)
    lens = rng.integers(0, width * page + 1, B)
    lens[0] = width * page
    table, free, pool = _pool(rng, lens, page, width, 3)
    lst = np.full(pool, -1)
    lst[:len(free)] = free
    refs = np.zeros(pool, int) if shared else None
    keep = np.where(rng.random(B) < 0.3, 0, (lens * rng.random(B)).astype(int))
    table, lst, n_free, refs, bits = _trim(keep, lens, table, lst, len(free), page, pool, refs)
    assert bits == 0 and n_free > len(free)
    table, lst, n_free, refs, bits = _trim(np.zeros(B, int), keep, table, lst, n_free, page, pool, refs)
    assert bits == 0 and sorted(lst) == list(range(pool)) and n_free == pool and (table == -1).all()
