"""Refusals of the calls on drafted tokens, shared pages and adjusted logits, all
of them made on the host before anything is launched (no GPU here), and of their
Python wrappers for CPU tensors."""
import ctypes

import numpy as np
import pytest
import torch

import decode_reference as D64
import serving_moe_route_gb300 as moe
import tree_reference as R
from serving_moe_route_gb300 import _binding as B
from test_decode_host import BAD, BAD_CACHES, FAKE, OK, UNSUPPORTED, cache

FAR = FAKE + (1 << 30)


@pytest.fixture(scope="module", autouse=True)
def library():
    from serving_moe_route_gb300 import _build

    _build.build()


def masks(**kw):
    a = dict(parents=FAKE, N=9, starts=FAKE, lens=FAKE, B=2, max_new=8, masks=FAKE, pos=FAKE)
    a.update(kw)
    return B.moe_tree_masks(*a.values(), 0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(B=-1), BAD), (dict(max_new=0), BAD), (dict(max_new=257), BAD),
    (dict(B=0), BAD), (dict(parents=0), BAD), (dict(starts=0), BAD), (dict(lens=0), BAD),
    (dict(masks=0), BAD), (dict(pos=0), BAD), (dict(B=0, N=0, starts=0), OK)])
def test_masks(kw, code):
    assert masks(**kw) == code


def accept(**kw):
    a = dict(tokens=FAKE, draws=FAKE, parents=FAKE, N=9, starts=FAKE, ctx=FAKE, B=2, max_path=8,
             path=FAKE, accepted=FAKE, next=FAKE, lens=FAKE)
    a.update(kw)
    return B.moe_tree_accept(*a.values(), 0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(B=-1), BAD), (dict(max_path=0), BAD), (dict(max_path=257), BAD),
    *((dict([(k, 0)]), BAD) for k in ("tokens", "draws", "parents", "starts", "ctx", "path",
                                      "accepted", "next", "lens")), (dict(B=0, N=0), OK)])
def test_accept(kw, code):
    assert accept(**kw) == code


def attend(c, **kw):
    a = dict(q=FAKE, qn=1024, qh=128, N=5, Hq=8, table=FAKE, max_pages=4, stride=4, starts=FAKE,
             lens=FAKE, B=2, masks=0, max_new=8, scale=1.0, window=0, out=FAKE, on=1024, oh=128, lse=0,
             ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return B.moe_attn_tree(c, *a.values(), 0, 0)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_descriptor(kw, code):
    assert attend(cache(**kw)) == code
    if "k_scale" not in kw and kw != dict(kv_dtype=B.MOE_KV_E4M3):  # scales do not matter to these
        assert compact(cache(**{"v": FAR, **kw})) == code
        assert copy(cache(**{"v": FAR, **kw})) == code


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(B=-1), BAD), (dict(Hq=0), BAD), (dict(Hq=7), BAD),
    (dict(N=1 << 28, Hq=8), BAD), (dict(max_pages=0), BAD), (dict(stride=3), BAD),
    (dict(window=-1), BAD), (dict(qn=-8), BAD), (dict(oh=-8), BAD), (dict(max_new=0), BAD),
    (dict(max_new=257), BAD), (dict(scale=float("nan")), BAD), (dict(q=0), BAD), (dict(table=0), BAD),
    (dict(starts=0), BAD), (dict(lens=0), BAD), (dict(out=0), BAD), (dict(ws=0), BAD),
    (dict(max_pages=1 << 28, stride=1 << 28), BAD), (dict(ws=FAKE + 16), BAD),
    (dict(on=0), BAD), (dict(oh=120), BAD), (dict(q=FAKE + 8), UNSUPPORTED),
    (dict(out=FAKE + 2), UNSUPPORTED), (dict(qh=129), UNSUPPORTED), (dict(on=1028), UNSUPPORTED),
    (dict(N=0, q=0, out=0, ws=0), OK), (dict(B=0, table=0, starts=0), OK)])
def test_attend(kw, code):
    assert attend(cache(), **kw) == code


def test_workspace():
    assert B.moe_attn_tree_workspace(7, 128) == 0
    assert B.moe_attn_tree_workspace(B.MOE_KV_BF16, 300) == 0
    with pytest.raises(ValueError, match="no cache"):
        moe.attn_tree_workspace(torch.float16, 128)


def compact(c, **kw):
    a = dict(path=FAKE, max_path=8, accepted=FAKE, ctx=FAKE, B=2, table=FAKE, max_pages=4, stride=4)
    a.update(kw)
    return B.moe_kv_compact(c, *a.values(), 0, 0)


def copy(c, **kw):
    a = dict(src=FAKE, dst=FAKE, tokens=0, n=3)
    a.update(kw)
    return B.moe_kv_copy_pages(c, *a.values(), 0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(max_path=0), BAD), (dict(B=-1), BAD), (dict(B=8193), BAD), (dict(max_pages=0), BAD),
    (dict(stride=3), BAD), (dict(path=0), BAD), (dict(accepted=0), BAD), (dict(ctx=0), BAD),
    (dict(table=0), BAD), (dict(B=0, path=0), OK)])
def test_compact(kw, code):
    assert compact(cache(v=FAR), **kw) == code


@pytest.mark.parametrize("kw,code", [(dict(n=-1), BAD), (dict(src=0), BAD), (dict(dst=0), BAD),
                                     (dict(n=0, src=0, dst=0), OK)])
def test_copy(kw, code):
    assert copy(cache(v=FAR), **kw) == code


@pytest.mark.parametrize("kw", [dict(stride_page=0), dict(stride_token=0), dict(stride_head=64),
                                dict(v=FAKE)])
def test_a_cache_that_overlaps_is_not_written(kw):
    c = cache(**{"v": FAR, **kw})
    assert compact(c) == BAD and copy(c) == BAD


def fork(**kw):
    a = dict(src=FAKE, dst=FAKE, F=3, ctx=FAKE, B=4, table=FAKE, max_pages=8, stride=8, refs=FAKE,
             free=FAKE, cap=9, n=FAKE, pages=9, page=16, from_=FAKE, to=FAKE, tokens=FAKE)
    a.update(kw)
    return B.moe_kv_fork(*a.values(), 0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(F=-1), BAD), (dict(F=8193), BAD), (dict(B=-1), BAD), (dict(B=0), BAD), (dict(B=8193), BAD),
    (dict(max_pages=0), BAD), (dict(stride=7), BAD), (dict(cap=-1), BAD), (dict(pages=0), BAD),
    (dict(page=0), BAD), (dict(pages=1 << 20, page=1 << 12), BAD),
    (dict(F=8192, max_pages=1 << 18, stride=1 << 18), BAD),
    *((dict([(k, 0)]), BAD) for k in ("src", "dst", "ctx", "table", "refs", "free", "n", "from_", "to",
                                      "tokens")), (dict(F=0, src=0), OK)])
def test_fork(kw, code):
    assert fork(**kw) == code


def trim(**kw):
    a = dict(keep=FAKE, lens=FAKE, B=4, table=FAKE, max_pages=8, stride=8, free=FAKE, cap=9, n=FAKE,
             refs=0, pages=9, page=16)
    a.update(kw)
    return B.moe_kv_trim(*a.values(), 0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(B=8193), BAD), (dict(max_pages=0), BAD), (dict(stride=7), BAD),
    (dict(cap=-1), BAD), (dict(pages=0), BAD), (dict(page=0), BAD),
    (dict(B=8192, max_pages=1 << 18, stride=1 << 18), BAD),
    *((dict([(k, 0)]), BAD) for k in ("keep", "lens", "table", "free", "n")),
    (dict(B=0, keep=0), OK)])
def test_trim(kw, code):
    assert trim(**kw) == code


def adjust(settings=(), **kw):
    s = dict(requests=2, max_history=10, n_bias=3, history_stride=10, allowed_stride=4, history=FAKE,
             history_lens=FAKE, bias_ids=FAKE, bias=FAKE, allowed=FAKE)
    s.update(settings)
    a = dict(x=FAKE, dtype=B.MOE_LOGITS_F32, N=2, V=100, stride=100, out=FAR, out_stride=100)
    a.update(kw)
    return B.moe_adjust_logits(B.MoeAdjust(**s), *a.values(), 0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(N=65536), BAD), (dict(V=0), BAD), (dict(V=(1 << 18) + 1), BAD),
    (dict(stride=-1), BAD), (dict(dtype=2), BAD), (dict(x=0), BAD), (dict(out=0), BAD),
    (dict(x=FAKE + 2), BAD), (dict(out=FAR + 1), BAD), (dict(out_stride=99), BAD),
    (dict(out=FAKE + 400), BAD),                              # overlaps the logits
    (dict(out=FAKE, out_stride=200), BAD), (dict(out=FAKE - 4), BAD),
    (dict(settings=dict(requests=-1)), BAD), (dict(settings=dict(requests=1)), BAD),
    (dict(settings=dict(max_history=-1)), BAD), (dict(settings=dict(n_bias=-1)), BAD),
    (dict(settings=dict(n_bias=1025)), BAD), (dict(settings=dict(history_lens=0)), BAD),
    (dict(settings=dict(bias=0)), BAD), (dict(settings=dict(bias_ids=0)), BAD),
    (dict(settings=dict(history_stride=-1)), BAD), (dict(settings=dict(allowed_stride=-1)), BAD),
    (dict(N=0, x=0, out=0), OK)])
def test_adjust(kw, code):
    assert adjust(**kw) == code


def test_struct_matches_the_header(tmp_path):
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_route.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu\\n", sizeof(moe_adjust_t),'
                   " offsetof(moe_adjust_t, history_stride), offsetof(moe_adjust_t, rows),"
                   " offsetof(moe_adjust_t, allowed)); return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    A = B.MoeAdjust
    assert got == [ctypes.sizeof(A), A.history_stride.offset, A.rows.offset, A.allowed.offset]


def test_wrappers_refuse_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 4, dtype=torch.int32)
    kc = torch.zeros(4, 16, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.tree_masks(i, i, i[:1], max_new=4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.tree_accept(i, i, i, i, i[:1], max_path=4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.attn_tree(torch.zeros(2, 2, 64), kc, kc, t, i, i[:1], max_new=4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.kv_compact(t, i, i, t, kc, kc)
    with pytest.raises(ValueError, match="CUDA"):
        moe.kv_copy_pages(i, i, kc, kc)
    with pytest.raises(ValueError, match="CUDA"):
        moe.kv_fork(i, i, i, t, i, i, i[:1], page_size=4, num_pages=2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.kv_trim(i, i, t, i, i[:1], page_size=4, num_pages=2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.adjust_logits(torch.zeros(2, 8))


@pytest.mark.parametrize("window", [1, 2, 4, 9, 30])
def test_plain_form_of_a_window_is_that_of_one_token_at_a_time(window):
    rng = np.random.default_rng(window)
    ctx, sizes, page = [3, 0, 20], [6, 15, 2], 4
    lens, starts = np.add(ctx, sizes), np.concatenate([[0], np.cumsum(sizes)])
    table = rng.permutation(30).reshape(3, 10)
    k, v, q = (rng.standard_normal(s) for s in ((30, page, 2, 8), (30, page, 2, 8), (sum(sizes), 4, 8)))
    of = [r for r, n in enumerate(sizes) for _ in range(n)]
    upto = [ctx[r] + i - starts[r] + 1 for i, r in enumerate(of)]
    want = D64.attend(q, k, v, table[of], upto, 0.3, window)
    got = R.attend(q, k, v, table, starts, lens, None, 15, 0.3, window)
    # either form: logits of 8 products that add up to 40 at most, so off by 8 x 40 x 2^-53;
    # values below 5, their weights off by twice that, sums of 30: 5 (640 + 30) 2^-53
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=2 * 5 * 670 * 2.0 ** -53)


@pytest.mark.parametrize("kw,code", [
    (dict(mask_words=-1), BAD), (dict(mask_words=5), BAD), (dict(mask_words=1), BAD),
    (dict(mask_words=1, tokens=FAKE, masks=FAKE), BAD), (dict(mask_words=4, tokens=FAKE, starts=FAKE), BAD),
    (dict(mask_words=4, masks=FAKE, starts=FAKE), BAD)])
def test_adjust_of_drafted_tokens(kw, code):
    assert adjust(settings=kw) == code


def test_where_the_struct_has_drafted_tokens(tmp_path):
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_route.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu\\n", offsetof(moe_adjust_t, mask_words),'
                   " offsetof(moe_adjust_t, tokens), offsetof(moe_adjust_t, masks),"
                   " offsetof(moe_adjust_t, starts)); return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    A = B.MoeAdjust
    assert got == [A.mask_words.offset, A.tokens.offset, A.masks.offset, A.starts.offset]
