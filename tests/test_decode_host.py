"""Refusals of the decode-step calls, all of them made on the host before
anything is launched (no GPU here), and of their Python wrappers for CPU
tensors: there is no CPU fallback."""
import ctypes

import pytest
import torch

import serving_moe_route_gb300 as moe
from serving_moe_route_gb300 import _binding as B

FAKE = 1 << 20  # never dereferenced: validation fails first
OK = B.MOE_OK
BAD, UNSUPPORTED, SHORT = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def library():
    from serving_moe_route_gb300 import _build

    _build.build()


def cache(**kw):
    a = dict(kv_dtype=B.MOE_KV_BF16, num_pages=8, page_size=16, kv_heads=2, head_dim=128,
             reserved0=0, stride_page=16 * 256, stride_token=256, stride_head=128, k=FAKE, v=FAKE,
             k_scale=None, v_scale=None)
    a.update(kw)
    return B.MoeKvCache(**a)


BAD_CACHES = [
    (dict(kv_dtype=3), BAD), (dict(kv_dtype=-1), BAD), (dict(num_pages=0), BAD),
    (dict(page_size=0), BAD), (dict(kv_heads=0), BAD), (dict(head_dim=0), BAD),
    (dict(num_pages=1 << 20, page_size=1 << 12), BAD),        # slots past 2^31
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(stride_token=-256), BAD),
    (dict(k_scale=FAKE), BAD),                                # scales without an 8-bit cache
    (dict(kv_dtype=B.MOE_KV_E4M3), BAD),                      # and the other way round
    (dict(kv_dtype=B.MOE_KV_E4M3, k_scale=FAKE), BAD),
    (dict(head_dim=264), UNSUPPORTED), (dict(head_dim=100), UNSUPPORTED),
    (dict(kv_dtype=B.MOE_KV_E4M3, k_scale=FAKE, v_scale=FAKE, head_dim=72), UNSUPPORTED),
    (dict(k=FAKE + 8), UNSUPPORTED), (dict(v=FAKE + 2), UNSUPPORTED),
    (dict(stride_token=260), UNSUPPORTED), (dict(stride_head=129), UNSUPPORTED),
]


def append(c, **kw):
    a = dict(k=FAKE, ks=(256, 128), v=FAKE, vs=(256, 128), N=4, slots=FAKE)
    a.update(kw)
    return B.moe_kv_append(c, a["k"], *a["ks"], a["v"], *a["vs"], a["N"], a["slots"], 0, 0)


def attend(c, **kw):
    a = dict(q=FAKE, qb=1024, qh=128, B=2, Hq=8, table=FAKE, max_pages=4, stride=4, lens=FAKE,
             scale=1.0, window=0, out=FAKE, ob=1024, oh=128, lse=0, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return B.moe_attn_decode(c, a["q"], a["qb"], a["qh"], a["B"], a["Hq"], a["table"],
                             a["max_pages"], a["stride"], a["lens"], a["scale"], a["window"],
                             a["out"], a["ob"], a["oh"], a["lse"], a["ws"], a["ws_bytes"], 0, 0)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_descriptor(kw, code):
    assert append(cache(**kw)) == code
    assert attend(cache(**kw)) == code
    assert B.strerror(code)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(k=0), BAD), (dict(v=0), BAD), (dict(slots=0), BAD),
    (dict(ks=(-256, 128)), BAD), (dict(vs=(256, -1)), BAD), (dict(k=FAKE + 1), BAD),
    (dict(N=0, k=0, v=0, slots=0), OK)])
def test_append(kw, code):
    assert append(cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(Hq=0), BAD), (dict(Hq=7), BAD), (dict(max_pages=0), BAD),
    (dict(stride=3), BAD), (dict(window=-1), BAD), (dict(qb=-8), BAD), (dict(oh=-8), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(q=0), BAD),
    (dict(table=0), BAD), (dict(lens=0), BAD), (dict(out=0), BAD), (dict(ws=0), BAD),
    (dict(max_pages=1 << 28, stride=1 << 28), BAD),           # lengths past an int
    (dict(ws=FAKE + 16), BAD), (dict(q=FAKE + 8), UNSUPPORTED), (dict(out=FAKE + 2), UNSUPPORTED),
    (dict(qh=129), UNSUPPORTED), (dict(ob=1028), UNSUPPORTED),
    (dict(B=0, q=0, table=0, lens=0, out=0, ws=0), OK)])
def test_attend(kw, code):
    assert attend(cache(), **kw) == code


def step(**kw):
    a = dict(ctx=FAKE, new=FAKE, B=4, table=FAKE, max_pages=8, stride=8, free=FAKE, cap=100,
             n_in=FAKE, n_out=FAKE, pages=100, page=16, tokens=4, slots=FAKE, pos=FAKE, starts=FAKE,
             lens=FAKE)
    a.update(kw)
    return B.moe_kv_step(a["ctx"], a["new"], a["B"], a["table"], a["max_pages"], a["stride"],
                         a["free"], a["cap"], a["n_in"], a["n_out"], a["pages"], a["page"],
                         a["tokens"], a["slots"], a["pos"], a["starts"], a["lens"], 0, 0)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(B=8193), dict(max_pages=0), dict(stride=7), dict(cap=-1), dict(pages=0),
    dict(page=0), dict(tokens=-1), dict(pages=1 << 20, page=1 << 12), dict(n_in=0), dict(n_out=0),
    dict(starts=0), dict(ctx=0), dict(new=0), dict(table=0), dict(lens=0), dict(slots=0),
    dict(pos=0), dict(free=0)])
def test_step(kw):
    assert step(**kw) == BAD


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(B=8193), BAD), (dict(max_pages=0), BAD), (dict(stride=7), BAD),
    (dict(cap=-1), BAD), (dict(pages=0), BAD), (dict(done=0), BAD), (dict(table=0), BAD),
    (dict(n=0), BAD), (dict(free=0), BAD), (dict(B=0, done=0, table=0, n=0), OK)])
def test_release(kw, code):
    a = dict(done=FAKE, B=4, table=FAKE, max_pages=8, stride=8, free=FAKE, cap=9, n=FAKE, pages=9)
    a.update(kw)
    assert B.moe_kv_release(a["done"], a["B"], a["table"], a["max_pages"], a["stride"], a["free"],
                            a["cap"], a["n"], a["pages"], 0, 0) == code


def sample(**kw):
    a = dict(logits=FAKE, dtype=B.MOE_LOGITS_F32, B=2, V=100, stride=100, u=FAKE, t=0, k=0, p=0,
             m=0, ids=FAKE, probs=0)
    a.update(kw)
    return B.moe_sample(a["logits"], a["dtype"], a["B"], a["V"], a["stride"], a["u"], a["t"],
                        a["k"], a["p"], a["m"], a["ids"], a["probs"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(B=65536), BAD), (dict(V=0), BAD), (dict(V=(1 << 18) + 1), BAD),
    (dict(stride=-1), BAD), (dict(dtype=2), BAD), (dict(logits=0), BAD), (dict(u=0), BAD),
    (dict(ids=0), BAD), (dict(logits=FAKE + 2), BAD), (dict(B=0, logits=0, u=0, ids=0), OK)])
def test_sample(kw, code):
    assert sample(**kw) == code


def test_check_word_and_workspace():
    assert B.moe_check_word(0, 0)[0] == BAD
    assert B.moe_attn_workspace(7, 128) == 0
    assert B.moe_attn_workspace(B.MOE_KV_BF16, 300) == 0
    with pytest.raises(ValueError, match="no cache"):
        moe.attn_workspace(torch.float16, 128)


def test_struct_matches_the_header(tmp_path):
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_route.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu\\n", sizeof(moe_kv_cache_t),'
                   " offsetof(moe_kv_cache_t, stride_page), offsetof(moe_kv_cache_t, k),"
                   " offsetof(moe_kv_cache_t, v_scale)); return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    C = B.MoeKvCache
    assert got == [ctypes.sizeof(C), C.stride_page.offset, C.k.offset, C.v_scale.offset]


def test_wrappers_refuse_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 4, dtype=torch.int32)
    kc = torch.zeros(4, 16, 2, 64)
    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.kv_step(i, i, t, i, i[:1], page_size=16, num_pages=4, max_tokens=2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.kv_release(i, t, i, i[:1], num_pages=4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.kv_append(x, x, i, kc, kc)
    with pytest.raises(ValueError, match="CUDA"):
        moe.attn_decode(x, kc, kc, t, i)
    with pytest.raises(ValueError, match="CUDA"):
        moe.sample_tokens(torch.zeros(2, 8), torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        moe.check_word(i[:1])


@pytest.mark.parametrize("kw", [
    dict(stride_page=0), dict(stride_token=0), dict(stride_head=0), dict(stride_head=64),
    dict(stride_token=120), dict(v=FAKE)])
def test_append_refuses_a_cache_that_overlaps(kw):
    # heads, rows or pages that are one memory, or keys and values that are
    assert append(cache(**{"v": FAKE + (1 << 30), **kw})) == BAD


@pytest.mark.parametrize("kw", [dict(ob=0), dict(oh=0), dict(oh=120), dict(ob=64)])
def test_attend_refuses_an_output_that_overlaps(kw):
    assert attend(cache(), **kw) == BAD
