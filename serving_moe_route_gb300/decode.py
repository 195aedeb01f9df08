"""The rest of a decode step around the layer: block tables and slot maps of a
paged key-value cache, the write of new keys and values, attention of one new
token per request over the cache, and sampling.

A cache is two tensors ``[num_pages, page_size, kv_heads, head_dim]`` of the
same strides, float32, bfloat16 or float8_e4m3fn (then with one float32 scale
per head for each); a permuted view of ``[num_pages, kv_heads, page_size,
head_dim]`` serves as well.  Like the layer, this module checks arguments and
passes pointers: the arithmetic runs in ``libmoe_route.so``.

One step of a server with its state on the GPU::

    step = kv_step(ctx_lens, new_lens, block_table, free_pages, n_free, page_size=16,
                   num_pages=P, max_tokens=B, n_free_out=n_free, err=err)
    for each layer:
        kv_append(k, v, step.slots, k_cache, v_cache, err=err)
        out = attn_decode(q, k_cache, v_cache, block_table, step.seq_lens, err=err)
        ...
    ids, probs = sample_tokens(logits, u, temperature=t, top_p=p)
    kv_release(done, block_table, free_pages, n_free, num_pages=P, err=err)

``err`` is an int32 tensor of one zero that collects error bits
(``MOE_DEVERR_*``) on the device; ``check_word`` reads and clears it.  Every
function enqueues on ``stream`` (the current one by default) and returns at
once, so the step can be captured into a CUDA graph.  Outputs and workspaces
are allocated for that stream; a tensor of one stream used on another is the
caller's to order, as everywhere in PyTorch.

Like the layer, none of these has a backward pass: outputs are cut off from the
graph of the inputs.  What is written in place counts as modified, so autograd
refuses a graph that needs its old values.
"""
from __future__ import annotations

import importlib.util
import os
from typing import NamedTuple

import torch

from . import _binding as B
from . import _build
from .layer import _stream

_KV_DTYPE = {torch.float32: B.MOE_KV_F32, torch.bfloat16: B.MOE_KV_BF16,
             torch.float8_e4m3fn: B.MOE_KV_E4M3}


class KVStep(NamedTuple):
    """What ``kv_step`` returns (int32 tensors)."""
    slots: torch.Tensor      # [max_tokens] slot of each new token, -1: none
    positions: torch.Tensor  # [max_tokens] its position in its request
    starts: torch.Tensor     # [B + 1] request r's tokens are starts[r] .. starts[r + 1] - 1
    seq_lens: torch.Tensor   # [B] tokens of each request, the new ones included
    n_free: torch.Tensor     # [1] free pages left


_ext_module = None


def _ext():
    """The extension module that makes the calls; raise if it has not been built."""
    global _ext_module
    if _ext_module is None:
        build = "build it with serving_moe_route_gb300._build.build() (or __graft_entry__.build())"
        if not os.path.exists(_build.EXT_PATH):
            raise RuntimeError(f"extension {_build.EXT_PATH} is missing: {build}")
        if not _build.ext_abi_matches():
            raise RuntimeError(f"extension {_build.EXT_PATH} was built against another PyTorch: "
                               f"{build}")
        B.lib()
        spec = importlib.util.spec_from_file_location("moe_decode_ext", _build.EXT_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _ext_module = module
    return _ext_module


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def kv_step(ctx_lens, new_lens, block_table, free_pages, n_free, *, page_size, num_pages,
            max_tokens, n_free_out=None, err=None, stream=None) -> KVStep:
    """Grow the block tables for one step and map its new tokens to slots.

    Request r has ``ctx_lens[r]`` tokens in the cache and gets ``new_lens[r]``
    more; the pages it needs beyond those it has are taken from the end of
    ``free_pages[:n_free]`` and written into its row of ``block_table`` (in
    place).  ``max_tokens`` is the number of token rows to map; rows past the
    last new token get slot -1.  ``n_free_out`` may be ``n_free`` itself; by
    default the number left is a new tensor and the call can be repeated."""
    return KVStep(*_ext().kv_step(ctx_lens, new_lens, block_table, free_pages, n_free, page_size,
                                  num_pages, max_tokens, n_free_out, err, _handle(stream)))


def kv_release(done, block_table, free_pages, n_free, *, num_pages, err=None, stream=None):
    """Give the pages of the requests with ``done[r] != 0`` back: they go to
    the end of ``free_pages[:n_free]``, ``n_free`` grows, and their rows of
    ``block_table`` become -1 (all in place).  A row must hold -1 where it
    holds no page."""
    _ext().kv_release(done, block_table, free_pages, n_free, num_pages, err, _handle(stream))


def kv_append(k, v, slots, k_cache, v_cache, *, k_scale=None, v_scale=None, err=None, stream=None):
    """Write N tokens' keys and values ``[N, kv_heads, head_dim]`` (float32 for
    a float32 cache, else bfloat16) into the cache at ``slots`` (int32 [N], -1
    skips).  A float8 cache gets ``x / scale``, rounded and saturated."""
    _ext().kv_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, err, _handle(stream))


def attn_decode(q, k_cache, v_cache, block_table, seq_lens, *, scale=None, window=0, k_scale=None,
                v_scale=None, out=None, return_lse=False, workspace=None, err=None, stream=None):
    """Attention of one new token per request: q ``[B, Hq, head_dim]`` over the
    last ``window`` (0: all) of the request's ``seq_lens[b]`` cached tokens,
    query head h on kv head ``h // (Hq // kv_heads)``.  ``scale`` is
    1/sqrt(head_dim) by default.  Returns out, or (out, lse) with the
    softmax's log-sum-exp ``[B, Hq]`` in float32; a request without tokens
    gets zeros and -inf.  ``workspace`` is a uint8 tensor of
    ``attn_workspace(...)`` bytes (by default one is allocated)."""
    return _ext().attn_decode(q, k_cache, v_cache, block_table, seq_lens, scale, window, k_scale,
                              v_scale, out, return_lse, workspace, err, _handle(stream))


def attn_workspace(kv_dtype: torch.dtype, head_dim: int) -> int:
    """Bytes of workspace that ``attn_decode`` needs on the current device."""
    if kv_dtype not in _KV_DTYPE:
        raise ValueError(f"no cache of {kv_dtype}")
    return B.moe_attn_workspace(_KV_DTYPE[kv_dtype], head_dim)


def sample_tokens(logits, u, *, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
    """The next token of each row of ``logits`` [B, V] (float32 or bfloat16)
    from one uniform random number in [0, 1) per row, ``u`` float32 [B].
    ``temperature``, ``top_p``, ``min_p`` (float32 [B]) and ``top_k`` (int32
    [B]) hold per row, None leaves that restriction out; temperature <= 0 is
    greedy.  Returns (ids int32 [B], probs float32 [B]): the drawn tokens and
    their shares of what was kept; -1 and 0 for a row without a token."""
    return _ext().sample_tokens(logits, u, temperature, top_k, top_p, min_p, _handle(stream))


def check_word(err, stream=None):
    """Synchronise, read and clear an error word: (rc, device error bits)."""
    if err.device.type != "cuda":
        raise ValueError("err must be a CUDA tensor")
    if err.dtype != torch.int32 or err.numel() != 1:
        raise ValueError(f"err must be one torch.int32, got {err.dtype} {tuple(err.shape)}")
    with torch.cuda.device(err.device):
        return B.moe_check_word(err.data_ptr(), _stream(stream))
