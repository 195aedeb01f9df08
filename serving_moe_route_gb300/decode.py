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

A step may check several drafted tokens per request (speculation): a tree whose
node 0 follows the context, packed by request like any new tokens::

    step = kv_step(ctx_lens, nodes, block_table, free_pages, n_free, page_size=16,
                   num_pages=P, max_tokens=N, n_free_out=n_free, err=err)
    tree = tree_masks(parents, step.starts, step.seq_lens, max_new=M, err=err)
    for each layer:                                  # rotary embeddings: tree.positions
        kv_append(k, v, step.slots, k_cache, v_cache, err=err)
        out = attn_tree(q, k_cache, v_cache, block_table, step.starts, step.seq_lens,
                        tree.masks, max_new=M, err=err)
        ...
    logits = adjust_logits(logits, rows=request_of_row, history=..., allowed=..., tokens=tokens,
                           masks=tree.masks, starts=step.starts, err=err)
    draws, _ = sample_tokens(logits, u, temperature=t)
    walk = tree_accept(tokens, draws, parents, step.starts, ctx_lens, max_path=M, err=err)
    for each layer:
        kv_compact(walk.path, walk.accepted, ctx_lens, block_table, k_cache, v_cache, err=err)
    kv_trim(walk.seq_lens, step.seq_lens, block_table, free_pages, n_free, page_size=16,
            num_pages=P, err=err)

Requests may share pages: ``kv_fork`` lets rows go on from another one's pages,
``kv_copy_pages`` copies the partial ones, and ``kv_trim`` with the same
``page_refs`` gives a page back when its last holder does (``kv_release`` does not
look at them).  A request that was trimmed back into a page that it shares goes on
in another row, as a fork of its own: its next token would be written to that page.

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


class TreeMasks(NamedTuple):
    """What ``tree_masks`` returns."""
    masks: torch.Tensor      # int64 [N, ceil(max_new / 64)] nodes that each row attends
    positions: torch.Tensor  # int32 [N] context tokens + depth


class TreeAccept(NamedTuple):
    """What ``tree_accept`` returns (int32 tensors)."""
    path: torch.Tensor      # [B, max_path] accepted nodes, -1 behind them
    accepted: torch.Tensor  # [B] how many
    next_ids: torch.Tensor  # [B] the token drawn at the last one
    seq_lens: torch.Tensor  # [B] context tokens, the accepted ones included


class KVFork(NamedTuple):
    """What ``kv_fork`` returns (int32 [F]): the partial pages to copy."""
    src_pages: torch.Tensor
    dst_pages: torch.Tensor
    tokens: torch.Tensor


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


def tree_masks(parents, starts, seq_lens, *, max_new, err=None, stream=None) -> TreeMasks:
    """Masks and positions of trees of drafted tokens.  ``parents`` (int32 [N],
    packed by request) holds each node's parent by its number in the request,
    lower than its own, -1 for the root; ``starts`` and ``seq_lens`` are those of
    ``kv_step``; ``max_new`` (up to 256) bounds a request's nodes.  A node attends
    itself and its ancestors.  Rows of no request get zeros."""
    return TreeMasks(*_ext().tree_masks(parents, starts, seq_lens, max_new, err, _handle(stream)))


def attn_tree(q, k_cache, v_cache, block_table, starts, seq_lens, masks=None, *, max_new,
              scale=None, window=0, k_scale=None, v_scale=None, out=None, return_lse=False,
              workspace=None, err=None, stream=None):
    """Attention of several new tokens per request: q ``[N, Hq, head_dim]`` packed
    by request.  A row attends its request's context and the new tokens whose bits
    are set in its mask (``tree_masks``), by default those up to itself.  With a
    ``window``, it attends the last ``window`` of these, and where they are fewer, c,
    the last ``window - c`` of the context.  Otherwise as ``attn_decode``: returns out,
    or (out, lse) with lse ``[N, Hq]``; a row that attends nothing gets zeros and -inf,
    rows of no request are left as they are.  ``workspace`` is a uint8 tensor of
    ``attn_tree_workspace(...)`` bytes (by default one is allocated)."""
    return _ext().attn_tree(q, k_cache, v_cache, block_table, starts, seq_lens, masks, max_new,
                            scale, window, k_scale, v_scale, out, return_lse, workspace, err,
                            _handle(stream))


def attn_tree_workspace(kv_dtype: torch.dtype, head_dim: int) -> int:
    """Bytes of workspace that ``attn_tree`` needs on the current device."""
    if kv_dtype not in _KV_DTYPE:
        raise ValueError(f"no cache of {kv_dtype}")
    return B.moe_attn_tree_workspace(_KV_DTYPE[kv_dtype], head_dim)


def tree_accept(tokens, draws, parents, starts, ctx_lens, *, max_path, err=None,
                stream=None) -> TreeAccept:
    """Walk each tree from node 0 along the tokens drawn: the next node is the
    lowest child of the current one whose drafted token (``tokens``, int32 [N]) is
    the one drawn there (``draws``, int32 [N]); at most ``max_path`` nodes."""
    return TreeAccept(*_ext().tree_accept(tokens, draws, parents, starts, ctx_lens, max_path, err,
                                          _handle(stream)))


def kv_compact(path, accepted, ctx_lens, block_table, k_cache, v_cache, *, err=None, stream=None):
    """Move the keys and values of the accepted nodes (``path`` int32 [B, P],
    rising, ``accepted`` int32 [B]) together: token ``ctx + path[j]`` of a request
    goes to ``ctx + j``, in place."""
    _ext().kv_compact(path, accepted, ctx_lens, block_table, k_cache, v_cache, err,
                      _handle(stream))


def kv_fork(src_rows, dst_rows, ctx_lens, block_table, page_refs, free_pages, n_free, *, page_size,
            num_pages, err=None, stream=None) -> KVFork:
    """Let rows ``dst_rows`` of the block table (int32 [F], without pages) go on
    from rows ``src_rows``: full pages are shared (``page_refs``, int32
    [num_pages], counts a page's holders beyond the first), a partial last page is
    replaced by one from the end of ``free_pages[:n_free]``.  ``ctx_lens``,
    ``block_table``, ``page_refs`` and ``n_free`` are updated in place.  Returns
    the partial pages, for ``kv_copy_pages`` on each layer's cache."""
    return KVFork(*_ext().kv_fork(src_rows, dst_rows, ctx_lens, block_table, page_refs, free_pages,
                                  n_free, page_size, num_pages, err, _handle(stream)))


def kv_copy_pages(src_pages, dst_pages, k_cache, v_cache, *, tokens=None, err=None, stream=None):
    """Copy the first ``tokens[i]`` tokens (all by default) of page
    ``src_pages[i]`` to page ``dst_pages[i]`` (int32 [n]; -1 skips a pair).  A page
    that is written must stand in the call once."""
    _ext().kv_copy_pages(src_pages, dst_pages, k_cache, v_cache, tokens, err, _handle(stream))


def kv_trim(keep_lens, seq_lens, block_table, free_pages, n_free, *, page_size, num_pages,
            page_refs=None, err=None, stream=None):
    """Give back the pages of each request past its first ``keep_lens[r]`` of
    ``seq_lens[r]`` tokens: their entries of ``block_table`` become -1 and they go
    to the end of ``free_pages[:n_free]``, ``n_free`` grows (all in place).  With
    ``page_refs`` a shared page loses a holder, and is freed with its last one."""
    _ext().kv_trim(keep_lens, seq_lens, block_table, free_pages, n_free, page_size, num_pages,
                   page_refs, err, _handle(stream))


def adjust_logits(logits, *, rows=None, history=None, history_lens=None, prompt_lens=None,
                  repetition=None, presence=None, frequency=None, bias_ids=None, bias=None,
                  allowed=None, tokens=None, masks=None, starts=None, out=None, err=None,
                  stream=None):
    """Logits [N, V] (float32 or bfloat16) with penalties, biases and a grammar's
    mask applied, before ``sample_tokens``.  Row i belongs to request ``rows[i]``
    (int32 [N]; by default i).  In this order: the logits of tokens in
    ``history[r, :history_lens[r]]`` (int32) are divided by ``repetition[r]`` if
    positive, multiplied otherwise; ``frequency[r]`` times a token's count in the
    history from ``prompt_lens[r]`` on, and ``presence[r]`` if there is any, are
    subtracted; ``bias[r, j]`` is added to token ``bias_ids[r, j]`` (-1 pads; of
    several for one token the last counts); tokens whose bit in ``allowed`` (int32
    [N, ceil(V / 32)], one row per row of logits) is not set become -inf.
    At the nodes of trees the drafted tokens on a node's path count as the end of its
    request's history: give ``tokens`` (int32 [N], as for ``tree_accept``), ``masks``
    (``tree_masks``) and ``starts``.  Node 0's token is the last of the history.
    ``out`` may be ``logits`` itself, or lie before or behind all of them; by default
    the result is a new tensor."""
    return _ext().adjust_logits(logits, rows, history, history_lens, prompt_lens, repetition,
                                presence, frequency, bias_ids, bias, allowed, tokens, masks, starts,
                                out, err, _handle(stream))


def check_word(err, stream=None):
    """Synchronise, read and clear an error word: (rc, device error bits)."""
    if err.device.type != "cuda":
        raise ValueError("err must be a CUDA tensor")
    if err.dtype != torch.int32 or err.numel() != 1:
        raise ValueError(f"err must be one torch.int32, got {err.dtype} {tuple(err.shape)}")
    with torch.cuda.device(err.device):
        return B.moe_check_word(err.data_ptr(), _stream(stream))
