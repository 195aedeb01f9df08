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
once, so the step can be captured into a CUDA graph.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _binding as B
from .layer import _p, _stream

_KV_DTYPE = {torch.float32: B.MOE_KV_F32, torch.bfloat16: B.MOE_KV_BF16,
             torch.float8_e4m3fn: B.MOE_KV_E4M3}
_LOGITS_DTYPE = {torch.float32: B.MOE_LOGITS_F32, torch.bfloat16: B.MOE_LOGITS_BF16}


class KVStep(NamedTuple):
    """What ``kv_step`` returns (int32 tensors)."""
    slots: torch.Tensor      # [max_tokens] slot of each new token, -1: none
    positions: torch.Tensor  # [max_tokens] its position in its request
    starts: torch.Tensor     # [B + 1] request r's tokens are starts[r] .. starts[r + 1] - 1
    seq_lens: torch.Tensor   # [B] tokens of each request, the new ones included
    n_free: torch.Tensor     # [1] free pages left


def _vec(t, dtype, n, name, device):
    """A contiguous vector of n elements (n None: any length) on `device`."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must have shape {'[n]' if n is None else (n,)}, "
                         f"got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _table(t, rows, device):
    if not t.is_cuda:
        raise ValueError("block_table must be a CUDA tensor")
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != rows or t.shape[1] < 1:
        raise ValueError(f"block_table must be int32 [{rows}, max_pages], got {t.dtype} "
                         f"{tuple(t.shape)}")
    if rows and (t.shape[1] > 1 and t.stride(1) != 1 or rows > 1 and t.stride(0) < t.shape[1]):
        raise ValueError("block_table's rows must be contiguous and must not overlap")
    if t.device != device:
        raise ValueError(f"block_table must be on {device}, got {t.device}")
    return max(t.stride(0), t.shape[1])


def _strides(t):
    """Strides with 0 for axes of one element (their stride has no meaning)
    but the last."""
    n = t.shape
    return [s if n[i] > 1 else 0 for i, s in enumerate(t.stride()[:-1])] + [
        t.stride(-1) if n[-1] > 1 else 1]


def _cache(k, v, k_scale, v_scale):
    """The C descriptor of a cache."""
    if not k.is_cuda or k.device != v.device:
        raise ValueError("k_cache and v_cache must be CUDA tensors of one device")
    kv = _KV_DTYPE.get(k.dtype)
    if kv is None:
        raise ValueError(f"k_cache must be float32, bfloat16 or float8_e4m3fn, got {k.dtype}")
    shape, stride = k.shape, _strides(k)
    if v.dtype != k.dtype or len(shape) != 4 or v.shape != shape or _strides(v) != stride:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, kv_heads, head_dim] "
                         "of one type and the same strides")
    if stride[3] != 1:
        raise ValueError("a cached vector's elements must be contiguous")
    ks = vs = None
    if kv == B.MOE_KV_E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale")
        _vec(k_scale, torch.float32, shape[2], "k_scale", k.device)
        _vec(v_scale, torch.float32, shape[2], "v_scale", k.device)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales are only used by a float8_e4m3fn cache")
    return B.MoeKvCache(kv, shape[0], shape[1], shape[2], shape[3], 0, stride[0], stride[1],
                        stride[2], k.data_ptr(), v.data_ptr(), ks, vs)


def _rows3(t, dtype, shape, name, device):
    """The strides of a [n, heads, head_dim] tensor with contiguous vectors."""
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    stride = _strides(t)
    if stride[2] != 1:
        raise ValueError(f"{name}'s vectors must be contiguous")
    return stride


def _err(err, device):
    if err is None:
        return 0
    _vec(err, torch.int32, 1, "err", device)
    return err.data_ptr()


def kv_step(ctx_lens, new_lens, block_table, free_pages, n_free, *, page_size, num_pages,
            max_tokens, n_free_out=None, err=None, stream=None) -> KVStep:
    """Grow the block tables for one step and map its new tokens to slots.

    Request r has ``ctx_lens[r]`` tokens in the cache and gets ``new_lens[r]``
    more; the pages it needs beyond those it has are taken from the end of
    ``free_pages[:n_free]`` and written into its row of ``block_table`` (in
    place).  ``max_tokens`` is the number of token rows to map; rows past the
    last new token get slot -1.  ``n_free_out`` may be ``n_free`` itself; by
    default the number left is a new tensor and the call can be repeated."""
    n = ctx_lens.shape[0]
    dev = ctx_lens.device
    _vec(ctx_lens, torch.int32, None, "ctx_lens", dev)
    _vec(new_lens, torch.int32, n, "new_lens", dev)
    stride = _table(block_table, n, dev)
    _vec(free_pages, torch.int32, None, "free_pages", dev)
    _vec(n_free, torch.int32, 1, "n_free", dev)
    if n_free_out is not None:
        _vec(n_free_out, torch.int32, 1, "n_free_out", dev)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    # one allocation, cut so that every output is 16-byte aligned
    pad_t, pad_b = (max_tokens + 3) & ~3, (n + 4) & ~3
    buf = torch.empty(2 * pad_t + 2 * pad_b + 4, dtype=torch.int32, device=dev)
    slots, positions = buf[:max_tokens], buf[pad_t:pad_t + max_tokens]
    at = 2 * pad_t
    starts, seq_lens = buf[at:at + n + 1], buf[at + pad_b:at + pad_b + n]
    if n_free_out is None:
        n_free_out = buf[at + 2 * pad_b:at + 2 * pad_b + 1]
    base = buf.data_ptr()
    rc = B.moe_kv_step(_p(ctx_lens), _p(new_lens), n, _p(block_table), block_table.shape[1],
                       stride, _p(free_pages), free_pages.shape[0], _p(n_free), _p(n_free_out),
                       num_pages, page_size, max_tokens, base, base + 4 * pad_t, base + 4 * at,
                       base + 4 * (at + pad_b), _err(err, dev), _stream(stream))
    B._check(rc, "moe_kv_step")
    return KVStep(slots, positions, starts, seq_lens, n_free_out)


def kv_release(done, block_table, free_pages, n_free, *, num_pages, err=None, stream=None):
    """Give the pages of the requests with ``done[r] != 0`` back: they go to
    the end of ``free_pages[:n_free]``, ``n_free`` grows, and their rows of
    ``block_table`` become -1 (all in place).  A row must hold -1 where it
    holds no page."""
    n, dev = done.shape[0], done.device
    _vec(done, torch.int32, None, "done", dev)
    stride = _table(block_table, n, dev)
    _vec(free_pages, torch.int32, None, "free_pages", dev)
    _vec(n_free, torch.int32, 1, "n_free", dev)
    rc = B.moe_kv_release(_p(done), n, _p(block_table), block_table.shape[1], stride,
                          _p(free_pages), free_pages.shape[0], _p(n_free), num_pages,
                          _err(err, dev), _stream(stream))
    B._check(rc, "moe_kv_release")


def kv_append(k, v, slots, k_cache, v_cache, *, k_scale=None, v_scale=None, err=None, stream=None):
    """Write N tokens' keys and values ``[N, kv_heads, head_dim]`` (float32 for
    a float32 cache, else bfloat16) into the cache at ``slots`` (int32 [N], -1
    skips).  A float8 cache gets ``x / scale``, rounded and saturated."""
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    n = slots.shape[0]
    dt = torch.float32 if c.kv_dtype == B.MOE_KV_F32 else torch.bfloat16
    shape = (n, c.kv_heads, c.head_dim)
    ks, vs = _rows3(k, dt, shape, "k", dev), _rows3(v, dt, shape, "v", dev)
    _vec(slots, torch.int32, n, "slots", dev)
    rc = B.moe_kv_append(c, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], n, slots.data_ptr(), _err(err, dev), _stream(stream))
    B._check(rc, "moe_kv_append")


def attn_decode(q, k_cache, v_cache, block_table, seq_lens, *, scale=None, window=0, k_scale=None,
                v_scale=None, out=None, return_lse=False, workspace=None, err=None, stream=None):
    """Attention of one new token per request: q ``[B, Hq, head_dim]`` over the
    last ``window`` (0: all) of the request's ``seq_lens[b]`` cached tokens,
    query head h on kv head ``h // (Hq // kv_heads)``.  ``scale`` is
    1/sqrt(head_dim) by default.  Returns out, or (out, lse) with the
    softmax's log-sum-exp ``[B, Hq]`` in float32; a request without tokens
    gets zeros and -inf.  ``workspace`` is a uint8 tensor of
    ``attn_workspace(...)`` bytes (by default one is allocated)."""
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, head_dim]")
    n, hq = q.shape[0], q.shape[1]
    dt = torch.float32 if c.kv_dtype == B.MOE_KV_F32 else torch.bfloat16
    qs = _rows3(q, dt, (n, hq, c.head_dim), "q", dev)
    if hq < 1 or hq % c.kv_heads:
        raise ValueError(f"Hq={hq} is not a multiple of kv_heads={c.kv_heads}")
    stride = _table(block_table, n, dev)
    _vec(seq_lens, torch.int32, n, "seq_lens", dev)
    if out is None:
        out = torch.empty(n, hq, c.head_dim, dtype=dt, device=dev)
    os = _rows3(out, dt, (n, hq, c.head_dim), "out", dev)
    lse = torch.empty(n, hq, dtype=torch.float32, device=dev) if return_lse else None
    if workspace is None:
        workspace = torch.empty(attn_workspace(k_cache.dtype, c.head_dim), dtype=torch.uint8,
                                device=dev)
    else:
        _vec(workspace, torch.uint8, None, "workspace", dev)
    if scale is None:
        scale = c.head_dim ** -0.5
    rc = B.moe_attn_decode(c, q.data_ptr(), qs[0], qs[1], n, hq, block_table.data_ptr(),
                           block_table.shape[1], stride, seq_lens.data_ptr(), scale, window,
                           out.data_ptr(), os[0], os[1], _p(lse), workspace.data_ptr(), workspace.numel(),
                           _err(err, dev), _stream(stream))
    B._check(rc, "moe_attn_decode")
    return (out, lse) if return_lse else out


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
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    ldt = _LOGITS_DTYPE.get(logits.dtype)
    if ldt is None:
        raise ValueError("logits must be float32 or bfloat16")
    if logits.dim() != 2 or logits.shape[1] < 1 or logits.shape[1] > 1 and logits.stride(1) != 1:
        raise ValueError("logits must be [B, V] with contiguous rows")
    n, V = logits.shape
    dev = logits.device
    _vec(u, torch.float32, n, "u", dev)
    for t, dt, name in ((temperature, torch.float32, "temperature"), (top_k, torch.int32, "top_k"),
                        (top_p, torch.float32, "top_p"), (min_p, torch.float32, "min_p")):
        if t is not None:
            _vec(t, dt, n, name, dev)
    ids = torch.empty(n, dtype=torch.int32, device=dev)
    probs = torch.empty(n, dtype=torch.float32, device=dev)
    rc = B.moe_sample(logits.data_ptr(), ldt, n, V, logits.stride(0) if n > 1 else V, u.data_ptr(),
                      _p(temperature), _p(top_k), _p(top_p), _p(min_p), ids.data_ptr(),
                      probs.data_ptr(), _stream(stream))
    B._check(rc, "moe_sample")
    return ids, probs


def check_word(err, stream=None):
    """Synchronise, read and clear an error word: (rc, device error bits)."""
    _vec(err, torch.int32, 1, "err", err.device)
    return B.moe_check_word(err.data_ptr(), _stream(stream))
