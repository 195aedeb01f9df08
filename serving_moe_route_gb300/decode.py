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


# The current stream's handle for a device number: a tenth of a microsecond
# where torch.cuda.current_stream() builds an object in three
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _on(t, stream):
    """(device number, stream handle) for a call whose tensors live with t."""
    dev = t.get_device()
    if stream is not None:
        return dev, stream.cuda_stream
    return dev, _raw_stream(dev) if dev >= 0 else 0


def _refuse(t, dtype, n, name, dev):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have shape {(n,)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _vec(t, dtype, n, name, dev):
    """The address of a contiguous vector of n elements on device dev."""
    if (t.dtype is not dtype or t.shape != (n,) or t.get_device() != dev or dev < 0
            or not t.is_contiguous()):
        _refuse(t, dtype, n, name, dev)
    return t.data_ptr()


def _table(t, rows, dev):
    """(address, max_pages, stride) of a block table."""
    shape = t.shape
    if t.dtype is not torch.int32 or len(shape) != 2 or shape[0] != rows or shape[1] < 1:
        raise ValueError(f"block_table must be int32 [{rows}, max_pages], got {t.dtype} "
                         f"{tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"block_table must be on cuda:{dev}, got {t.device}")
    width = shape[1]
    stride, inner = t.stride()
    if rows and (width > 1 and inner != 1 or rows > 1 and stride < width):
        raise ValueError("block_table's rows must be contiguous and must not overlap")
    return t.data_ptr(), width, stride if rows > 1 else width


def _strides(t):
    """Strides, with 0 for axes of one element (theirs have no meaning) and 1
    for a last axis of one."""
    st, shape = t.stride(), t.shape
    if 1 in shape:
        last = len(shape) - 1
        st = tuple(x if n != 1 else int(i == last) for i, (x, n) in enumerate(zip(st, shape)))
    return st


def _cache(k, v, k_scale, v_scale, dev):
    """The C descriptor of a cache."""
    dtype, shape = k.dtype, k.shape
    kv = _KV_DTYPE.get(dtype)
    if dev < 0 or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("the cache and what goes with it must be CUDA tensors of one device")
    if kv is None:
        raise ValueError(f"k_cache must be float32, bfloat16 or float8_e4m3fn, got {dtype}")
    st = _strides(k)
    if v.dtype is not dtype or len(shape) != 4 or v.shape != shape or _strides(v) != st:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, kv_heads, head_dim] "
                         "of one type and the same strides")
    if st[3] != 1:
        raise ValueError("a cached vector's elements must be contiguous")
    ks = vs = None
    if kv == B.MOE_KV_E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale")
        ks = _vec(k_scale, torch.float32, shape[2], "k_scale", dev)
        vs = _vec(v_scale, torch.float32, shape[2], "v_scale", dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales are only used by a float8_e4m3fn cache")
    return B.MoeKvCache(kv, *shape, 0, st[0], st[1], st[2], k.data_ptr(), v.data_ptr(), ks, vs)


def _rows3(t, dtype, shape, name, dev):
    """The strides of a [n, heads, head_dim] tensor with contiguous vectors."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    st = _strides(t)
    if st[2] != 1:
        raise ValueError(f"{name}'s vectors must be contiguous")
    return st


def _err(err, dev):
    return 0 if err is None else _vec(err, torch.int32, 1, "err", dev)


def kv_step(ctx_lens, new_lens, block_table, free_pages, n_free, *, page_size, num_pages,
            max_tokens, n_free_out=None, err=None, stream=None) -> KVStep:
    """Grow the block tables for one step and map its new tokens to slots.

    Request r has ``ctx_lens[r]`` tokens in the cache and gets ``new_lens[r]``
    more; the pages it needs beyond those it has are taken from the end of
    ``free_pages[:n_free]`` and written into its row of ``block_table`` (in
    place).  ``max_tokens`` is the number of token rows to map; rows past the
    last new token get slot -1.  ``n_free_out`` may be ``n_free`` itself; by
    default the number left is a new tensor and the call can be repeated."""
    n = len(ctx_lens)
    dev, st = _on(ctx_lens, stream)
    ctx = _vec(ctx_lens, torch.int32, n, "ctx_lens", dev)
    new = _vec(new_lens, torch.int32, n, "new_lens", dev)
    table, width, stride = _table(block_table, n, dev)
    free = _vec(free_pages, torch.int32, len(free_pages), "free_pages", dev)
    left = _vec(n_free, torch.int32, 1, "n_free", dev)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    # one allocation for all outputs
    slots, positions, starts, seq_lens, left_out = torch.empty(
        2 * max_tokens + 2 * n + 2, dtype=torch.int32, device=ctx_lens.device).split_with_sizes(
            (max_tokens, max_tokens, n + 1, n, 1))
    if n_free_out is None:
        n_free_out = left_out
    rc = B.lib().moe_kv_step(
        ctx, new, n, table, width, stride, free, len(free_pages), left,
        _vec(n_free_out, torch.int32, 1, "n_free_out", dev), num_pages, page_size, max_tokens,
        slots.data_ptr(), positions.data_ptr(), starts.data_ptr(), seq_lens.data_ptr(),
        _err(err, dev), st)
    B._check(rc, "moe_kv_step")
    return KVStep(slots, positions, starts, seq_lens, n_free_out)


def kv_release(done, block_table, free_pages, n_free, *, num_pages, err=None, stream=None):
    """Give the pages of the requests with ``done[r] != 0`` back: they go to
    the end of ``free_pages[:n_free]``, ``n_free`` grows, and their rows of
    ``block_table`` become -1 (all in place).  A row must hold -1 where it
    holds no page."""
    n = len(done)
    dev, st = _on(done, stream)
    at = _vec(done, torch.int32, n, "done", dev)
    table, width, stride = _table(block_table, n, dev)
    free = _vec(free_pages, torch.int32, len(free_pages), "free_pages", dev)
    rc = B.lib().moe_kv_release(at, n, table, width, stride, free, len(free_pages),
                                _vec(n_free, torch.int32, 1, "n_free", dev), num_pages,
                                _err(err, dev), st)
    B._check(rc, "moe_kv_release")


def kv_append(k, v, slots, k_cache, v_cache, *, k_scale=None, v_scale=None, err=None, stream=None):
    """Write N tokens' keys and values ``[N, kv_heads, head_dim]`` (float32 for
    a float32 cache, else bfloat16) into the cache at ``slots`` (int32 [N], -1
    skips).  A float8 cache gets ``x / scale``, rounded and saturated."""
    dev, st = _on(k_cache, stream)
    c = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    n = len(slots)
    dt = torch.float32 if c.kv_dtype == B.MOE_KV_F32 else torch.bfloat16
    shape = (n, c.kv_heads, c.head_dim)
    ks, vs = _rows3(k, dt, shape, "k", dev), _rows3(v, dt, shape, "v", dev)
    rc = B.lib().moe_kv_append(c, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], n,
                               _vec(slots, torch.int32, n, "slots", dev), _err(err, dev), st)
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
    dev, st = _on(k_cache, stream)
    c = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, head_dim]")
    shape = q.shape
    n, hq, dim = shape
    if dim != c.head_dim:
        raise ValueError(f"q must have shape {(n, hq, c.head_dim)}, got {tuple(shape)}")
    dt = torch.float32 if c.kv_dtype == B.MOE_KV_F32 else torch.bfloat16
    qs = _rows3(q, dt, shape, "q", dev)
    if hq < 1 or hq % c.kv_heads:
        raise ValueError(f"Hq={hq} is not a multiple of kv_heads={c.kv_heads}")
    table, width, stride = _table(block_table, n, dev)
    lens = _vec(seq_lens, torch.int32, n, "seq_lens", dev)
    device = k_cache.device
    if out is None:
        out = torch.empty(shape, dtype=dt, device=device)
        os = (hq * dim, dim)
    else:
        os = _rows3(out, dt, shape, "out", dev)
    lse = torch.empty((n, hq), dtype=torch.float32, device=device) if return_lse else None
    if workspace is None:
        size = _WORKSPACE.get((dev, k_cache.dtype, dim))
        if size is None:
            with torch.cuda.device(dev):
                size = attn_workspace(k_cache.dtype, dim)
            _WORKSPACE[dev, k_cache.dtype, dim] = size
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
        ws = workspace.data_ptr()
    else:
        size = len(workspace)
        ws = _vec(workspace, torch.uint8, size, "workspace", dev)
    rc = B.lib().moe_attn_decode(c, q.data_ptr(), qs[0], qs[1], n, hq, table, width, stride, lens,
                                 dim ** -0.5 if scale is None else scale, window, out.data_ptr(),
                                 os[0], os[1], 0 if lse is None else lse.data_ptr(), ws, size,
                                 _err(err, dev), st)
    B._check(rc, "moe_attn_decode")
    return (out, lse) if return_lse else out


_WORKSPACE = {}  # bytes by (device, cache type, head_dim)


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
    dev, st = _on(logits, stream)
    if dev < 0:
        raise ValueError("logits must be a CUDA tensor")
    ldt = _LOGITS_DTYPE.get(logits.dtype)
    if ldt is None:
        raise ValueError("logits must be float32 or bfloat16")
    if logits.dim() != 2 or logits.shape[1] < 1 or logits.shape[1] > 1 and logits.stride(1) != 1:
        raise ValueError("logits must be [B, V] with contiguous rows")
    n, V = logits.shape
    f32 = torch.float32
    at = _vec(u, f32, n, "u", dev)
    t = 0 if temperature is None else _vec(temperature, f32, n, "temperature", dev)
    k = 0 if top_k is None else _vec(top_k, torch.int32, n, "top_k", dev)
    p = 0 if top_p is None else _vec(top_p, f32, n, "top_p", dev)
    m = 0 if min_p is None else _vec(min_p, f32, n, "min_p", dev)
    ids = torch.empty(n, dtype=torch.int32, device=logits.device)
    probs = torch.empty(n, dtype=f32, device=logits.device)
    rc = B.lib().moe_sample(logits.data_ptr(), ldt, n, V, logits.stride(0) if n > 1 else V, at, t,
                            k, p, m, ids.data_ptr(), probs.data_ptr(), st)
    B._check(rc, "moe_sample")
    return ids, probs


def check_word(err, stream=None):
    """Synchronise, read and clear an error word: (rc, device error bits)."""
    dev, st = _on(err, stream)
    return B.moe_check_word(_vec(err, torch.int32, 1, "err", dev), st)
