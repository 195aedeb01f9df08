"""moe_sample on the GPU against the definition in 64 bits.

Ids have to be equal wherever the draw and the top-p cut are further from
their borders than the rounding of the weights explains (the reference gives
both; the weights' own error is part of what the kernel promises).  A
probability is a quotient of two sums rounded to fp32 three times: 3 x 2^-24,
and the weights' error."""
import numpy as np
import pytest
import torch

import decode_reference as R
import serving_moe_route_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _check(x, u, least=0.9, **kw):
    dev = {k: None if v is None else torch.as_tensor(
        np.asarray(v), dtype=torch.int32 if k == "top_k" else torch.float32, device=DEV)
        for k, v in kw.items()}
    u = torch.as_tensor(u, dtype=torch.float32, device=DEV)
    ids, probs = moe.sample_tokens(x, u, **dev)
    again, _ = moe.sample_tokens(x, u, **dev)
    assert torch.equal(ids, again)
    host = {k: None if v is None else v.cpu().numpy() for k, v in dev.items()}
    want, p, near, off = R.sample(R.f64(x), u.cpu().numpy(), largest=torch.finfo(x.dtype).max,
                                  **host)
    far = near > off
    assert far.mean() >= least
    np.testing.assert_array_equal(ids.cpu().numpy()[far], want[far])
    np.testing.assert_allclose(probs.cpu().numpy()[far], p[far], rtol=4 * 2.0 ** -24)
    return ids.cpu().numpy()


def _logits(seed, B, V, dt, spread=1.8, likely=40):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = spread * torch.randn(B, V, generator=g, device=DEV)
    if likely:
        at = torch.randint(V, (B, likely), generator=g, device=DEV)
        x.scatter_reduce_(1, at, 6 + 2 * torch.randn(B, likely, generator=g, device=DEV), "amax")
    return x.to(DT[dt]), torch.rand(B, generator=g, device=DEV)


def _settings(seed, B, V):
    rng = np.random.default_rng(seed)
    return dict(
        temperature=np.where(rng.random(B) < 0.15, 0.0, rng.uniform(0.3, 1.6, B)),
        top_k=np.where(rng.random(B) < 0.3, 0, rng.integers(1, max(2, min(V, 120)), B)),
        top_p=np.where(rng.random(B) < 0.3, 1.0, rng.uniform(0.05, 0.999, B)),
        min_p=np.where(rng.random(B) < 0.5, 0.0, rng.uniform(0.001, 0.3, B)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (5, 7), (40, 33), (64, 1000), (17, 4097),
                                 (9, 32000), (33, 50257), (3, 131072), (2, 262144), (200, 5001)])
def test_sizes_with_every_setting(dt, B, V):
    x, u = _logits(B * 7 + V, B, V, dt)
    _check(x, u, **_settings(V, B, V))
    _check(x, u)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p"])
def test_each_setting_alone(dt, name):
    x, u = _logits(3, 48, 20011, dt)
    _check(x, u, **{name: _settings(5, 48, 20011)[name]})


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_wide_restrictions(dt):
    # far more kept tokens than the short list holds
    B, V = 24, 50257
    x, u = _logits(4, B, V, dt, likely=0)
    rng = np.random.default_rng(1)
    k = rng.integers(600, 40000, B)
    p = rng.uniform(0.5, 0.9999, B)
    t = rng.uniform(0.5, 3.0, B)
    _check(x, u, top_k=k)
    _check(x, u, top_k=k, temperature=t)
    _check(x, u, top_p=p, temperature=t)
    _check(x, u, top_p=p, top_k=k, temperature=t)
    _check(x, u, top_p=p, top_k=k, temperature=t, min_p=np.full(B, 1e-3))
    _check(x, u, top_p=np.full(B, 0.3), top_k=np.full(B, V + 5))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_ties_go_to_the_lowest_index(dt):
    B, V = 12, 9001
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randint(0, 3, (B, V), generator=g, device=DEV).float()  # thousands of ties
    x[0] = 1.0
    x[1] = -torch.finfo(DT[dt]).max
    x[2, ::2] = -0.0
    x[2, 1::2] = 0.0
    x = x.to(DT[dt])
    u = torch.rand(B, generator=g, device=DEV)
    # u away from the borders of equal weights: the middle of a token's share
    for k in (1, 7, 700, 2999, 8000):
        want_n = k
        mid = ((u * want_n).floor() + 0.5) / want_n
        _check(x, mid, least=0.2, top_k=np.full(B, k))
        _check(x, mid, least=0.2, top_k=np.full(B, k), top_p=np.full(B, 0.5003))
        _check(x, mid, least=0.2, top_p=np.full(B, 0.70007))
    ids, _ = moe.sample_tokens(x, u, temperature=torch.zeros(B, device=DEV))
    top = [int((R.f64(x[b]) == R.f64(x[b]).max()).argmax()) for b in range(B)]
    assert ids.tolist() == top


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_masks_infinities_and_nan(dt):
    V = 3001
    low = torch.finfo(DT[dt]).min
    x, u = _logits(8, 10, V, dt)
    x[0] = float("-inf")                       # nothing to draw
    x[1] = float("nan")
    x[2] = float("-inf")
    x[2, 77] = -5.0                            # one token left
    x[3] = low                                 # all at the lowest value: all alike
    x[4, 100:] = low
    x[5, ::3] = float("nan")
    x[6, 9] = float("inf")
    x[6, 2000] = float("inf")                  # share the draw
    x[7, :] = float("-inf")
    x[7, 5:9] = low
    x[8, 50] = torch.finfo(DT[dt]).max
    u = torch.tensor([.5, .5, .5, .50005, .3, .7, .75, .8, .1, .9], device=DEV)
    s = _settings(9, 10, V)
    s["temperature"][:] = 0.9
    for kw in ({}, dict(top_k=s["top_k"]), dict(top_p=s["top_p"]), dict(min_p=s["min_p"]), s):
        ids = _check(x, u, least=0.3, **kw)
        assert list(ids[:3]) == [-1, -1, 77]
    ids = _check(x, u, temperature=np.zeros(10))
    assert ids[0] == ids[1] == -1 and ids[6] == 9


def test_odd_settings():
    x, u = _logits(10, 8, 5000, "f32")
    n = np.full
    ids = _check(x, u, top_p=n(8, 0.0))                      # the likeliest token
    assert list(ids) == x.argmax(1).tolist()
    assert list(_check(x, u, min_p=n(8, 1.0))) == list(ids)
    assert list(_check(x, u, min_p=n(8, 7.0))) == list(ids)
    assert list(_check(x, u, temperature=n(8, 1e-30))) == list(ids)
    assert list(_check(x, u, temperature=n(8, -1.0))) == list(ids)
    _check(x, u, temperature=n(8, 1e4), top_k=n(8, 20))      # nearly alike
    _check(x, u, temperature=n(8, 1e30))
    _check(x, u, top_k=n(8, -3), top_p=n(8, 2.0), min_p=n(8, -1.0))
    _check(x, n(8, 0.0))                                     # the first token of any weight
    last = np.nextafter(np.float32(1), np.float32(0))
    _check(x, n(8, last), least=0.0)
    a, _ = moe.sample_tokens(x, torch.full((8,), 1.5, device=DEV))  # taken as just below 1
    b, _ = moe.sample_tokens(x, torch.full((8,), float(last), device=DEV))
    assert ((a >= b) & (a < 5000)).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-6, 1e-2, 30.0, 1e4])
def test_logits_of_other_sizes(dt, scale):
    # all in one bin of the first histogram, or spread far past its last
    x, u = _logits(12, 16, 7001, dt)
    s = _settings(13, 16, 7001)
    y = (x.float() * scale).to(DT[dt])
    _check(y, u, **s)
    _check(y, u, top_k=np.full(16, 3000))
    _check(y, u, top_p=np.full(16, 0.83))
    _check(-y.abs(), u, **s)


@pytest.mark.parametrize("off", [0, 1, 3])
def test_rows_of_any_alignment_and_stride(off):
    for dt in ("f32", "bf16"):
        x, u = _logits(14, 6, 10007, dt)
        room = torch.full((6, 10007 + 9), 50.0, device=DEV).to(DT[dt])
        room[:, off:off + 10007] = x
        a, pa = moe.sample_tokens(x, u)
        b, pb = moe.sample_tokens(room[:, off:off + 10007], u)
        assert torch.equal(a, b) and torch.equal(pa, pb)
    c, _ = moe.sample_tokens(x[:1].expand(6, -1), u)  # one row for all
    assert c[0] == a[0]


def test_no_rows_and_refusals():
    x, u = _logits(15, 4, 100, "f32")
    ids, probs = moe.sample_tokens(x[:0], u[:0])
    assert ids.numel() == probs.numel() == 0
    for why, args, kw in [
            ("float32 or bfloat16", (x.half(), u), {}), ("contiguous rows", (x[0], u), {}),
            ("contiguous rows", (x.t(), u), {}), ("u must", (x, u[:3]), {}),
            ("top_k must", (x, u), dict(top_k=u)), ("top_p must", (x, u), dict(top_p=u.double())),
            ("temperature must", (x, u), dict(temperature=u[:1]))]:
        with pytest.raises(ValueError, match=why):
            moe.sample_tokens(*args, **kw)


def test_in_a_graph():
    x, u = _logits(16, 20, 30000, "f32")
    p = torch.full((20,), 0.9, device=DEV)
    moe.sample_tokens(x, u, top_p=p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, probs = moe.sample_tokens(x, u, top_p=p)
    for seed in (17, 18):
        y, v = _logits(seed, 20, 30000, "f32")
        x.copy_(y)
        u.copy_(v)
        graph.replay()
        want, wp = moe.sample_tokens(y, v, top_p=p)
        assert torch.equal(ids, want) and torch.equal(probs, wp)


@pytest.mark.parametrize("dt,spread", [("bf16", 1.8), ("f32", 0.4), ("f32", 1.8)])
def test_borders_among_many_tokens(dt, spread):
    # hundreds of tokens, equal ones with bf16, in the bin of the cut
    B, V = 10, 262144
    x, u = _logits(21, B, V, dt, spread=spread, likely=12)
    rng = np.random.default_rng(2)
    _check(x, u, least=0.7, top_p=rng.uniform(0.6, 0.99, B), temperature=rng.uniform(0.9, 3.0, B))
    _check(x, u, least=0.7, top_k=rng.integers(5000, 200000, B))


def test_a_few_allowed_tokens():
    # fewer tokens than top-k left by a mask, and every one of them kept
    x, u = _logits(22, 9, 40000, "f32")
    keep = torch.zeros(40000, dtype=torch.bool, device=DEV)
    keep[::4001] = True
    x[:, ~keep] = float("-inf")
    ids = _check(x, u, top_k=np.full(9, 500))
    assert (ids % 4001 == 0).all()
    _check(x, u, top_k=np.full(9, 50), top_p=np.full(9, 0.9))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("likely,spread", [(3, 0.5), (40, 1.8), (0, 1.0)])
def test_top_p_beside_a_sum(dt, likely, spread):
    # top_p just below and just above the share of the first m tokens, where the
    # next one is close by or far away
    B, V = 64, 40000
    x, u = _logits(23, B, V, dt, spread=spread, likely=likely)
    l = np.sort(R.f64(x), axis=1)[:, ::-1]
    w = np.exp(l - l[:, :1])
    share = (np.cumsum(w, axis=1) / w.sum(axis=1, keepdims=True)).astype(np.float32)
    rng = np.random.default_rng(3)
    m = np.minimum(np.exp(rng.uniform(0, np.log(V / 2), B)).astype(int), V - 2)
    m[:16] = np.arange(16)
    top_p = share[np.arange(B), m]
    side = np.where(rng.random(B) < 0.5, np.float32(-1), np.float32(2))
    for _ in range(2):
        top_p = np.nextafter(top_p, side).astype(np.float32)
    _check(x, u, least=0.5, top_p=np.clip(top_p, 0, 1))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("values", [(2.0,), (0.5, 0.498), (-0.25, -0.251), (0.0, -0.001, 0.002),
                                    (1.0, 0.996, 0.992, 0.988)])
def test_many_tokens_of_few_values(dt, values):
    # the border's bin holds hundreds of tokens of one or of a few values, above
    # and below zero, with others around them
    B, V = 12, 30000
    x, u = _logits(31, B, V, "f32", spread=1.0, likely=5)
    g = torch.Generator(device=DEV).manual_seed(7)
    pick = torch.randint(len(values) + 1, (B, V), generator=g, device=DEV)
    for i, v in enumerate(values):
        x[pick == i] = v
    x = x.to(DT[dt])
    rng = np.random.default_rng(4)
    _check(x, u, least=0.7, top_p=rng.uniform(0.3, 0.95, B), temperature=rng.uniform(0.7, 2.0, B))
    _check(x, u, top_k=rng.integers(200, 20000, B))
    _check(x, u, least=0.7, top_k=rng.integers(200, 20000, B), top_p=rng.uniform(0.3, 0.95, B))
