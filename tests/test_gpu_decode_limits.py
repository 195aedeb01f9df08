"""The decode-step calls at their limits: sizes that take other paths than the
usual ones, calls from several streams and threads, and what they refuse."""
import threading

import numpy as np
import pytest
import torch

import decode_reference as R
import serving_moe_route_gb300 as moe
from serving_moe_route_gb300 import _binding as B
from test_gpu_decode import KV, _case, _i32, _pool, _run_step, _word

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kv,step", [(B.MOE_KV_F32, 8), (B.MOE_KV_BF16, 8), (B.MOE_KV_E4M3, 16)])
def test_workspace_is_0_for_what_attention_refuses(kv, step):
    for dim in range(-1, 273):
        fits = 0 < dim <= 256 and dim % step == 0
        assert (B.moe_attn_workspace(kv, dim) > 0) == fits, dim
    assert moe.attn_workspace(torch.float8_e4m3fn, 72) == 0


@pytest.mark.parametrize("n", [2730, 2731, 8192])
@pytest.mark.parametrize("in_place", [False, True])
def test_step_of_many_requests(n, in_place):
    # from 2731 requests on the lengths take more shared memory than the default
    rng = np.random.default_rng(n)
    ctx, new = rng.integers(0, 70, n), rng.integers(0, 4, n)
    spare = int(sum(-(-(c + k) // 16) - -(-c // 16) for c, k in zip(ctx, new))) + 5
    table, free, pool = _pool(rng, ctx, 16, 5, spare)
    tokens = int(new.sum())
    _run_step(ctx, new, table, free, len(free), 16, pool, tokens + 7, in_place=in_place)
    _run_step(ctx, new, table, free, len(free) // 2, 16, pool, tokens - 9, in_place=in_place)


@pytest.mark.parametrize("rows,width", [(8192, 9), (3, 20001), (300, 1025)])
def test_release_of_many_and_of_wide_rows(rows, width):
    rng = np.random.default_rng(rows)
    have = rng.integers(0, width + 1, rows)
    have[-1] = width
    table, free, pool = _pool(rng, have, 1, width, 11)
    done = rng.integers(0, 2, rows)
    done[-1] = 1
    lst = np.zeros(pool, int)
    lst[:len(free)] = free
    want = R.kv_release(done, table, lst, len(free), pool)
    t, f, n, err = _i32(table), _i32(lst), _i32([len(free)]), _word()
    moe.kv_release(_i32(done), t, f, n, num_pages=pool, err=err)
    assert moe.check_word(err) == (0, 0)
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    np.testing.assert_array_equal(f.cpu().numpy(), want[1])
    assert int(n) == want[2]


def test_calls_from_several_threads_and_streams():
    # nothing but the caller's tensors is shared between two calls
    cases = [_case(s, 5, 8, 2, 128, 16, kv, [900, 3, 0, 2500, 77])
             for s, kv in ((1, "bf16"), (2, "e4m3"), (3, "f32"), (4, "bf16"))]
    g = torch.Generator(device=DEV).manual_seed(5)
    logits = [torch.randn(B_, V, generator=g, device=DEV) * 2
              for B_, V in ((1, 131072), (40, 30001), (300, 9000), (7, 50257))]
    us = [torch.rand(len(x), generator=g, device=DEV) for x in logits]
    ps = [torch.full((len(x),), 0.93, device=DEV) for x in logits]

    def work(i, stream=None):
        q, kc, vc, table, lens, sc = cases[i]
        return [moe.attn_decode(q, kc, vc, table, lens, stream=stream, **sc),
                *moe.sample_tokens(logits[i], us[i], top_p=ps[i], stream=stream)]

    want = [work(i) for i in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [work(i) for _ in range(40)]
            torch.cuda.current_stream().synchronize()
        wrong.extend(i for x in got if not all(torch.equal(a, b) for a, b in zip(x, want[i])))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [[work(i, streams[i]) for i in range(4)] for _ in range(20)]
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(a, b) for i in range(4) for a, b in zip(x[i], want[i]))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
def test_one_cta_works_off_a_long_context(kv):
    """More than two requests a CTA, so that each has whole ones: a warp adds up
    a quarter of 2^18 values of one sign in one accumulator.

    The instructions' sums are cut, 2^-23 of what they hold each: 2^16 tokens in
    2^13 steps (bf16: 16 tokens and two terms of the weights a step) come to
    2^-10.  The sum of the weights is rounded four times a tile of 16: 2^14 times
    2^-24.  The rest is as in ``test_gpu_decode``."""
    n, D, page, Hq, rows = 1 << 18, 64, 64, 2, 950
    g = torch.Generator(device=DEV).manual_seed(1)
    kc, vc = (torch.empty(n // page, page, 1, D, device=DEV).to(KV[kv]) for _ in range(2))
    kc.copy_((torch.randn(kc.shape, generator=g, device=DEV) * 0.5).to(KV[kv]))
    vc.copy_((torch.rand(vc.shape, generator=g, device=DEV) + 0.5).to(KV[kv]))
    q = torch.randn(1, Hq, D, generator=g, device=DEV)
    q = q.to(torch.float32 if kv == "f32" else torch.bfloat16)
    table = torch.randperm(n // page, generator=g, device=DEV).int()[None]  # shared by all requests
    sc = dict(k_scale=torch.ones(1, device=DEV), v_scale=torch.ones(1, device=DEV)) if kv == "e4m3" else {}
    out, lse = moe.attn_decode(q.expand(rows, -1, -1).contiguous(), kc, vc,
                               table.expand(rows, -1).contiguous(), _i32([n] * rows),
                               return_lse=True, **sc)
    want, want_lse, pv, dot, _ = R.attend(R.f64(q), R.f64(kc), R.f64(vc), table.cpu().numpy(), [n],
                                          D ** -0.5)
    f32 = kv == "f32"
    ds = dot * (D * 2.0 ** -23 + (3 * 2.0 ** -22 if f32 else 0.0))
    w = {"f32": 2.0 ** -22, "bf16": 2.0 ** -16, "e4m3": 2.0 ** -11}[kv]
    share = 2 * ds + 2.0 ** -10 + 2.0 ** -10 + w + 2.0 ** -20
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(want) + share[..., None] * pv
    assert (np.abs(R.f64(out) - want) <= tol).all()
    tol = ds + 2.0 ** -10 + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse)
    assert (np.abs(R.f64(lse) - want_lse) <= tol).all()


def _sample_like_the_definition(x, u, least=0.9, **kw):
    dev = {k: torch.as_tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device=DEV)
           for k, v in kw.items()}
    ids, probs = moe.sample_tokens(x, u, **dev)
    with np.errstate(invalid="ignore"):  # -inf over an infinite temperature
        want, p, near, off = R.sample(R.f64(x), u.cpu().numpy(), largest=torch.finfo(x.dtype).max,
                                      **{k: v.cpu().numpy() for k, v in dev.items()})
    far = near > off
    assert far.mean() >= least
    np.testing.assert_array_equal(ids.cpu().numpy()[far], want[far])
    np.testing.assert_allclose(probs.cpu().numpy()[far], p[far], rtol=4 * 2.0 ** -24)
    return int(far.sum())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_sampling_of_many_drawn_rows(dt):
    # sizes, spreads and settings drawn at random; the ids are the definition's
    rng = np.random.default_rng(11)
    g = torch.Generator(device=DEV).manual_seed(11)
    rows = 0
    for _ in range(60):
        n, V = int(np.exp(rng.uniform(0, np.log(200)))), int(np.exp(rng.uniform(0, np.log(9000))))
        x = torch.randn(n, V, generator=g, device=DEV) * float(np.exp(rng.uniform(-3, 2)))
        likely = min(V, int(rng.integers(0, 40)))
        x[:, :likely] += 6
        x = x[:, torch.randperm(V, generator=g, device=DEV)].to(dt)
        u = torch.rand(n, generator=g, device=DEV)
        every = dict(temperature=np.where(rng.random(n) < 0.1, 0.0, rng.uniform(0.2, 3.0, n)),
                     top_k=np.where(rng.random(n) < 0.4, 0, rng.integers(1, max(2, V), n)),
                     top_p=np.where(rng.random(n) < 0.4, 1.0, rng.uniform(0.01, 0.9999, n)),
                     min_p=np.where(rng.random(n) < 0.6, 0.0, rng.uniform(1e-4, 0.5, n)))
        # equal logits (bf16) make borders out of ties: fewer rows say something
        rows += _sample_like_the_definition(
            x, u, least=0.0, **{k: v for k, v in every.items() if rng.random() < 0.7})
    assert rows > 1500


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_an_infinite_temperature_makes_tokens_alike(dt):
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(20, 5003, generator=g, device=DEV).to(dt)
    x[:, ::7] = -float("inf")
    live = 5003 - len(range(0, 5003, 7))
    t = np.full(20, np.inf)
    for kept, kw in ((live, {}), (300, dict(top_k=np.full(20, 300))), (live, dict(min_p=np.full(20, 1.0))),
                     (live, dict(min_p=np.full(20, 0.3))), (300, dict(top_k=np.full(20, 300),
                                                                      top_p=np.full(20, 0.9999)))):
        u = ((torch.rand(20, generator=g, device=DEV) * kept).floor() + 0.5) / kept
        _sample_like_the_definition(x, u, least=0.5, temperature=t, **kw)


def test_step_with_more_new_pages_than_an_int_counts():
    # lengths that ask for more pages than 2^31: what lies past the table stays
    rows, width, beyond = 8192, 270000, 8
    room = torch.full((rows + beyond, width), -5, dtype=torch.int32, device=DEV)
    room[:rows] = -1
    ctx, new, err = _i32([0] * rows), _i32([width] * rows), _word()
    step = moe.kv_step(ctx, new, room[:rows], _i32(range(10)), _i32([10]), page_size=1, num_pages=10,
                       max_tokens=16, err=err)
    assert moe.check_word(err) == (B.MOE_ERR_DEVICE, R.NO_SPACE)
    assert (room[rows:] == -5).all()
    assert room[0, :10].tolist() == step.slots[:10].tolist() == list(range(9, -1, -1))
    assert step.slots[10:].tolist() == [-1] * 6 and int(step.n_free) == 0
    assert int((room[:rows] != -1).sum()) == 10
