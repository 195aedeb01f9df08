"""Decode attention where what is attended is not a finite number, or near the
types' ends: NaNs of every bit pattern that kernels leave behind, infinities,
the largest finite values, and weights far below the largest one.

Rows and columns that such a value does not reach have to be what they are
without it, bit for bit; bounds elsewhere are those of ``test_gpu_decode``."""
import numpy as np
import pytest
import torch

import decode_reference as R
import serving_moe_route_gb300 as moe
from test_gpu_decode import _case

pytestmark = pytest.mark.gpu
DEV = "cuda"
BITS = {torch.float32: torch.int32, torch.bfloat16: torch.int16, torch.float8_e4m3fn: torch.uint8}
# the quiet NaN that arithmetic on a GPU gives, its negative, the one that a
# constant has, and the smallest signalling one
NANS = {torch.float32: (0x7fffffff, -1, 0x7fc00000, 0x7f800001),
        torch.bfloat16: (0x7fff, -1, 0x7fc0, 0x7f81), torch.float8_e4m3fn: (0x7f, 0xff)}


def _at(table, page, b, t):
    return int(table[b, t // page]), t % page


def _set_bits(t, index, bits):
    t.view(BITS[t.dtype])[index] = bits


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [23, 3000])
def test_an_attended_nan_stays_one(kv, D, n):
    # heads 2 and 3 of request 1 read what is set; the long request is cut over many CTAs
    page, tok, elem = 16, 17, 5
    q, kc, vc, table, lens, sc = _case(1, 3, 4, 2, D, page, kv, [5, n, 40])
    clean, clean_lse = moe.attn_decode(q, kc, vc, table, lens, return_lse=True, **sc)
    where = (*_at(table, page, 1, tok), 1, elem)
    rest = torch.ones(3, 4, dtype=torch.bool, device=DEV)
    rest[1, 2:] = False
    for bits in NANS[kc.dtype]:
        k, v = kc.clone(), vc.clone()
        _set_bits(k, where, bits)
        out, lse = moe.attn_decode(q, k, vc, table, lens, return_lse=True, **sc)
        assert out[1, 2:].isnan().all() and lse[1, 2:].isnan().all(), f"key {bits:#x}"
        assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
        _set_bits(v, where, bits)
        out, lse = moe.attn_decode(q, kc, v, table, lens, return_lse=True, **sc)
        assert out[1, 2:, elem].isnan().all(), f"value {bits:#x}"
        out[1, 2:, elem] = clean[1, 2:, elem]
        assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    rest[1, 2] = True
    for bits in NANS[q.dtype]:
        x = q.clone()
        _set_bits(x, (1, 3, elem), bits)
        out, lse = moe.attn_decode(x, kc, vc, table, lens, return_lse=True, **sc)
        assert out[1, 3].isnan().all() and lse[1, 3].isnan(), f"query {bits:#x}"
        assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [23, 3000])
def test_attended_infinities(kv, D, n):
    page, tok, elem = 16, 17, 5
    q, kc, vc, table, lens, _ = _case(2, 3, 4, 2, D, page, kv, [5, n, 40])
    q[1, 2, elem], q[1, 3, elem] = -0.5, 0.75   # logits of an infinite key: -inf and +inf
    clean = moe.attn_decode(q, kc, vc, table, lens)
    where = (*_at(table, page, 1, tok), 1, elem)
    k, v = kc.clone(), vc.clone()
    k[where] = float("inf")
    out, lse = moe.attn_decode(q, k, vc, table, lens, return_lse=True)
    assert out[1, 3].isnan().all()              # inf - inf
    assert torch.equal(out[1, :2], clean[1, :2]) and torch.equal(out[::2], clean[::2])
    # a logit of -inf has weight 0: the row is as finite as the others
    host = [R.f64(x) for x in (q, k, vc, kc)]
    tab, ns = table.cpu().numpy(), lens.cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, want_lse, pv, _, count = R.attend(host[0], host[1], host[2], tab, ns, D ** -0.5)
    dot = R.attend(host[0], host[3], host[2], tab, ns, D ** -0.5)[3]
    f32 = kv == "f32"
    ds = dot[1, 2] * (D * 2.0 ** -23 + (3 * 2.0 ** -22 if f32 else 0.0))
    share = 2 * ds + count[1, 2] * 2.0 ** -24 + (2.0 ** -22 if f32 else 2.0 ** -16) + 2.0 ** -20
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(want[1, 2]) + share * pv[1, 2]
    assert (np.abs(R.f64(out)[1, 2] - want[1, 2]) <= tol).all()
    assert abs(float(lse[1, 2]) - want_lse[1, 2]) <= \
        ds + count[1, 2] * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * abs(want_lse[1, 2])
    v[where] = -float("inf")
    out = moe.attn_decode(q, kc, v, table, lens)
    assert not out[1, 2:, elem].isfinite().any()
    if f32:
        assert (out[1, 2:, elem] == -float("inf")).all()
    out[1, 2:, elem] = clean[1, 2:, elem]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("bits", [0x7f7fe000, 0x7f7ff000, 0x7f7ff800])
def test_values_near_the_largest(bits):
    # as long as the sums themselves stay in range.  Queries and keys below
    # 2^-114 lose the lower half of their pair: 2^-136 of the other factor
    D, page = 64, 16
    q, kc, vc, table, lens, _ = _case(3, 3, 2, 1, D, page, "f32", [1, 30, 2])
    big = torch.tensor([bits], dtype=torch.int32, device=DEV).view(torch.float32)[0]

    def check(q, k, v):
        out, lse = moe.attn_decode(q, k, v, table, lens, return_lse=True)
        host = [R.f64(x) for x in (q, k, v)]
        want, want_lse, pv, dot, n = R.attend(*host, table.cpu().numpy(), lens.cpu().numpy(),
                                              D ** -0.5)
        largest = np.nan_to_num(np.abs(host[1])).max() + np.abs(host[0]).max()
        ds = dot * (D * 2.0 ** -23 + 3 * 2.0 ** -22) + D ** 0.5 * 2.0 ** -136 * largest
        share = 2 * ds + n * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -20
        tol = 2.0 ** -24 * np.abs(want) + share[..., None] * pv + 1e-37
        assert (np.abs(R.f64(out) - want) <= tol).all()
        tol = ds + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse)
        assert (np.abs(R.f64(lse) - want_lse) <= tol).all()

    v = vc.clone()
    v[_at(table, page, 0, 0)][0, 3] = big          # the only token of its request
    check(q, kc, v)
    k, x = kc.clone(), q.clone()
    x[1] *= 1e-38
    k[_at(table, page, 1, 4)][0, 7] = -big
    check(x, k, vc)
    k, x = kc.clone(), q.clone()
    x[1, 0, 9] = big
    for t in range(30):
        k[_at(table, page, 1, t)] *= 1e-38
    check(x, k, vc)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nats", [8.0, 12.0, 17.5])
def test_many_weights_far_below_the_largest(kv, D, nats):
    # one token that takes nearly all of the softmax and has no value, as a
    # context's first one often does: the answer is what the others leave.  An
    # f16 weight's last place, half of it, is 2^-38 of the largest weight.
    # Enough requests that a CTA has whole ones, so that a warp sees them all
    B, Hq, n, page = 450, 2, 1200, 16
    q, kc, vc, table, lens, sc = _case(4, 1, Hq, 1, D, page, kv, [n])
    table, lens = table.expand(B, -1).contiguous(), lens.expand(B).contiguous()
    q = torch.zeros(B, Hq, D, dtype=q.dtype, device=DEV)
    q[:, :, 0] = 1.0
    one = {k: torch.ones_like(v) for k, v in sc.items()}
    kc.copy_(torch.zeros_like(kc, dtype=torch.float32).to(kc.dtype))
    g = torch.Generator(device=DEV).manual_seed(0)
    kc[:, :, 0, 0] = (torch.rand(kc.shape[:2], generator=g, device=DEV) - 0.5).to(kc.dtype)
    kc[_at(table, page, 0, 3)][0, 0] = torch.tensor(16.0, device=DEV).to(kc.dtype)
    vc.copy_((torch.rand(vc.shape, generator=g, device=DEV) + 0.5).to(vc.dtype))
    vc[_at(table, page, 0, 3)] = torch.zeros((), device=DEV).to(vc.dtype)
    out, lse = moe.attn_decode(q, kc, vc, table, lens, scale=nats / 16, return_lse=True, **one)
    host = [R.f64(x) for x in (q[:1], kc, vc)]
    want, want_lse, pv, dot, count = R.attend(*host, table[:1].cpu().numpy(), [n], nats / 16)
    f32 = kv == "f32"
    ds = dot * (D * 2.0 ** -23 + (3 * 2.0 ** -22 if f32 else 0.0))
    w = {"f32": 2.0 ** -22, "bf16": 2.0 ** -16, "e4m3": 2.0 ** -11}[kv]
    share = 2 * ds + count * 2.0 ** -24 + w + 2.0 ** -20
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(want) + share[..., None] * pv
    tol += n * 2.0 ** -38 * 1.5 if kv == "e4m3" else 0.0
    got = R.f64(out)
    assert (np.abs(got - want) <= tol).all(), f"{(np.abs(got - want) / tol).max():.3g} of the tolerance"
    assert (np.abs(R.f64(lse) - want_lse) <= ds + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * nats).all()


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_logits_that_are_all_minus_infinity(kv, D):
    # a softmax over -inf alone has no value, unlike one over nothing; where one
    # warp's or one CTA's tokens are -inf and others are not, they only weigh nothing
    page = 16
    q, kc, vc, table, lens, _ = _case(5, 5, 2, 1, D, page, kv, [1, 300, 0, 6000, 6000])
    q[:, :, 2] = 0.5
    for b, live in ((0, 0), (1, 0), (3, 0), (4, 9)):
        for t in range(live, int(lens[b])):
            kc[_at(table, page, b, t)][0, 2] = -float("inf")
    out, lse = moe.attn_decode(q, kc, vc, table, lens, return_lse=True)
    assert out[[0, 1, 3]].isnan().all()
    assert (out[2] == 0).all()
    assert (lse[:4] == -float("inf")).all()
    short = lens.clone()
    short[4] = 9
    few, few_lse = moe.attn_decode(q, kc, vc, table, short, return_lse=True)
    assert out[4].isfinite().all()
    torch.testing.assert_close(out[4], few[4], rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(lse[4], few_lse[4], rtol=2.0 ** -20, atol=2.0 ** -19)
