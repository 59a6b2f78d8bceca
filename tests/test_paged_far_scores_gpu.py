"""Attention over a paged cache with finite scores far from zero, where neighbouring fp32 numbers are whole steps apart and later
tokens lie a few of them above the first.

Every score is exact.  In units of log 2 it is a whole number: the base 2^e, which all tokens share, and the token's own count of
steps of fp32 there (16 at most).  Queries and keys are powers of two and small whole numbers, so the products and their sums are
exact in 24 bits, and so are the differences of scores, on which alone the weights depend.  The softmax scale is log 2 rounded to
fp32, 2^-27 off: that is 2^-27 of a difference, below 2^-17 for weights that count.  What is left are a weight's exponential
(2^-21), the same of the sums they belong to, its rounding (half a step: 2^-11 in f16, 2^-22 in two; 2^-32 of the largest at least),
N sums and the output's rounding; for lse the scale's 2^-27 of the score, three roundings, and the sum's errors."""
import math

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from cache_util import E4M3

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
LOG2 = float(torch.tensor(math.log(2.0)))   # in fp32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def cache_of(k, v, page):
    """One row of whole numbers, scales 1."""
    N, H, D = k.shape
    P = -(-N // page)
    c = gdn.PagedCache.empty(1, P, H, D, 1, P, page_size=page)
    x = torch.zeros(2, P * page, H, D, device="cuda")
    x[0, :N], x[1, :N] = k, v
    c.pages.copy_(x.unflatten(1, (P, page)).permute(1, 0, 3, 2, 4)[None].to(E4M3))
    c.scales.fill_(1.0)
    c.table.copy_(torch.arange(P, dtype=torch.int32, device="cuda")[None])
    c.lens.fill_(N)
    c.refs.fill_(1)
    return c


def steps_of(kind, N, H, most, g):
    """How many steps above the base each token's score lies."""
    x = torch.randint(0, 2, (N, H), generator=g, device="cuda")
    if kind == "rises":            # by one or two steps at a time, early and late
        x += torch.arange(N, device="cuda")[:, None] * (most - 1) // N
    elif kind == "jumps":          # once, in the middle, by all of them
        x[N // 2:] += most - 1
    else:                          # at the last tokens alone
        x[-3:] = most
    return x


# (fp32 queries: any number of rows; bf16: 8 by warp-level products, 40 and 300 on the tensor cores)
@pytest.mark.parametrize("dtype, D, new, G", [(BF, 64, 2, 4), (BF, 128, 2, 4), (BF, 64, 10, 4), (BF, 128, 10, 4), (BF, 128, 75, 4),
                                              (F32, 64, 2, 4), (F32, 128, 10, 4), (BF, 32, 10, 4)])
@pytest.mark.parametrize("e", [12, 20, 21, 22, 23, 24, 25, 26, 27, 28, 30])
@pytest.mark.parametrize("kind", ["rises", "jumps", "late"])
@pytest.mark.parametrize("sign, side", [(1, 1), (-1, 1), (1, -1)])   # of the queries and the scale; of the base
def test_steps_above_the_first(dtype, D, new, G, e, kind, sign, side):
    g = torch.Generator(device="cuda").manual_seed(e)
    N, H, page = 400, 2, 16
    step = max(1.0, 2.0 ** (e - 23))
    for most in (2, 3, 5, 9, 16):
        for odd in (0, 1):         # the base's own last bit: which way a tie goes
            at = steps_of(kind, N, H, most, g)
            k = torch.zeros(N, H, D, device="cuda")
            k[..., 5], k[..., 17], k[..., 30] = 16.0 * side, at.float(), float(odd)
            v = torch.randn(N, H, D, generator=g, device="cuda").to(E4M3).float()
            q = torch.zeros(new, H * G, D, device="cuda")
            q[..., 5], q[..., 17], q[..., 30] = 2.0 ** (e - 4), step, step
            c = cache_of(k, v, page)
            r = gdn.gdn_paged_attention((q * sign).to(dtype), c, torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                                        scale=LOG2 * sign)
            torch.cuda.synchronize()
            assert gdn.read_status("cuda") == gdn.GDN_OK
            score = at.double() * step                                  # above the base, in units of log 2
            seen = torch.arange(N, device="cuda")[None] <= N - new + torch.arange(new, device="cuda")[:, None]
            x = torch.where(seen[..., None], score[None] * math.log(2.0), -math.inf)   # [new, N, H]
            p = torch.softmax(x, 1)
            want = torch.einsum("inh,nhd->ihd", p, v.double())
            size = torch.einsum("inh,nhd->ihd", p, v.double().abs())
            rel = 2 * (2.0 ** -21 + N * U + 2.0 ** -17) + (2.0 ** -11 if dtype == BF else 2.0 ** -22)
            tol = rel * size + N * 2.0 ** -32 * v.abs().max()
            tol = tol + (2.0 ** -8 if dtype == BF else U) * (want.abs() + tol)
            o = r["o"].double().unflatten(1, (H, G))
            off = (o - want[:, :, None]).abs()
            where = (most, odd)
            assert torch.isfinite(o).all(), where
            assert (off <= tol[:, :, None]).all(), (where, float((off / tol[:, :, None]).max()))
            base = (side * 2.0 ** e + odd * step) * math.log(2.0)
            lse = base + torch.logsumexp(x, 1)[..., None]
            off = (r["lse"].double().unflatten(1, (H, G)) - lse).abs()
            assert (off <= (2.0 ** -27 + 3 * U) * lse.abs() + 2.0 ** -17 + N * U).all(), (where, "lse")


@pytest.mark.parametrize("dtype, new", [(BF, 2), (BF, 10), (F32, 2)])
@pytest.mark.parametrize("e", [22, 23, 24, 26, 29])
def test_scores_around_zero_and_far(dtype, new, e):
    """A row's maximum far below zero, then near it, then far above: only the largest score of a row counts."""
    N, H, D, G = 300, 1, 64, 4
    k = torch.zeros(N, H, D, device="cuda")
    k[:100, :, 5], k[100:200, :, 5], k[200:, :, 5] = -16.0, 0.0, 15.0
    k[280, 0, 5] = 16.0
    v = torch.randn(N, H, D, generator=torch.Generator(device="cuda").manual_seed(e), device="cuda").to(E4M3).float()
    q = torch.zeros(new, H * G, D, device="cuda")
    q[..., 5] = 2.0 ** (e - 4)
    c = cache_of(k, v, 16)
    r = gdn.gdn_paged_attention(q.to(dtype), c, torch.tensor([0, new], dtype=torch.int32, device="cuda"), scale=LOG2)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    assert torch.equal(r["o"].float(), v[280, 0].expand(new, H * G, D))
    ref = 2.0 ** e * math.log(2.0)
    assert ((r["lse"].double() - ref).abs() <= (2.0 ** -27 + 3 * U) * ref).all()
