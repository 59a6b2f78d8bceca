"""Attention over blocks of values of very different sizes, of which a query attends to the small ones alone: what they keep.

Two tokens of the small block have scores near zero; every other token, those of the large block among them, is pushed
down by 100 units of log 2 at least and weighs nothing.  The tolerance goes by the tokens, not by the largest value of the row: a weight p is off by
2^-19 of itself (its score's two products and scalings, small here, its exponential, twice for numerator and denominator, and the
sums of two), and by its rounding.  In fp32 that is 2^-22 of p, or 2^-36 of the largest weight where that is more, whatever the
block.  In bf16 it is 2^-11 of p while the block's scale is at least 2^-21 of the largest, and a bit more for each power of two
below that."""
import math

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from cache_util import E4M3

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


@pytest.mark.parametrize("dtype, D, new", [(F32, 32, 1), (F32, 64, 1), (F32, 128, 1), (F32, 128, 9), (BF, 32, 1), (BF, 64, 1),
                                           (BF, 128, 1), (BF, 64, 30), (BF, 128, 30)])
@pytest.mark.parametrize("log2_ratio", [0, -8, -12, -16, -20, -21, -24, -28, -60])
@pytest.mark.parametrize("order", [0, 1])   # the small block before the large one, and behind it
@pytest.mark.parametrize("B", [1, 500])     # requests on the row: one that many CTAs share, and a CTA for several
def test_what_small_blocks_keep(dtype, D, new, log2_ratio, order, B):
    if dtype == BF and log2_ratio < -28:
        pytest.skip("bf16 holds nothing of such a block")
    H, G, page = 2, 2, 16
    P = 9                                                           # the queries see the tokens of six pages at least
    N = 6 * page + new
    g = torch.Generator(device="cuda").manual_seed(7 - log2_ratio)
    c = gdn.PagedCache.empty(1, P, H, D, 1, P, page_size=page)
    v = torch.randn(P, H, page, D, generator=g, device="cuda").mul(60).clamp(-448, 448).to(E4M3).float()
    k = torch.zeros(P, H, page, D, device="cuda")
    k[..., 3] = -208.0
    small = 1 if order == 0 else 4
    k[small, :, 2, 3], k[small, :, 11, 3] = 0.0, -1.0
    c.pages[0, :, 0], c.pages[0, :, 1] = k.to(E4M3), v.to(E4M3)
    c.scales.fill_(1.0)
    c.scales[0, :, 1] = 2.0
    c.scales[0, small, 1] = 2.0 * 2.0 ** log2_ratio
    c.table.copy_(torch.arange(P, dtype=torch.int32, device="cuda")[None])
    c.lens.fill_(N)
    q = torch.zeros(B * new, H * G, D, device="cuda")
    q[..., 3] = torch.tensor([1.0, 0.5, 2.0, 0.625], device="cuda")
    scale = float(torch.tensor(math.log(2.0)))
    r = gdn.gdn_paged_attention(q.to(dtype), c, torch.arange(0, B * new + 1, new, dtype=torch.int32, device="cuda"),
                                rows=torch.zeros(B, dtype=torch.int32, device="cuda"), max_new=new, scale=scale)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    x = torch.stack([torch.zeros(4, dtype=torch.float64, device="cuda"), -q[0, :, 3].double() * scale], -1).unflatten(0, (H, G))
    p = torch.softmax(x, -1)                                        # [H, G, 2]; of the others: 2^-100 of them at most
    top = p.amax(-1, keepdim=True)
    vs = v[small][:, [2, 11]].double() * 2.0 * 2.0 ** log2_ratio    # [H, 2, D]
    want = torch.einsum("hgk,hkd->hgd", p, vs)
    if dtype == F32:
        step = torch.maximum(p * 2.0 ** -22, top * 2.0 ** -36)
    else:
        step = torch.maximum(p * 2.0 ** -11, top * 2.0 ** (-32 - log2_ratio))
    tol = torch.einsum("hgk,hkd->hgd", torch.minimum(p, step) + p * 2.0 ** -19, vs.abs())
    if dtype == BF and log2_ratio < -21:
        # what is left of the rule for the tokens that count: a bit for each power of two below 2^-21
        assert (step <= 1.01 * top * 2.0 ** (-11 - (log2_ratio + 21))).all()
    assert (tol.amax((-1, -2)) < 0.25 * want.abs().amax((-1, -2))).all()      # the test can tell them from nothing
    tol = tol + (2.0 ** -8 if dtype == BF else U) * (want.abs() + tol)
    off = (r["o"].double().unflatten(1, (H, G)) - want).abs()
    assert (off <= tol).all(), float((off / tol).max())
