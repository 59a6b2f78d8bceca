"""Attention on a shared prefix with finite scores very far from zero, where neighbouring fp32 numbers are thousands apart: only
the largest score of a row counts, so a row is the value at its largest score, exactly, and lse is that score.

Keys and queries have one coordinate each, small whole numbers and such times a power of two: the products are exact, the largest
is at least 2^27 * 17 above the others, and the others' weights are 0.  lse takes three roundings of 2^-24 of itself (the scale, the score,
log 2) and a bf16 output none, as the value is bf16 already."""
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


@pytest.mark.parametrize("dtype, D", [(BF, 64), (BF, 128), (F32, 64)])
@pytest.mark.parametrize("B, n, Hq, Hkv, P, cap", [
    (2, 1, 4, 2, 700, 90),      # one row tile
    (5, 8, 16, 2, 700, 90),     # two
    (40, 17, 32, 4, 300, 90),   # whole requests
    (3, 1, 4, 2, 0, 90), (3, 1, 4, 2, 100, 0),
])
@pytest.mark.parametrize("log2_score", [30, 33, 40, 100])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_far_scores(dtype, D, B, n, Hq, Hkv, P, cap, log2_score, scale):
    g = torch.Generator(device="cuda").manual_seed(P + B)
    N = P + cap

    heads = torch.arange(Hkv, device="cuda")
    x = torch.randint(1, 200, (N, Hkv), generator=g, device="cuda").float()
    win = torch.randint(0, N - n if cap else N, (Hkv,), generator=g, device="cuda")   # seen by every query
    x[win, heads] = 217.0
    k = torch.zeros(N, Hkv, D, device="cuda")
    k[:, :, 3] = x * scale
    k = k.to(dtype)
    v = torch.randn(N, Hkv, D, generator=g, device="cuda").to(dtype)
    q = torch.zeros(B, n, Hq, D, device="cuda")
    q[..., 3] = 2.0 ** (log2_score - 3) * (1 + torch.arange(Hq, device="cuda") % 5)
    q = q.to(dtype)
    kt, vt = (y[None, P:].repeat(B, 1, 1, 1) if cap else None for y in (k, v))
    tl = torch.full((B,), cap, dtype=torch.int32, device="cuda") if cap else None
    r = gdn.gdn_prefix_attention(q, k[:P], v[:P], kt, vt, tl, scale=scale)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    of = torch.arange(Hq, device="cuda") // (Hq // Hkv)
    want = v[win[of], of].expand(B, n, Hq, D)
    assert torch.equal(r["o"], want)
    score = q[..., 3].double() * 217.0
    assert (score >= 2.0 ** (log2_score + 4)).all()
    assert ((r["lse"].double() - score).abs() <= 3 * 2.0 ** -24 * score).all()
