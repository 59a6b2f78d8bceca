"""Attention for a batch that shares a long prefix on the GPU, against the definition in 64 bits.

Tolerances, from the roundings (u = 2^-24; half a step of bf16 is 2^-8).  A score x (times log2 e) is a sum of D products
and two scalings: off by at most e = (D + 4) u scale sum |q||k| + 4 u |x|; a weight by 2 e + 2^-21 of itself with its
exponential, and by 2^-8 where the weights are rounded to bf16 for the product; numerator and denominator each add N terms.
So |o - o'| <= (2 (2 e + 2^-21 + N u) + 2^-8) sum p |v|, and the output's own rounding; lse is off by 2 e + 2^-21 + N u and
its rounding."""
import math

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def make(B, n, Hq, Hkv, D, P, cap, dtype, lens, seed=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    q = r(B, n, Hq, D) * gain
    kt, vt = r(B, cap, Hkv, D), r(B, cap, Hkv, D)
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # what lies past a request's tail is whatever the buffer held
    past = torch.arange(cap, device="cuda")[None, :] >= tl.clamp(0, cap)[:, None]
    kt[past], vt[past] = float("nan"), float("inf")
    return q, r(P, Hkv, D), r(P, Hkv, D), kt, vt, tl


def check(q, kp, vp, kt, vt, tl, *, scale=None, max_tail=None, **kw):
    B, n, Hq, D = q.shape
    P, Hkv = kp.shape[:2]
    G = Hq // Hkv
    r = gdn.gdn_prefix_attention(q, kp, vp, kt, vt, tl, scale=scale, max_tail=max_tail, **kw)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    scale = D ** -0.5 if scale is None else scale
    cap = 0 if kt is None else kt.shape[1]
    lens = [0] * B if tl is None else [min(max(x, 0), cap if max_tail is None else max_tail) for x in tl.tolist()]
    rnd, out_rnd = (2.0 ** -8, 2.0 ** -8) if q.dtype == BF else (0.0, U)
    for b in range(B):
        keys = torch.cat([kp] + ([kt[b, :lens[b]]] if lens[b] else [])).double()      # [N, Hkv, D]
        vals = torch.cat([vp] + ([vt[b, :lens[b]]] if lens[b] else [])).double()
        N = len(keys)
        qs = q[b].double().reshape(n, Hkv, G, D)
        seen = P + torch.clamp(lens[b] - n + torch.arange(1, n + 1, device="cuda"), min=0)
        o, lse = r["o"][b].double().reshape(n, Hkv, G, D), r["lse"][b].double().reshape(n, Hkv, G)
        empty = seen == 0
        assert not o[empty].any() and (lse[empty] == -math.inf).all()
        live = ~empty
        if N == 0 or not live.any():
            continue
        x = torch.einsum("ihgd,khd->ihgk", qs, keys) * scale
        hide = torch.arange(N, device="cuda")[None, :] >= seen[:, None]
        x = x.masked_fill(hide[:, None, None, :], -math.inf)
        e = (D + 4) * U * abs(scale) * torch.einsum("ihgd,khd->ihgk", qs.abs(), keys.abs()).masked_fill(
            hide[:, None, None, :], 0).amax(-1) + 4 * U * x.masked_fill(hide[:, None, None, :], 0).abs().amax(-1)
        p = torch.softmax(x[live], -1)
        e = e[live]
        want = torch.einsum("ihgk,khd->ihgd", p, vals)
        mag = torch.einsum("ihgk,khd->ihgd", p, vals.abs())
        tol = (2 * (2 * e + 2.0 ** -21 + N * U) + rnd)[..., None] * mag
        bound = tol + (want.abs() + tol) * out_rnd
        err = (o[live] - want).abs()
        assert (err <= bound).all(), f"o of request {b}: {(err / bound).max().item():.3g} of the tolerance"
        wl = torch.logsumexp(x[live], -1)
        err = (lse[live] - wl).abs()
        bound = 2 * e + 2.0 ** -21 + N * U + 4 * U * wl.abs()
        assert (err <= bound).all(), f"lse of request {b}: {(err / bound).max().item():.3g} of the tolerance"
    return r


TYPES = [(BF, 128), (BF, 64), (BF, 32), (F32, 128), (F32, 64), (F32, 32)]


@pytest.mark.parametrize("dtype, D", TYPES)
@pytest.mark.parametrize("P", [0, 1, 127, 128, 129, 1000])
def test_decode(dtype, D, P):
    """One query a request, ragged tails from nothing to the whole buffer (and lengths out of its range)."""
    check(*make(8, 1, 8, 2, D, P, 140, dtype, [0, 1, 127, 128, 129, 140, 200, -3]))


@pytest.mark.parametrize("dtype, D", TYPES)
@pytest.mark.parametrize("n, Hq, Hkv", [(2, 4, 4), (5, 6, 2), (33, 8, 1), (130, 4, 2)])
def test_several_queries(dtype, D, n, Hq, Hkv):
    """The last n tokens of each tail; tails shorter than n leave the first queries the prefix alone."""
    check(*make(4, n, Hq, Hkv, D, 300, 150, dtype, [150, n, max(n - 2, 0), 0]))


@pytest.mark.parametrize("dtype, D", TYPES[:4])
@pytest.mark.parametrize("n", [3, 140])
def test_rows_that_see_nothing(dtype, D, n):
    check(*make(3, n, 4, 2, D, 0, 160, dtype, [160, 1, 0]))
    q, kp, vp, *_ = make(3, n, 4, 2, D, 0, 1, dtype, [0, 0, 0])
    r = gdn.gdn_prefix_attention(q, kp, vp)
    assert not r["o"].any() and (r["lse"] == -math.inf).all()


@pytest.mark.parametrize("dtype, D", TYPES[:4])
def test_prefix_alone(dtype, D):
    q, kp, vp, *_ = make(9, 1, 4, 1, D, 777, 1, dtype, [0] * 9)
    check(q, kp, vp, None, None, None)


@pytest.mark.parametrize("dtype, D", TYPES[:4])
def test_long_prefix(dtype, D):
    """Split over the multiprocessors and joined."""
    check(*make(3, 1, 4, 2, D, 20001, 300, dtype, [300, 7, 0]))


@pytest.mark.parametrize("dtype, D", TYPES[:4])
def test_many_rows(dtype, D):
    """Several tiles of stacked rows, the last one part full."""
    check(*make(67, 1, 10, 2, D, 513, 20, dtype, [i % 21 for i in range(67)]))


@pytest.mark.parametrize("dtype, D", TYPES[:4])
def test_peaked_and_shifted_scores(dtype, D):
    """Scores far from zero, all of one sign for some rows: only the differences to a row's maximum count."""
    q, kp, vp, kt, vt, tl = make(3, 2, 4, 2, D, 300, 50, dtype, [50, 9, 2], gain=8.0)
    kp[:, :, 0] += 40.0
    q[:, :, 0, 0] = -30.0
    q[:, :, 1, 0] = 30.0
    check(q, kp, vp, kt, vt, tl)
    check(q, kp, vp, kt, vt, tl, scale=-0.07)
    check(q, kp, vp, kt, vt, tl, scale=0.0)


@pytest.mark.parametrize("dtype, D", TYPES[:4])
def test_rising_maximum(dtype, D):
    """Keys that grow along the prefix, so that the running maximum rises at every tile."""
    q, kp, vp, kt, vt, tl = make(2, 1, 2, 2, D, 2000, 50, dtype, [50, 3])
    q = q.abs()
    kp = (kp.float().abs() * torch.linspace(0.01, 4, 2000, device="cuda")[:, None, None]).to(dtype)
    check(q, kp, vp, kt, vt, tl)


@pytest.mark.parametrize("dtype, D", TYPES[:4])
def test_strides(dtype, D):
    """Heads before tokens, slices of a fused projection and of a larger cache."""
    q, kp, vp, kt, vt, tl = make(4, 2, 8, 2, D, 261, 70, dtype, [70, 2, 31, 64])
    ref = gdn.gdn_prefix_attention(q, kp, vp, kt, vt, tl)
    qkv = torch.full((4, 2, 12, D), float("nan"), dtype=dtype, device="cuda")
    qkv[:, :, :8] = q
    cache = torch.full((2, 2, 400, D), float("nan"), dtype=dtype, device="cuda")     # [k/v, head, token, D]
    cache[0, :, 50:311], cache[1, :, 50:311] = kp.transpose(0, 1), vp.transpose(0, 1)
    tails = torch.full((2, 2, 6, 90, D), float("nan"), dtype=dtype, device="cuda")   # [k/v, head, request, token, D]
    tails[0, :, 1:5, :70], tails[1, :, 1:5, :70] = kt.permute(2, 0, 1, 3), vt.permute(2, 0, 1, 3)
    args = (qkv[:, :, :8], cache[0, :, 50:311].transpose(0, 1), cache[1, :, 50:311].transpose(0, 1),
            tails[0, :, 1:5, :70].permute(1, 2, 0, 3), tails[1, :, 1:5, :70].permute(1, 2, 0, 3), tl)
    got = gdn.gdn_prefix_attention(*args)
    assert torch.equal(got["o"], ref["o"]) and torch.equal(got["lse"], ref["lse"])
    check(*args, max_tail=64)


@pytest.mark.parametrize("dtype, D", TYPES[:4])
def test_repeats_on_another_stream_and_in_a_graph(dtype, D):
    q, kp, vp, kt, vt, tl = make(5, 1, 8, 2, D, 3001, 64, dtype, [64, 3, 0, 40, 1])
    ref = gdn.gdn_prefix_attention(q, kp, vp, kt, vt, tl)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = gdn.gdn_prefix_attention(q, kp, vp, kt, vt, tl, stream=s)
    s.synchronize()
    assert torch.equal(got["o"], ref["o"]) and torch.equal(got["lse"], ref["lse"])
    graph = torch.cuda.CUDAGraph()
    o, lse = torch.empty_like(ref["o"]), torch.empty_like(ref["lse"])
    with torch.cuda.graph(graph):
        gdn.gdn_prefix_attention(q, kp, vp, kt, vt, tl, o=o, lse=lse)
    tl -= 1   # the tails are read on the device at every replay
    graph.replay()
    want = gdn.gdn_prefix_attention(q, kp, vp, kt, vt, tl)
    assert torch.equal(o, want["o"]) and torch.equal(lse, want["lse"])
