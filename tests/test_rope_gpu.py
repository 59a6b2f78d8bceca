"""Norm of the heads and rotation in one pass, on the GPU, against the formula in 64 bits.

Tolerances (u = 2^-24).  The norm's sum of D squares is off by D u at most, its root by half of that, with the root's
own 4 u and two products (D / 2 + 8) u of a value; a cosine or sine by its angle's rounding to fp32 (an eighth of a turn at
most: 0.8 u), 4 u of its own and one product, 6 u; the rotation adds two products and a sum.  So an output is off by
(|a| + |b|) mscale (D / 2 + 20) u and its own rounding."""
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


def check_one(x, y, w, pos, freq, layout, eps, mscale):
    D, rd = x.shape[-1], 0 if freq is None else 2 * len(freq)
    z = x.double()
    if eps is not None:
        z = z / torch.sqrt(z.square().mean(-1, keepdim=True) + eps) * (1 if w is None else w.double())
    want, size = z.clone(), z.abs()
    if rd:
        p = torch.arange(rd // 2, device="cuda")
        a, b = (p, p + rd // 2) if layout == "half" else (2 * p, 2 * p + 1)
        t = pos.double()[:, None, None] * freq
        c, s = torch.cos(t) * mscale, torch.sin(t) * mscale
        want[..., a], want[..., b] = z[..., a] * c - z[..., b] * s, z[..., b] * c + z[..., a] * s
        both = (z[..., a].abs() + z[..., b].abs()) * abs(mscale)
        size[..., a] = size[..., b] = both
    tol = size * (D / 2 + 20) * U
    tol = tol + (2.0 ** -8 if x.dtype == BF else U) * (want.abs() + tol) + 1e-38
    off = (y.double() - want).abs()
    assert (off <= tol).all(), float((off / tol).max())


def check(T=37, Hq=4, Hk=2, D=64, rd=None, dtype=BF, layout="half", eps=1e-6, weights=True, mscale=1.0, far=5000, seed=0, pos=None,
          **freqs):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    rd = D if rd is None else rd
    qkv = (r(T, (Hq + 2 * Hk) * D) * 3).to(dtype)
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    if pos is None:
        pos = torch.randint(-far, far, (T,), generator=g, device="cuda", dtype=torch.int32)
    f = gdn.gdn_rope_frequencies(rd, **freqs)
    qw, kw = ((1 + 0.2 * r(D)).to(dtype) if weights and eps is not None else None for _ in "qk")
    kw = kw if Hk else None
    y, z = gdn.gdn_qk_norm_rope(q, k, pos, f, layout=layout, q_weight=qw, k_weight=kw, eps=eps, mscale=mscale)
    check_one(q, y, qw, pos, f, layout, eps, mscale)
    if Hk:
        check_one(k, z, kw, pos, f, layout, eps, mscale)
    return q, k, pos, f, qw, kw, y, z


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D, rd", [(32, 0), (32, 16), (32, 32), (64, 16), (64, 48), (64, 64), (128, 0), (128, 32), (128, 80), (128, 128)])
def test_widths(dtype, layout, D, rd):
    check(D=D, rd=rd, dtype=dtype, layout=layout)
    check(D=D, rd=rd, dtype=dtype, layout=layout, eps=None, mscale=1.3, T=5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T, Hq, Hk", [(1, 1, 0), (1, 16, 2), (3, 5, 5), (67, 32, 8), (1000, 7, 1), (5000, 3, 3)])
def test_tokens_and_heads(dtype, T, Hq, Hk):
    check(T=T, Hq=Hq, Hk=Hk, D=128, dtype=dtype, seed=T)
    check(T=T, Hq=Hq, Hk=Hk, D=32, dtype=dtype, seed=T, weights=False)


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 24, 2 ** 31])
def test_far_positions(far):
    """Angles of far positions: the 64-bit formula's own angle, position times frequency, is off by 2^-53 of itself, so that
    fp32's tolerance holds up to a few million radians; beyond, the sum of angles is compared."""
    if far <= 2 ** 20:
        check(far=far, dtype=F32, D=128, eps=None)
        return
    # the rotation by a + b is that by a, then by b, in exact arithmetic; frequencies that are whole parts of a turn
    n = torch.arange(1, 33, dtype=torch.float64, device="cuda")
    f = 2 * math.pi * n / 64
    pos = torch.tensor([far - 1, -far + 5, far // 3], dtype=torch.int32, device="cuda")
    x = torch.randn(3, 2, 64, device="cuda")
    y, _ = gdn.gdn_qk_norm_rope(x, None, pos, f)
    near, _ = gdn.gdn_qk_norm_rope(x, None, torch.remainder(pos, 64).to(torch.int32), f)
    # (a frequency is off by 2^-53 of itself, half a turn at most: its angle by pos 2^-53 turns)
    assert (y - near).abs().max() <= (2 * math.pi * far * 2.0 ** -53 * 8 + 40 * U) * 2 * x.abs().max()


@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                     dict(scaling="parts", factor=16.0, original_len=2048), dict(base=500000.0)])
def test_scaled_frequencies(scaling):
    check(D=128, dtype=F32, layout="half", **scaling)


def test_in_place_and_own_outputs():
    for dtype in (BF, F32):
        q, k, pos, f, qw, kw, y, z = check(T=50, Hq=6, Hk=2, D=64, dtype=dtype)
        a, b = gdn.gdn_qk_norm_rope(q, k, pos, f, q_weight=qw, k_weight=kw, eps=1e-6, q_out=q, k_out=k)
        assert a is q and torch.equal(q, y) and torch.equal(k, z)


def test_zero_and_huge_heads():
    """A head of zeros stays zero; one whose squares leave fp32 gives zeros (its norm is infinite), and touches no other."""
    x = torch.zeros(2, 4, 64, device="cuda")
    x[0, 1] = 1e30
    x[1, 2] = 1.0
    f = gdn.gdn_rope_frequencies(64)
    y, _ = gdn.gdn_qk_norm_rope(x, None, torch.zeros(2, dtype=torch.int32, device="cuda"), f, eps=1e-6)
    assert not y[0].any() and torch.allclose(y[1, 2], torch.ones(64, device="cuda"))


def test_no_tokens_and_streams_and_graphs():
    f = gdn.gdn_rope_frequencies(64)
    e = torch.zeros(0, 4, 64, device="cuda")
    y, _ = gdn.gdn_qk_norm_rope(e, None, torch.zeros(0, dtype=torch.int32, device="cuda"), f)
    assert y.shape == (0, 4, 64)
    q, k, pos, f, qw, kw, y, z = check(T=9, Hq=4, Hk=2, D=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = gdn.gdn_qk_norm_rope(q, k, pos, f, q_weight=qw, k_weight=kw, eps=1e-6, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, y) and torch.equal(b, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = gdn.gdn_qk_norm_rope(q, k, pos, f, q_weight=qw, k_weight=kw, eps=1e-6)
    pos += 1
    graph.replay()
    torch.cuda.synchronize()
    check_one(q, a, qw, pos, f, "half", 1e-6, 1.0)
