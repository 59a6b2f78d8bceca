"""Rotation at far positions against angles worked out in whole numbers.

The angle is position * inv_freq, inv_freq as given, without rounding: 2 pi and the frequency are held here as fractions of more
than 130 bits.  The kernel's fraction of a turn has 64 bits, 2^-64 off with the rounding of its second part, so the angle
is off by |position| 2^-64 turns; what is left of the turn goes to fp32 and its sine and cosine are off by 4 u of themselves
(u = 2^-24).  The heads are (1, 0) pairs, so that an output is a cosine or a sine by itself; those near a whole turn are
where an angle's error shows."""
import math
from fractions import Fraction

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
BITS = 140


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def exact_angles(pos, freq):
    """position * frequency less whole turns, in -pi .. pi."""
    out = []
    for f in freq:
        turn = Fraction(f) / (2 * PI)
        whole = round(turn * 2 ** BITS)                              # (off by 2^-140: 2^-108 at the farthest position)
        for p in pos:
            a = p * whole % 2 ** BITS
            out.append((a - 2 ** BITS if a >= 2 ** (BITS - 1) else a) / 2 ** BITS * 2 * math.pi)
    return torch.tensor(out, dtype=torch.float64).reshape(len(freq), len(pos)).T


def rotate(pos, freq):
    D = 2 * len(freq)
    x = torch.zeros(len(pos), 1, D, device="cuda")
    x[..., :D // 2] = 1.0
    y, _ = gdn.gdn_qk_norm_rope(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                                torch.tensor(freq, dtype=torch.float64, device="cuda"))
    torch.cuda.synchronize()
    return y[:, 0, :D // 2].double().cpu(), y[:, 0, D // 2:].double().cpu()


def check(pos, freq):
    t = exact_angles(pos, freq)
    c, s = rotate(pos, freq)
    far = torch.tensor(pos, dtype=torch.float64).abs()[:, None] * 2.0 ** -64 * 2 * math.pi
    for got, want in ((c, torch.cos(t)), (s, torch.sin(t))):
        off = (got - want).abs()
        tol = 4 * U * want.abs() + far + 1e-15
        assert (off <= tol).all(), (float((off / tol).max()), [pos[i] for i in (off > tol).any(1).nonzero()[:3, 0]])
    return t


MODEL = [10000.0 ** (-i / 32) for i in range(32)]
# near and far from a whole number of turns a token; negative ones; ones above a turn a token; tiny ones, of either sign
ODD = [1.0, -1.0, 3.0, -3.0, math.pi * (1 - 2.0 ** -52), 0.1, -0.1, 6.2, 7.0, 40.0, -40.0, 1e-3, -1e-3, 1e-9, -1e-9, 1e-20, -1e-20,
       2.0 ** -40, -2.0 ** -60, 0.0, 1 / 3, 2 / 3, 5 / 7, -5 / 7, 0.7, 0.9, 1.1, 1.3, 1.7, 2.3, 2.9, 3.1]


@pytest.mark.parametrize("freq", [MODEL, ODD], ids=["model", "odd"])
@pytest.mark.parametrize("far", [2 ** 20, 2 ** 24, 2 ** 28, 2 ** 31])
def test_far_positions(freq, far):
    pos = [far - 1 - 7 * i for i in range(1200)] + [-far + 11 * i for i in range(1200)] + [0, 1, -1]
    t = check(pos, freq)
    assert (torch.sin(t).abs() < 2.0 ** -7).any(0).sum() >= 10        # there are angles near a whole turn for many frequencies


def test_every_position_of_a_long_context():
    check(list(range(0, 131072, 97)), MODEL)
