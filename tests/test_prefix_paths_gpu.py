"""The plans of the tensor-core attention on a shared prefix, one by one, against the definition in 64 bits (tolerances:
test_prefix_attention_gpu.py).  Which plan a call takes shows in the scratch that it asks for: none where an item writes its rows
itself, else one set of partial sums for each range of the prefix and of the tails."""
import ctypes

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from test_prefix_attention_gpu import check, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def parts(q, kp, cap):
    """Ranges that the call's prefix and tails are cut into; 0: its items write their rows themselves."""
    B, n, Hq, D = q.shape
    P, Hkv = kp.shape[:2]
    pr = gdn._PrefixProblem(B, n, Hq, Hkv, D, gdn.GDN_BF16, P, cap, cap, 1.0)
    groups = -(-B * n * (Hq // Hkv) // 32)
    total = gdn.lib().gdn_prefix_scratch_bytes(ctypes.byref(pr))
    one = Hkv * groups * 32 * (8 + 4 * D)
    assert total % one == 0
    return total // one


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [0, 1, 129, 300])
def test_whole_requests(D, P):
    """Requests with row tiles of their own that fill the GPU: prefix and tail in one go, the last row tile with 8 rows alone.
    Tails that are empty, shorter than the queries, out of range, full, and ending inside a tile."""
    q, kp, vp, kt, vt, tl = make(40, 33, 32, 4, D, P, 150, BF, [(0, 150, 20, 33, 200, -3, 128, 129, 1, 32)[i % 10] for i in range(40)])
    assert parts(q, kp, 150) == 0
    check(q, kp, vp, kt, vt, tl)


@pytest.mark.parametrize("D", [64, 128])
def test_whole_requests_without_tails(D):
    q, kp, vp, *_ = make(20, 40, 32, 4, D, 300, 1, BF, [0] * 20)
    assert parts(q, kp, 0) == 0
    check(q, kp, vp, None, None, None)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B, n, Hq, Hkv", [(3, 2, 4, 2), (9, 1, 8, 1), (30, 5, 8, 2)])   # 12, 72 and 600 stacked rows
@pytest.mark.parametrize("P", [1, 100, 128])
def test_prefix_of_one_part(D, B, n, Hq, Hkv, P):
    """One range in all: the stacked rows' items write the results."""
    q, kp, vp, *_ = make(B, n, Hq, Hkv, D, P, 1, BF, [0] * B)
    assert parts(q, kp, 0) == 0
    check(q, kp, vp, None, None, None)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_tails_of_one_part(D, n):
    """No prefix and short tails, some of them empty: rows that see nothing are written by the item as well."""
    q, kp, vp, kt, vt, tl = make(7, n, 8, 2, D, 0, 120, BF, [0, 1, 2, 3, 64, 119, 120])
    assert parts(q, kp, 120) == 0
    check(q, kp, vp, kt, vt, tl)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B, n, Hq, Hkv, P, ranges", [
    (700, 1, 4, 2, 0, 0),       # 1400 items of one row tile, written directly
    (128, 1, 16, 16, 100, 2),   # 2064 of one row tile, joined
    (700, 1, 4, 2, 100, 2),     # 1412 of two row tiles, most of which use one, in turn
    (400, 33, 8, 2, 0, 0),      # 800 of two row tiles, one full and one with 4 rows
])
def test_items_taken_over(D, B, n, Hq, Hkv, P, ranges):
    """Many times as many items as run at once, of mixed lengths, none among them: every CTA takes several."""
    q, kp, vp, kt, vt, tl = make(B, n, Hq, Hkv, D, P, 120, BF, [(0, 120, 1, 60, n, 119, 5)[i * i % 7] for i in range(B)])
    got = parts(q, kp, 120)
    assert got == ranges
    check(q, kp, vp, kt, vt, tl)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B, n, Hq, Hkv, P, tiles", [
    (2, 8, 128, 16, 40000, 8),   # 128 stacked rows: one row tile, 16 heads
    (4, 8, 64, 8, 40000, 8),     # 256: two
    (20, 34, 32, 4, 4000, 0),    # whole requests
])
def test_rising_maximum_in_long_items(D, B, n, Hq, Hkv, P, tiles):
    """Keys that grow along the prefix, so that an item's running maximum rises by more than 2^8 many times and the sums so far
    are rescaled."""
    q, kp, vp, kt, vt, tl = make(B, n, Hq, Hkv, D, P, 50, BF, [(50, 3, 0, 40)[i % 4] for i in range(B)], gain=16.0)
    got = parts(q, kp, 50)
    assert got == 0 if tiles == 0 else -(-P // 128) >= tiles * (got - 1)   # tiles of a range of the prefix
    q = q.abs()
    kp = (kp.float().abs() * torch.linspace(0.01, 4, P, device="cuda")[:, None, None]).to(BF)
    check(q, kp, vp, kt, vt, tl)
    check(q, kp.flip(0), vp, kt, vt, tl)   # and one that never rises
