"""Appending to a paged 8-bit cache on the GPU, bit for bit against the definition in 64 bits (every step of it is exact but
the rounding to e4m3, so there is nothing to tolerate)."""
import ctypes

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from cache_util import E4M3, NAN_BYTE, block_scale, make_cache, round_e4m3

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def define(pages, scales, table, lens, page, k, v, cu, rows):
    """The pool after the append: pages as values (64 bits), scales."""
    for b, r in enumerate(rows):
        n = cu[b + 1] - cu[b]
        if not 0 <= r < len(lens) or n == 0:
            continue
        t = max(lens[r] - n, 0)
        while t < lens[r]:
            pg, at = int(table[r][t // page]), t % page
            m = min(page - at, lens[r] - t)
            i = cu[b] + t - (lens[r] - n)
            for kv, x in ((0, k), (1, v)):
                for h in range(x.shape[1]):
                    y = x[i:i + m, h].double()
                    fine = torch.isfinite(y)
                    s = block_scale(float(y[fine].abs().max()) if fine.any() else 0.0)
                    if at > 0:   # what the block holds already: its scale stays, or its values are rounded anew
                        was = float(scales[pg, kv, h])
                        s = max(s, was)
                        pages[pg, kv, h, :at] = round_e4m3(pages[pg, kv, h, :at] * (was / s))
                    pages[pg, kv, h, at:at + m] = torch.where(fine, round_e4m3(torch.where(fine, y, 0.0) / s), torch.nan)
                    scales[pg, kv, h] = s
            t += m
    return pages, scales


def run(lens, new, *, page=16, H=2, D=32, dtype=BF, rows=None, size=1.0, seed=0, edit=None, layers=1, layer=0, max_new=None, k=None,
        check_all=True):
    c = make_cache(lens, page=page, H=H, D=D, seed=seed, poison=False, L=layers)
    at = list(range(len(lens))) if rows is None else rows
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    kv = (torch.randn(cu[-1] + 2, 2 * H, D, generator=g, device="cuda") * size).to(dtype)   # (two rows behind the last request)
    k, v = kv[:, :H], kv[:, H:]
    if edit:
        edit(k, v)
    before = c.pages.view(torch.uint8).clone()
    pages, scales = define(c.pages[layer].double().cpu(), c.scales[layer].double().cpu(), c.table.tolist(), list(lens), page,
                           k.cpu(), v.cpu(), cu, at)
    gdn.gdn_cache_append(k, v, c, ints(*cu), rows=None if rows is None else ints(*rows), layer=layer,
                         max_new=max_new or max(max(new), 1))
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    assert torch.equal(c.scales[layer].double().cpu(), scales)
    got = c.pages[layer].double().cpu()
    both = torch.isnan(got) & torch.isnan(pages)
    assert bool((torch.where(both, 0.0, got) == torch.where(both, 0.0, pages)).all())
    for other in range(layers):
        if other != layer:
            assert torch.equal(c.pages.view(torch.uint8)[other], before[other])
    return c


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_turns(dtype, page, D):
    """Ragged turns: a first token, page ends inside, whole pages, none, behind old tokens; scales that stay and that grow."""
    run([1, page, page + 1, 3 * page, 40, 7, 2 * page + 5], [1, page, 1, 2 * page + 3, 0, 7, 9], page=page, D=D, dtype=dtype)
    run([20, 33], [19, 20], page=page, D=D, dtype=dtype, size=50.0, seed=4)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H, D", [(1, 32), (3, 64), (9, 128), (16, 32)])
def test_single_tokens(dtype, H, D):
    """Decode: blocks shared by a CTA's warps, odd numbers of heads, every place in a page."""
    run([1, 2, 15, 16, 17, 32, 33, 64], [1] * 8, H=H, D=D, dtype=dtype, size=3.0)
    run([5, 18, 16, 64], [4, 8, 3, 7], H=H, D=D, dtype=dtype, size=0.01)


@pytest.mark.parametrize("size", [0.0, 1e-42, 1e-38, 1e-30, 1e-3, 447.9, 1e20, 3e38])
def test_sizes(size):
    """Scales over the whole range of fp32: the least and the largest powers of two, blocks of zeros."""
    def fill(k, v):
        k.copy_((torch.rand_like(k) * 2 - 1) * size)
        v.copy_((torch.rand_like(v) * 2 - 1) * size)
    run([3, 17, 70], [3, 2, 40], dtype=F32, edit=fill)
    run([3, 17, 70], [1, 1, 1], dtype=F32, edit=fill)


def test_edges_of_the_scale():
    """Largest values at exactly 448 times a power of two, and one step of fp32 above."""
    def fill(k, v):
        k.zero_(), v.zero_()
        k[:, :, 0], v[:, :, 0] = 448.0, torch.nextafter(torch.tensor(448.0), torch.tensor(1e3)).item()
        k[:, :, 1], v[:, :, 1] = 448 * 2.0 ** -9, 448 * 2.0 ** -10
        k[:, :, 2], v[:, :, 2] = -17.0, 2.0 ** -9 * 1.5     # ties
        k[:, :, 3], v[:, :, 3] = 19.0, 2.0 ** -10
    c = run([5], [5], dtype=F32, edit=fill)
    pg = int(c.table[0, 0])
    assert c.scales[0, pg].tolist() == [[1.0, 1.0], [2.0, 2.0]]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_and_nan(dtype):
    """They are held as NaN, and neither the scale nor any other value changes."""
    def fill(k, v):
        k[0, 0, 3], k[1, 1, 5], v[2, 0, 0] = float("inf"), float("nan"), float("-inf")
        v[3] = float("nan")   # a token without a finite value
    run([4, 20], [4, 4], dtype=dtype, edit=fill)
    run([1, 20, 4, 8], [1, 1, 1, 1], dtype=dtype, edit=fill)


def test_rows_padding_and_layers():
    run([40, 9, 30], [2, 1, 3, 2], rows=[2, -1, 0, 7], layers=3, layer=1)
    run([40, 9, 30], [20, 11, 30], rows=[2, 2 ** 31 - 1, 0], layers=2, layer=1)


def test_more_new_tokens_than_the_row_has():
    """Only a row's own positions are written: the first new tokens of a row that counts fewer are passed over."""
    run([3, 0, 17], [5, 4, 17])
    run([3, 0, 40], [20, 14, 40])


def test_values_do_not_depend_on_the_cut():
    """One call of 50 tokens and 50 calls of one token leave the same values (all larger than 2^-14 of their block's)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    size = torch.exp2(torch.arange(50, device="cuda") % 7 - 3.0)[:, None, None]
    x = torch.randn(50, 2, 64, generator=g, device="cuda")
    k, v = ((x + torch.sign(x) * 0.01) * size).to(BF), ((x + torch.sign(x) * 0.01) * size.flip(0)).to(BF)
    caches = [make_cache([50], page=16, H=2, D=64, poison=False) for _ in range(2)]
    gdn.gdn_cache_append(k, v, caches[0], ints(0, 50))
    for i in range(50):
        caches[1].lens[0] = i + 1
        gdn.gdn_cache_append(k[i:i + 1], v[i:i + 1], caches[1], ints(0, 1))
    pg = caches[0].table[0, :4].long()
    a, b = (c.pages[0].float()[pg] * c.scales[0][pg][..., None, None] for c in caches)
    assert torch.equal(a[:3], b[:3]) and torch.equal(a[3, :, :, :2], b[3, :, :, :2])


def test_bad_pages_and_counts_are_reported():
    c = make_cache([40, 50], page=16, H=2, D=32, poison=False)
    before = c.pages.view(torch.uint8).clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x = torch.ones(8, 2, 32, device="cuda")
    for bad in (-1, 2 ** 31 - 1, c.pages.shape[1]):
        c.table[0, 2] = bad
        gdn.gdn_cache_append(x, x, c, ints(0, 1), ws=ws, max_new=1)
        assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
        gdn.clear_status(ws=ws)
    gdn.gdn_cache_append(x, x, c, ints(0, 1, 8), ws=ws, max_new=3)
    assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
    assert torch.equal(c.pages.view(torch.uint8), before)


def test_rows_longer_than_the_table_and_bounds_for_attention():
    """A row past what the table holds is reported and nothing of it written; max_len, attention's bound, moves no tokens."""
    c = make_cache([40, 50], page=16, H=2, D=32, W=4, poison=False)
    before = c.pages.view(torch.uint8).clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x = torch.ones(2, 2, 32, device="cuda")
    c.lens[1] = 65
    gdn.gdn_cache_append(x[:1], x[:1], c, ints(0, 0, 1), ws=ws)
    assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
    assert torch.equal(c.pages.view(torch.uint8), before)
    gdn.clear_status(ws=ws)
    c.lens[1] = 50
    cu = ints(0, 1, 2)
    b = gdn._batch(c, 2, cu, None, 1, 5)
    gdn._call("gdn_cache_append", c.device, ctypes.byref(c._c), 0, ctypes.byref(b), x.data_ptr(), x.data_ptr(), gdn._dtype_code(x.dtype),
              0, 0, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert gdn.read_status(ws=ws) == gdn.GDN_OK
    other = make_cache([40, 50], page=16, H=2, D=32, W=4, poison=False)
    gdn.gdn_cache_append(x, x, other, cu)
    assert torch.equal(c.pages.view(torch.uint8), other.pages.view(torch.uint8)) and torch.equal(c.scales, other.scales)


def test_captured_and_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(2, 2, 32, generator=g, device="cuda").to(BF)
    a, b, c = (make_cache([20, 31], page=16, H=2, D=32, poison=False) for _ in range(3))
    gdn.gdn_cache_append(x, x, a, ints(0, 1, 2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cu = ints(0, 1, 2)
    torch.cuda.synchronize()
    gdn.gdn_cache_append(x, x, b, cu, stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_cache_append(x, x, c, cu)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.pages.view(torch.uint8), b.pages.view(torch.uint8)) and torch.equal(a.scales, b.scales)
    assert torch.equal(a.pages.view(torch.uint8), c.pages.view(torch.uint8)) and torch.equal(a.scales, c.scales)
    # the next replay goes where the lengths point then
    for cache in (a, c):
        cache.lens.add_(1)
    gdn.gdn_cache_append(x, x, a, cu)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.pages.view(torch.uint8), c.pages.view(torch.uint8)) and torch.equal(a.scales, c.scales)
