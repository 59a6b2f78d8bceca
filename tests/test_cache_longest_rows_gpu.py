"""Append and growth at the end of the longest rows that a table may hold (2^31 - 1024 tokens), where a token's number and a page's
width leave 32 bits together: the same few pages stand in the table again and again, so the pool is small."""
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("new, T", [(1, 1), (1, 4000), (30, 30), (30, 4000), (300, 4000)])
def test_append_at_the_end_of_the_longest_row(dtype, page, new, T):
    """max_new is what the streams hold: room for tokens past 2^31, had the row as many new ones."""
    W = (2 ** 31 - 1024) // page
    n = 2 ** 31 - 1100
    c = gdn.PagedCache.empty(1, 64, 2, 32, 1, W, page_size=page)
    last = (n - 1) // page
    first = (n - new) // page                              # pages that the new tokens lie in: 10 .. of the pool
    c.table[0, first:last + 1] = torch.arange(10, 10 + last + 1 - first, dtype=torch.int32, device="cuda")
    c.table[0, last + 1:] = 7                              # nobody's
    c.lens.fill_(n)
    c.refs.fill_(1)
    g = torch.Generator(device="cuda").manual_seed(new)
    k, v = (torch.randn(T, 2, 32, generator=g, device="cuda").to(dtype) for _ in "kv")
    gdn.gdn_cache_append(k, v, c, ints(0, new))
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    x = c.pages[0].float() * c.scales[0][..., None, None]  # [N, 2, H, page, D]
    for i, kv in ((0, k), (1, v)):
        row = x[10:10 + last + 1 - first, i].permute(0, 2, 1, 3).flatten(0, 1)
        at = n - new - first * page
        own = row[at:at + new]
        # e4m3 of a block: half a step of the value, or of the block's smallest, 2^-10 of its scale (448 of them are not twice the largest)
        tol = 2.0 ** -4 * kv[:new].float().abs() + 2.0 ** -10 * 2 * kv[:new].float().abs().max() / 448
        assert ((own - kv[:new].float()).abs() <= tol).all()
        rest = row.clone()
        rest[at:at + new] = 0
        assert not rest.any()
    x[10:10 + last + 1 - first] = 0
    assert not x.any()


@pytest.mark.parametrize("page", [16, 128])
def test_growth_up_to_the_longest_row(page):
    W = (2 ** 31 - 1024) // page
    n = 2 ** 31 - 1100
    c = gdn.PagedCache.empty(1, 64, 1, 32, 2, W, page_size=page)
    c.lens[0] = n
    c.refs[0] = 1                                          # page 0, in every place of the row's
    assert gdn.gdn_cache_update(c, grow=ints(77, 0)).tolist() == [-1, 0] and c.lens.tolist() == [n, 0]
    assert gdn.gdn_cache_update(c, grow=ints(76, 5)).tolist() == [76, 5] and c.lens.tolist() == [n + 76, 5]
    used = -(-n // page)
    assert c.table[0, used:].tolist() == list(range(1, W - used + 1)) and int(c.table[1, 0]) == W - used + 1
    assert gdn.gdn_cache_update(c, grow=ints(1, 0)).tolist() == [-1, 0]
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
