"""Attention on caches whose rows may become very long, whatever they hold (sizes on the host, calls on the GPU)."""
import ctypes

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from cache_util import check_attention, make_cache

FAKE = 0x7f0000000000  # never dereferenced
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def scratch(dtype, Hq, H=1, D=64, page=64, W=8, rows=5000, B=1, new=1, T=None, max_len=0):
    c = gdn._Cache(1, 10, page, H, D, rows, W, FAKE, FAKE, FAKE, FAKE, FAKE)
    b = gdn._Batch(B, new, B * new if T is None else T, max_len, FAKE, None)
    return gdn.lib().gdn_paged_scratch_bytes(ctypes.byref(c), ctypes.byref(b), dtype, Hq)


@pytest.mark.parametrize("dtype", [gdn.GDN_BF16, gdn.GDN_F32])
@pytest.mark.parametrize("new", [1, 33])   # few rows; many (bf16: on the tensor cores)
def test_rows_as_long_as_the_table_allows(dtype, new):
    """One request on rows of up to 2^31 - 1024 tokens, by the bound of the call or by the table's."""
    at_2m = scratch(dtype, 4, new=new, max_len=2 ** 21 - 2 ** 12, W=2 ** 15)
    assert at_2m > 0
    for n in (2 ** 21, 2 ** 24, 2 ** 28, 2 ** 31 - 1024):
        assert scratch(dtype, 4, new=new, max_len=n, W=2 ** 25 - 16) == at_2m
        assert scratch(dtype, 4, new=new, W=n // 64) == at_2m
    assert scratch(dtype, 4, new=new, page=128, W=2 ** 24 - 8) == at_2m


@pytest.mark.parametrize("dtype, unit, tile", [(gdn.GDN_F32, 64, 32), (gdn.GDN_BF16, 128, 256)])
def test_the_limit(dtype, unit, tile):
    """Items (tiles of rows, for each request and key/value head) times units (of tokens, and four more) stay below 2^31 - 2^20: just
    below it a call is taken, from it on refused."""
    B, H, new = 64, 8, tile           # a tile a request and head
    items = B * H
    most = (2 ** 31 - 2 ** 20) // items - 4
    assert scratch(dtype, H, H=H, B=B, new=new, max_len=most * unit, W=2 ** 25 - 16) > 0
    assert scratch(dtype, H, H=H, B=B, new=new, max_len=most * unit + 1, W=2 ** 25 - 16) == 0


def test_many_heads_and_tokens_do_not_wrap():
    """Counts whose product is past 64 bits are refused."""
    assert scratch(gdn.GDN_F32, 4096, H=4096, D=32, B=4096, new=2 ** 22, T=2 ** 30 - 1, max_len=2 ** 31 - 1024, W=2 ** 25 - 16) == 0
    assert scratch(gdn.GDN_F32, 65536, H=1024, D=32, B=4096, new=2 ** 24, T=2 ** 30 - 1, max_len=2 ** 31 - 1024, W=2 ** 25 - 16) == 0


def cu_of(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, G, new", [(BF, 4, 1), (F32, 4, 1), (BF, 4, 9), (F32, 4, 9)])
@pytest.mark.parametrize("W", [2 ** 17, 2 ** 22])
def test_short_rows_of_a_wide_table(dtype, G, new, W):
    """Short rows in a table for 2^21 and 2^26 tokens, without a bound from the caller."""
    lens = [100, 33, 700]
    c = make_cache(lens, page=16, H=2, D=64, W=W)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(3 * new, 2 * G, 64, generator=g, device="cuda").to(dtype)
    check_attention(c, q, cu_of([new] * 3), max_new=new, **(dict(cut=2.0 ** -24) if dtype == BF and new * G > 16 else {}))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, new", [(BF, 1), (F32, 1), (BF, 20)])
def test_a_row_of_four_million_tokens(dtype, new):
    """A row that holds the same few pages again and again gives what a row does that holds each once: every token as often as
    every other, only more of them.  (Its sums have 2^14 times the terms; they are fp32, off by less than N u as a whole, and for
    values of both signs and parts of a few thousand terms by far less: 2^-9 of the largest value here.)"""
    D, page, few, times = 64, 128, 2, 2 ** 14
    W = few * times
    c = make_cache([page * few, 5], page=page, H=1, D=D, W=W)
    own = c.table[0, :few].clone()
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(new, 4, D, generator=g, device="cuda").to(dtype)
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    # the last query sees all tokens of both rows; the one before it, all but one of the long row's
    short = gdn.gdn_paged_attention(q[-1:], c, one, rows=one[:1], max_new=1)
    c.table[0] = own.repeat(times)
    c.lens[0] = W * page
    r = gdn.gdn_paged_attention(q, c, cu_of([new]), rows=one[:1], max_new=new)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    top = float((c.pages[0, own.long(), 1].float().abs() * c.scales[0, own.long(), 1][..., None, None]).max())
    for i in range(new):
        want = short if i == new - 1 else gdn.gdn_paged_attention(q[i:i + 1], c, one, rows=one[:1], max_new=1)
        assert (r["o"][i].float() - want["o"][0].float()).abs().max() <= 2.0 ** -9 * top + 2.0 ** -7 * want["o"].float().abs().max()
    assert (r["lse"][-1] - short["lse"][0] - 14 * 0.6931471805599453).abs().max() <= 2.0 ** -10
