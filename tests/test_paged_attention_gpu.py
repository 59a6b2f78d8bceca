"""Attention over a paged 8-bit cache on the GPU, against the definition in 64 bits (tolerances: tests/cache_util.py)."""
import math

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from cache_util import E4M3, NAN_BYTE, check_attention, make_cache

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return ints(*out)


TC = dict(cut=2.0 ** -24)


def step_of(dtype, D, rows):
    """The tensor cores take many rows of bf16."""
    return TC if dtype == BF and D >= 64 and rows > 16 else {}


def queries(T, Hq, D, dtype, seed=1, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, Hq, D, generator=g, device="cuda") * gain).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode(dtype, D, page):
    """One token a request: lengths from one token on, page ends, a length that leaves one token in its last page."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 129, 400, 1000, 2049]
    c = make_cache(lens, page=page, H=2, D=D, seed=D + page)
    q = queries(len(lens), 8, D, dtype)
    check_attention(c, q, cu_of([1] * len(lens)), max_new=1)
    check_attention(c, q, cu_of([1] * len(lens)), max_new=1, max_len=2049)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H, G", [(1, 1), (3, 3), (2, 5), (1, 16), (1, 17), (2, 40), (1, 128)])
def test_head_groups(dtype, H, G):
    c = make_cache([5, 333, 70], page=32, H=H, D=64, seed=G)
    check_attention(c, queries(3, H * G, 64, dtype), cu_of([1, 1, 1]), max_new=1, **step_of(dtype, 64, G))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_several_queries(dtype, D, G):
    """Drafts and turns: ragged numbers of queries, none, more than the row has tokens (which see nothing), whole prompts."""
    lens, new = [100, 40, 7, 300, 64, 33, 0, 1], [4, 0, 9, 33, 64, 33, 2, 1]
    c = make_cache(lens, page=16, H=2, D=D, seed=G)
    check_attention(c, queries(sum(new), 2 * G, D, dtype), cu_of(new), max_new=64, **step_of(dtype, D, 64 * G))
    check_attention(c, queries(sum(new), 2 * G, D, dtype), cu_of(new), **step_of(dtype, D, 64 * G))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_the_table(dtype):
    """A batch is some of the rows, in any order; padding rows give zeros; a row may be attended twice."""
    c = make_cache([10, 200, 31, 90], page=16, H=2, D=64)
    rows = ints(3, -1, 1, 4, 0, 1, 2 ** 31 - 1, -2 ** 31)
    new = [1, 1, 3, 2, 1, 1, 1, 1]
    check_attention(c, queries(sum(new), 4, 64, dtype), cu_of(new), rows=rows, max_new=3)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_queries_and_own_outputs(dtype):
    """q as a slice of one projection's output; rows of o and lse behind the last request are left as they were."""
    c = make_cache([50, 77], page=16, H=2, D=64)
    qkv = queries(9, 12, 64, dtype)
    q = qkv[:, 2:10]
    o, lse = torch.full((9, 8, 64), 7.0, dtype=dtype, device="cuda"), torch.full((9, 8), 7.0, device="cuda")
    check_attention(c, q, ints(0, 2, 5), max_new=3, o=o, lse=lse)
    assert (o[5:] == 7).all() and (lse[5:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gain", [1e-30, 1e-3, 30.0, 1e4, -1.0])
def test_sizes_of_queries_and_scales(dtype, gain):
    """Queries far from one and a negative scale: the rows' powers of two."""
    c = make_cache([300, 41], page=16, H=2, D=64)
    q = queries(2, 4, 64, dtype, gain=abs(gain))
    check_attention(c, q, ints(0, 1, 2), scale=0.1 / abs(gain) * math.copysign(1, gain))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_blocks_of_very_different_sizes(dtype):
    """Blocks whose values differ by 2^24: a query that attends to the small ones alone keeps their precision."""
    c = make_cache([256], page=16, H=1, D=64, poison=False, spread=1)
    big = c.table[0, ::2].long()
    c.scales[0, big, 1] *= 2.0 ** 12
    c.scales[0, c.table[0, 1::2].long(), 1] *= 2.0 ** -12
    c.scales[0, big, 0] = 2.0 ** -9
    q = queries(3, 2, 64, dtype, gain=2.0)
    check_attention(c, q, ints(0, 3))
    # keys of the large blocks pushed far down: the row's own scale of values decides, not the largest block's
    kb = c.pages.view(torch.uint8)
    kb[0, big, 0] = 0x80 | 0x78   # -256
    c.scales[0, big, 0] = 2.0 ** -2
    q = queries(1, 2, 64, dtype).abs() + 0.5
    check_attention(c, q.to(dtype), ints(0, 1))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_that_rise_late(dtype):
    """The maximum rises by little, by much and at the last token: weights are rescaled."""
    for step in (0.5, 3.0, 100.0):
        c = make_cache([700], page=16, H=1, D=32, poison=False, spread=1)
        kb = c.pages.view(torch.uint8)
        w = torch.arange(44, device="cuda")
        kb[0, c.table[0, :44].long(), 0] = 0x38                       # every key element 1 ..
        c.scales[0, c.table[0, :44].long(), 0, 0] = (w + 1).float() * step / 44   # .. times a rising scale
        q = torch.full((1, 2, 32), 0.25, device="cuda", dtype=dtype)
        check_attention(c, q, ints(0, 1), scale=1.0)


def test_zero_values_and_zero_queries():
    c = make_cache([40], page=16, H=1, D=64, poison=False)
    c.pages.view(torch.uint8)[:, :, 1] = 0
    c.scales[:, :, 1] = 2.0 ** -126
    r = check_attention(c, queries(2, 4, 64, BF), ints(0, 2))
    assert not r["o"].any()
    check_attention(make_cache([40], page=16, H=1, D=64), torch.zeros(2, 4, 64, dtype=BF, device="cuda"), ints(0, 2))


def test_a_nan_stays_within_its_request():
    c = make_cache([40, 50], page=16, H=2, D=64)
    c.pages.view(torch.uint8)[0, c.table[0, 1], 0, 1, 3] = NAN_BYTE
    q = queries(2, 4, 64, BF)
    r = gdn.gdn_paged_attention(q, c, ints(0, 1, 2))
    assert torch.isnan(r["o"][0, 2:]).all() and torch.isfinite(r["o"][0, :2]).all() and torch.isfinite(r["o"][1]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_requests_few_units(dtype):
    """More requests than threads look through at once, many of them without tokens or queries."""
    lens = [(7 * i) % 90 if i % 3 else 0 for i in range(700)]
    new = [i % 3 for i in range(700)]
    c = make_cache(lens, page=16, H=1, D=32)
    check_attention(c, queries(sum(new), 2, 32, dtype), cu_of(new), max_new=2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_long_row(dtype):
    """A single long row is cut over the whole GPU: parts of many CTAs are joined."""
    c = make_cache([50003], page=64, H=2, D=128)
    check_attention(c, queries(3, 8, 128, dtype), ints(0, 3), max_new=3)
    check_attention(c, queries(1, 2, 128, dtype), ints(0, 1), max_new=1)


def test_layers_and_pages_past_32_bits():
    """Pages behind the first 2^32 bytes of the pool, and a layer behind the first."""
    H, page, D, N = 8, 128, 128, 9000
    c = gdn.PagedCache.empty(2, N, H, D, 1, 4, page_size=page)   # 2.4 GB a layer
    g = torch.Generator(device="cuda").manual_seed(3)
    c.table[0, :2] = ints(N - 1, N - 2)
    c.lens[0] = 200
    c.pages.view(torch.uint8)[1, N - 2:] = (torch.randn(2, 2, H, page, D, generator=g, device="cuda") * 60).clamp(-448, 448).to(
        E4M3).view(torch.uint8)
    c.scales[1, N - 2:] = 2.0 ** -6
    check_attention(c, queries(1, 16, D, BF), ints(0, 1), layer=1)
    assert not gdn.gdn_paged_attention(queries(1, 16, D, BF), c, ints(0, 1), layer=0)["o"].any()


def test_bad_pages_and_counts_are_reported():
    """A page number outside the pool, and a request with more new tokens than the bound, are reported and followed nowhere."""
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        c = make_cache([40, 50], page=16, H=2, D=64)
        want = gdn.gdn_paged_attention(queries(2, 4, 64, BF), c, ints(0, 1, 2))["o"]
        c.table[0, 1] = bad
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        r = gdn.gdn_paged_attention(queries(2, 4, 64, BF), c, ints(0, 1, 2), ws=ws)
        assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
        assert torch.equal(r["o"][1], want[1])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    gdn.gdn_paged_attention(queries(9, 4, 64, BF), make_cache([40, 50], page=16, H=2, D=64), ints(0, 7, 9), max_new=3, ws=ws)
    assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
    gdn.clear_status(ws=ws)
    assert gdn.read_status(ws=ws) == gdn.GDN_OK


@pytest.mark.parametrize("dtype, G", [(BF, 2), (BF, 40), (F32, 2)])
def test_lengths_past_their_bound_are_reported(dtype, G):
    """A row longer than max_len, a loop replayed for too long for instance, is reported; the others keep their results."""
    c = make_cache([40, 50], page=16, H=2, D=64)
    q, cu = queries(2, 2 * G, 64, dtype), ints(0, 1, 2)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = gdn.gdn_paged_attention(q, c, cu, max_len=50, ws=ws)["o"]
    assert gdn.read_status(ws=ws) == gdn.GDN_OK
    r = gdn.gdn_paged_attention(q, c, cu, max_len=49, ws=ws)
    assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
    torch.testing.assert_close(r["o"][0], want[0], rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.parametrize("dtype, W", [(BF, 2 ** 14), (F32, 2 ** 13)])
def test_counts_that_fall_are_reported(dtype, W):
    """cu_new that falls again and again: more queries than the streams hold, past what 31 bits count; nothing is done."""
    B, new, page = 4096, 4096, 128
    c = gdn.PagedCache.empty(1, 1, 8, 64, 1, W, page_size=page)
    c.lens.fill_(W * page)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = new
    q = torch.zeros(new, 8, 64, dtype=dtype, device="cuda")
    o = torch.full_like(q, 7.0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    gdn.gdn_paged_attention(q, c, cu, rows=torch.zeros(B, dtype=torch.int32, device="cuda"), max_new=new, o=o, ws=ws)
    assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
    assert (o == 7).all()


@pytest.mark.parametrize("dtype, G, new", [(BF, 4, 1), (BF, 16, 20), (F32, 4, 2)])
def test_captured_and_on_another_stream(dtype, G, new):
    """A captured call follows lengths, tables and counts that change between replays; two calls on two streams at once."""
    lens = [120, 500, 64]
    c = make_cache(lens, page=16, H=2, D=64, poison=False)
    q, cu = queries(3 * new, 2 * G, 64, dtype), cu_of([new] * 3)
    want = gdn.gdn_paged_attention(q, c, cu, max_new=new)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = (gdn.gdn_paged_attention(q, c, cu, max_new=new, stream=x) for x in (s, None))
    torch.cuda.synchronize()
    assert torch.equal(a["o"], want["o"]) and torch.equal(b["o"], want["o"]) and torch.equal(a["lse"], want["lse"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = gdn.gdn_paged_attention(q, c, cu, max_new=new)
    for again in ([30, 499, 64], [500, 120, 1]):
        c.lens.copy_(ints(*again))
        rows = c.table.clone()
        if again[0] == 500:
            c.table.copy_(rows[[1, 0, 2]])
        graph.replay()
        torch.cuda.synchronize()
        eager = check_attention(c, q, cu, max_new=new, **step_of(dtype, 64, new * G))
        assert torch.equal(r["o"], eager["o"]) and torch.equal(r["lse"], eager["lse"])
        c.table.copy_(rows)


def test_results_do_not_change():
    """The same call gives the same bits, every time."""
    c = make_cache([5000, 333, 1200], page=64, H=2, D=128)
    q = queries(30, 8, 128, BF)
    first = gdn.gdn_paged_attention(q, c, ints(0, 10, 20, 30))
    for _ in range(5):
        r = gdn.gdn_paged_attention(q, c, ints(0, 10, 20, 30))
        assert torch.equal(r["o"], first["o"]) and torch.equal(r["lse"], first["lse"])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_many_queries(D, page, G):
    """Turns and whole prompts on the tensor cores: ragged counts around the tiles' rows, lengths around their tokens, queries
    that see nothing, requests without any."""
    lens, new = [300, 129, 128, 700, 64, 1, 0, 90, 1500, 257], [130, 129, 1, 33, 64, 1, 3, 100, 0, 256]
    c = make_cache(lens, page=page, H=2, D=D, seed=G)
    check_attention(c, queries(sum(new), 2 * G, D, BF), cu_of(new), max_new=256, **TC)
    check_attention(c, queries(sum(new), 2 * G, D, BF), cu_of(new), **TC)


def test_many_queries_of_rows_padding_and_strides():
    c = make_cache([300, 129, 515], page=16, H=2, D=64, L=2)
    qkv = queries(520, 12, 64, BF)
    new = [100, 17, 300, 90]
    o, lse = torch.full((520, 8, 64), 7.0, dtype=BF, device="cuda"), torch.full((520, 8), 7.0, device="cuda")
    check_attention(c, qkv[:, 4:], cu_of(new), rows=ints(2, -1, 0, 9), max_new=300, o=o, lse=lse, layer=1, **TC)
    assert (o[507:] == 7).all() and (lse[507:] == 7).all()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e7, 1e9])
def test_many_queries_and_scales(scale):
    """A negative scale, one of zero, and scores so far from zero that a maximum's rounding error matters."""
    c = make_cache([400], page=64, H=1, D=64)
    q = queries(60, 4, 64, BF)
    r = gdn.gdn_paged_attention(q, c, ints(0, 60), scale=scale)
    assert torch.isfinite(r["o"]).all()
    if abs(scale) < 10:
        check_attention(c, q, ints(0, 60), scale=scale, **TC)


def test_many_queries_long_and_few():
    """Few items of many tokens: cut inside an item, by several CTAs; and items of one row tile in turn."""
    c = make_cache([20011], page=64, H=1, D=128)
    check_attention(c, queries(130, 2, 128, BF), ints(0, 130), **TC)
    check_attention(c, queries(40, 2, 128, BF), ints(0, 40), **TC)
    c = make_cache([777 + 50 * i for i in range(12)], page=32, H=2, D=64)
    check_attention(c, queries(12 * 40, 4, 64, BF), cu_of([40] * 12), max_new=40, **TC)


@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_many_items(D):
    """Items of one row tile, short, long and without tokens, and of two, one after another on the same multiprocessors."""
    lens, new = [], []
    for i in range(90):
        lens.append((0, 40, 700, 130, 1500, 520, 511)[i % 7] + i)
        new.append((1, 20, 5, 3, 70, 0, 9)[i % 7])
    lens[0] = lens[21] = lens[70] = 0
    c = make_cache(lens, page=32, H=8, D=D)
    check_attention(c, queries(sum(new), 16, D, BF), cu_of(new), max_new=70, **TC)
    check_attention(c, queries(sum(new), 48, D, BF), cu_of(new), max_new=70, **TC)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_prompt_among_single_tokens(dtype):
    """Requests of one token around one of hundreds: cuts in both kinds, tiles and heads of one request after one another."""
    lens, new = [700, 90, 5, 1000, 333, 64, 2000], [1, 1, 1, 900, 1, 1, 40]
    c = make_cache(lens, page=32, H=3, D=64)
    check_attention(c, queries(sum(new), 6, 64, dtype), cu_of(new), max_new=900, **step_of(dtype, 64, 1800))
    lens, new = [50 + i for i in range(300)], [1] * 299 + [349]   # few tokens: one launch; 600 * 7 units: those of few rows by themselves
    c = make_cache(lens, page=32, H=2, D=64, W=30)
    q, cu = queries(sum(new), 4, 64, dtype), cu_of(new)
    for longest in (0, 860):
        check_attention(c, q, cu, max_new=349, max_len=longest or 349, **step_of(dtype, 64, 698))
    new = [1] * 100 + [9] * 99 + [8] * 100 + [349]               # 16 and 18 rows a head
    lens = [n + 20 for n in new]
    c = make_cache(lens, page=32, H=2, D=64, W=30)
    check_attention(c, queries(sum(new), 4, 64, dtype), cu_of(new), max_new=349, max_len=900, **step_of(dtype, 64, 698))
    # a prompt alone that is not there: all requests are the other launch's
    c = make_cache([30] * 300, page=32, H=2, D=64, W=30)
    check_attention(c, queries(300, 4, 64, dtype), cu_of([1] * 300), max_len=900, **step_of(dtype, 64, 600))


def test_many_queries_many_requests():
    lens = [(37 * i) % 300 for i in range(400)]
    new = [(5 * i) % 23 for i in range(400)]
    c = make_cache(lens, page=16, H=1, D=64)
    check_attention(c, queries(sum(new), 2, 64, BF), cu_of(new), max_new=22, **TC)


def test_many_queries_blocks_of_different_sizes():
    c = make_cache([700], page=16, H=1, D=128, spread=12)
    check_attention(c, queries(80, 2, 128, BF, gain=0.1), ints(0, 80), **TC)


def test_many_queries_bad_pages():
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        c = make_cache([400, 50], page=16, H=2, D=64)
        want = gdn.gdn_paged_attention(queries(90, 4, 64, BF), c, ints(0, 60, 90))["o"]
        c.table[0, 3] = bad
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        r = gdn.gdn_paged_attention(queries(90, 4, 64, BF), c, ints(0, 60, 90), ws=ws)
        assert gdn.read_status(ws=ws) == gdn.GDN_ERR_INVALID_ARG
        assert torch.equal(r["o"][60:], want[60:])


@pytest.mark.parametrize("D", [64, 128])
def test_many_queries_wait_limit(D):
    """With the testing hook the converting warps stop; the waits run out, are reported, and the next call is right again."""
    c = make_cache([900, 800], page=16, H=2, D=D)
    q, cu = queries(300, 4, D, BF), ints(0, 200, 300)
    ws = torch.zeros(int(gdn.lib().gdn_workspace_size()), dtype=torch.uint8, device="cuda")
    want = gdn.gdn_paged_attention(q, c, cu, ws=ws)["o"]
    torch.cuda.synchronize()
    assert gdn.read_status(ws=ws) == gdn.GDN_OK
    try:
        gdn.set_wait_limit_ns(20_000_000)   # 20 ms
        for stall in (0, 1):
            gdn.debug_stall_after(stall)
            gdn.gdn_paged_attention(q, c, cu, ws=ws)
            torch.cuda.synchronize()
            if stall == 0:
                assert gdn.read_status(ws=ws) == gdn.GDN_ERR_DEVICE_TIMEOUT
    finally:
        gdn.debug_stall_after(-1)
        gdn.set_wait_limit_ns(0)
    gdn.clear_status(ws=ws)
    again = gdn.gdn_paged_attention(q, c, cu, ws=ws)["o"]
    torch.cuda.synchronize()
    assert gdn.read_status(ws=ws) == gdn.GDN_OK and torch.equal(again, want)
