"""The operators of include/gdn_cache.h together, as a server uses them: a prefix, forks of it, ragged turns, decode from a
captured graph with the rows' growth, requests that leave and others in their places, compaction.  What the cache holds is
followed on the host bit for bit, every attention checked against the definition in 64 bits."""
import importlib.util
import os

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from cache_util import E4M3, check_attention
from test_cache_append_gpu import define

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Served:
    """A layer's queries, keys and values for new tokens, through the four operators, and a shadow of the cache."""

    def __init__(self, R, dtype, page=16, H=2, D=64, Hq=4, N=60, W=12):
        self.c = gdn.PagedCache.empty(1, N, H, D, R, W, page_size=page)
        self.H, self.D, self.Hq, self.dtype, self.page = H, D, Hq, dtype, page
        self.freq = gdn.gdn_rope_frequencies(D)
        self.g = torch.Generator(device="cuda").manual_seed(5)

    def streams(self, T):
        x = torch.randn(T, self.Hq + 2 * self.H, self.D, generator=self.g, device="cuda").to(self.dtype)
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.H], x[:, self.Hq + self.H:]

    def tokens(self, rows, new):
        """New tokens of some rows, whose lens count them already."""
        c = self.c
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        lens = c.lens.tolist()
        q, k, v = self.streams(cu[-1])
        pos = ints(lens[r] - n + i for r, n in zip(rows, new) for i in range(n))
        q, k = gdn.gdn_qk_norm_rope(q, k, pos, self.freq, eps=1e-6)
        pages, scales = define(c.pages[0].double().cpu(), c.scales[0].double().cpu(), c.table.tolist(), lens, self.page, k.cpu(),
                               v.cpu(), cu, rows)
        gdn.gdn_cache_append(k, v, c, ints(cu), rows=ints(rows), max_new=max(new))
        assert torch.equal(c.pages[0].double().cpu(), pages) and torch.equal(c.scales[0].double().cpu(), scales)
        rows_at_once = max(new) * self.Hq // self.H
        check_attention(c, q, ints(cu), rows=ints(rows), max_new=max(new),
                        **(dict(cut=2.0 ** -24) if self.dtype == BF and rows_at_once > 16 else {}))

    def held(self, row):
        """What a row's cache holds, as values."""
        n = int(self.c.lens[row])
        pg = self.c.table[row, :-(-n // self.page)].long()
        x = self.c.pages.view(torch.uint8)[0, pg].view(E4M3).float() * self.c.scales[0, pg][..., None, None]
        return x.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n].clone()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_server(dtype):
    s = Served(5, dtype)
    c = s.c
    gdn.gdn_cache_update(c, grow=ints([41, 0, 0, 0, 0]))
    s.tokens([0], [41])                                              # the prefix
    prefix = s.held(0)
    gdn.gdn_cache_update(c, fork_from=ints([0, 0, 0, 0]), fork_to=ints([1, 2, 3, 4]))
    gdn.gdn_cache_update(c, grow=ints([0, 7, 1, 30, 20]))
    s.tokens([1, 2, 3, 4], [7, 1, 30, 20])                           # turns of four requests on it
    assert torch.equal(s.held(0), prefix)
    gdn.gdn_cache_update(c, grow=ints([0, 1, 1, 1, 1]))
    s.tokens([1, 2, 3, 4], [1] * 4)                                  # a token of each
    kept = s.held(3)
    gdn.gdn_cache_update(c, drop=ints([1]), fork_from=ints([0, 3]), fork_to=ints([2, 1]), grow=ints([0, 2, 3, 0, 0]))
    s.tokens([1, 2], [2, 3])                                         # row 2 anew, row 1 a branch of row 3
    assert torch.equal(s.held(3), kept) and torch.equal(s.held(0), prefix) and torch.equal(s.held(1)[:, :, :72], kept)
    before = [s.held(r) for r in range(5)]
    gdn.gdn_cache_update(c, drop=ints([4]))
    assert int(gdn.gdn_cache_compact(c)) == int((c.refs > 0).sum())
    for r in range(4):
        assert torch.equal(s.held(r), before[r])
    gdn.gdn_cache_update(c, grow=ints([0, 1, 1, 1, 0]))
    s.tokens([3, 1, 2], [1, 1, 1])
    assert gdn.read_status("cuda") == gdn.GDN_OK


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_from_a_graph(dtype):
    """Growth, rotation, append and attention of one token a row in one captured graph, replayed over page ends; the same
    calls made one by one leave the same bits."""
    runs = []
    for captured in (False, True):
        s = Served(3, dtype)
        c = s.c
        gdn.gdn_cache_update(c, grow=ints([20, 31, 5]))
        s.tokens([0, 1, 2], [20, 31, 5])
        q, k, v = (x.clone() for x in s.streams(3))
        grow, cu, pos = ints([1, 1, 1]), ints([0, 1, 2, 3]), c.lens.clone()

        def step():
            gdn.gdn_cache_update(c, grow=grow)
            a, b = gdn.gdn_qk_norm_rope(q, k, pos, s.freq, eps=1e-6)
            gdn.gdn_cache_append(b, v, c, cu, max_new=1)
            return gdn.gdn_paged_attention(a, c, cu, max_new=1)

        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step()
        outs = []
        for i in range(40):
            for x in (q, k, v):
                x.copy_(torch.randn(x.shape, generator=s.g, device="cuda"))
            pos.copy_(c.lens)
            if captured:
                graph.replay()
            else:
                out = step()
            outs.append((out["o"].clone(), out["lse"].clone()))
        torch.cuda.synchronize()
        assert c.lens.tolist() == [60, 71, 45] and gdn.read_status("cuda") == gdn.GDN_OK
        runs.append((outs, [s.held(r) for r in range(3)]))
    for (a, b), (x, y) in zip(*(r[0] for r in runs)):
        assert torch.equal(a, x) and torch.equal(b, y)
    for a, b in zip(*(r[1] for r in runs)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_example(dtype):
    """examples/hybrid_serve.py with a paged cache: it runs, requests with the same prompts answer alike, and one that starts anew
    answers as it did."""
    spec = importlib.util.spec_from_file_location("hybrid_serve_paged", os.path.join(ROOT, "examples", "hybrid_serve.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    g = torch.Generator().manual_seed(1)
    prefix = torch.randint(ex.VOCAB, (300,), generator=g).cuda()
    one, two = (torch.randint(ex.VOCAB, (n,), generator=g).cuda() for n in (9, 9))
    s = ex.PagedServer(ex.weights(dtype), prefix, 3, 40)
    first = s.turn([one, two, one])
    assert first.shape == (3, ex.VOCAB) and torch.isfinite(first).all()
    tokens = first.argmax(-1)
    for _ in range(12):
        logits = s.step(tokens)
        assert torch.isfinite(logits).all()
        tokens = logits.argmax(-1)
    assert s.cache.lens.tolist() == [300, 321, 321, 321]
    s.restart([1])
    assert s.cache.lens.tolist() == [300, 321, 300, 321]
    s.turn([one, two, one])
    with pytest.raises(ValueError, match="capacity"):
        s.turn([one, torch.cat([two] * 4), one])
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK


def test_the_example_with_one_request():
    """A single request that starts anew goes on from the prefix as it did the first time."""
    spec = importlib.util.spec_from_file_location("hybrid_serve_paged_one", os.path.join(ROOT, "examples", "hybrid_serve.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    g = torch.Generator().manual_seed(2)
    prefix, one = (torch.randint(ex.VOCAB, (n,), generator=g).cuda() for n in (100, 1))
    s = ex.PagedServer(ex.weights(F32), prefix, 1, 10)
    first = s.step(one)
    s.step(one)
    s.restart([0])
    assert torch.equal(s.step(one), first)
