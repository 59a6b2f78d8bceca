"""What the paged example answers: requests with the same prompt alike, one that starts anew as the first time, others not; and the
wait limit of the tensor-core attention when copies stop in the middle of an item.

How alike: the same prompt in another place of the batch is cut differently over the GPU, so sums differ by roundings; a rounding
may move a held key or value to its neighbour in e4m3, an eighth of itself at most, and nothing moves further.  So alike means
within an eighth of what different prompts differ by, which a fork of the wrong row or a state of another request does not meet."""
import importlib.util
import os

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from cache_util import make_cache

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    gdn.build()
    spec = importlib.util.spec_from_file_location("hybrid_serve_alike", os.path.join(ROOT, "examples", "hybrid_serve.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def apart(a, b):
    return float((a - b).float().norm())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_prompts_answer_alike(ex, dtype):
    g = torch.Generator().manual_seed(1)
    prefix = torch.randint(ex.VOCAB, (300,), generator=g).cuda()
    one, two, three = (torch.randint(ex.VOCAB, (n,), generator=g).cuda() for n in (9, 9, 5))
    s = ex.PagedServer(ex.weights(dtype), prefix, 3, 60)
    first = s.turn([one, two, one])
    differ = apart(first[0], first[1])
    assert differ > 0.1 * float(first[0].norm())
    assert apart(first[0], first[2]) <= differ / 8
    token = first[0].argmax()
    then = s.step(torch.stack([token, token, token]))                 # the same again, behind equal and different turns
    assert apart(then[0], then[2]) <= apart(then[0], then[1]) / 8
    s.restart([1])
    again = s.turn([three, two, three])                               # request 1 anew, the others go on
    assert apart(again[1], first[1]) <= differ / 8
    assert apart(again[0], again[2]) <= apart(again[0], again[1]) / 8
    s.restart([0, 2])
    last = s.turn([two, three, one])
    assert apart(last[0], first[1]) <= differ / 8 and apart(last[2], first[0]) <= differ / 8
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("stall", [0, 1, 3])
def test_copies_that_stop_inside_an_item(D, stall):
    """With the testing hook a multiprocessor's copies stop after some tiles, of six or more that it has; the waits of 20 ms run out and are
    reported, and the next call is right again."""
    gdn.build()
    c = make_cache([20000], page=64, H=2, D=D)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(700, 4, D, generator=g, device="cuda").to(BF)
    cu = torch.tensor([0, 700], dtype=torch.int32, device="cuda")
    ws = torch.zeros(int(gdn.lib().gdn_workspace_size()), dtype=torch.uint8, device="cuda")
    want = gdn.gdn_paged_attention(q, c, cu, ws=ws)["o"]
    torch.cuda.synchronize()
    assert gdn.read_status(ws=ws) == gdn.GDN_OK
    try:
        gdn.set_wait_limit_ns(20_000_000)
        gdn.debug_stall_after(stall)
        gdn.gdn_paged_attention(q, c, cu, ws=ws)
        torch.cuda.synchronize()
        assert gdn.read_status(ws=ws) == gdn.GDN_ERR_DEVICE_TIMEOUT
    finally:
        gdn.debug_stall_after(-1)
        gdn.set_wait_limit_ns(0)
    gdn.clear_status(ws=ws)
    again = gdn.gdn_paged_attention(q, c, cu, ws=ws)["o"]
    torch.cuda.synchronize()
    assert gdn.read_status(ws=ws) == gdn.GDN_OK and torch.equal(again, want)
