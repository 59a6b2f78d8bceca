"""Several turns and decode steps of examples/hybrid_serve.py on the GPU, against the whole model in 64 bits (tolerance and plain
model: test_hybrid_serve_gpu.py)."""
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn
from test_hybrid_serve_gpu import ex, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_turns_and_steps_follow_one_another(dtype):
    gdn.build()
    w = ex.weights(dtype, seed=4)
    g = torch.Generator().manual_seed(6)

    def toks(n):
        return torch.randint(ex.VOCAB, (n,), generator=g).cuda()

    prefix = toks(200)
    s, seqs = ex.Server(w, prefix, 3, 260), [prefix] * 3
    tol = 52 * torch.finfo(dtype).eps / 2
    for lens in ((130, 1, 40), None, (3, 100, 17), None, (1, 1, 129)):
        new = [toks(n) for n in (lens or (1, 1, 1))]
        seqs = [torch.cat(x) for x in zip(seqs, new)]
        logits = s.turn(new) if lens else s.step(torch.cat(new))
        for b, seq in enumerate(seqs):
            want = plain(w, seq)
            err = (logits[b].double() - want).abs().max() / want.abs().max()
            assert err <= tol, f"request {b}: {err.item():.3g} of the largest logit, {tol:.3g} allowed"
    assert gdn.read_status("cuda") == gdn.GDN_OK
