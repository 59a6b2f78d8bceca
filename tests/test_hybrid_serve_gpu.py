"""The example that runs the three operators of include/gdn_hybrid.h together, against the whole model recomputed in 64 bits
for every request and token.

Tolerance: a value passes through about 12 roundings a layer (norm, projections, operator, product, sum), each of at most
half a step relative to the value, and the logits through 4 more: 52 half steps of the largest logit for 4 layers."""
import importlib.util
import os

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("hybrid_serve", os.path.join(ROOT, "examples", "hybrid_serve.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


def plain(w, tokens):
    """Logits of the last token, the whole sequence in 64 bits."""
    x = w["embed"][tokens].double()
    n = len(tokens)
    al = w["alpha"].double()
    t = torch.arange(n, device=x.device)
    for ly in w["layers"]:
        h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        q, k, v = ((h @ ly[c].double().T).unflatten(-1, (-1, ex.D_HEAD)).transpose(0, 1) for c in "qkv")
        s = q @ k.repeat_interleave(ex.HEADS // k.shape[0], 0).transpose(1, 2) * ex.D_HEAD ** -0.5
        gap = t[:, None] - t[None, :]
        if ly["kind"] == "linear":
            s = torch.where(gap >= 0, s * al[:, None, None] ** gap.clamp(min=0), 0.0)
        else:
            s = torch.softmax(s.masked_fill(gap < 0, float("-inf")), -1)
        y = (s @ v.repeat_interleave(ex.HEADS // v.shape[0], 0)).transpose(0, 1).flatten(1)
        x = x + y @ ly["o"].double().T
    x = x[-1]
    return (x * torch.rsqrt(x.square().mean() + 1e-6)) @ w["embed"].double().T / 16


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_serving_equals_the_whole_model(dtype):
    gdn.build()
    w = ex.weights(dtype, seed=3)
    g = torch.Generator().manual_seed(5)

    def toks(n):
        return torch.randint(ex.VOCAB, (n,), generator=g).cuda()

    prefix, turns = toks(333), [toks(n) for n in (1, 30, 129, 7)]
    s = ex.Server(w, prefix, 4, 140)
    logits = s.turn(turns)
    seqs = [torch.cat([prefix, t]) for t in turns]
    tol = 52 * torch.finfo(dtype).eps / 2
    for step in range(4):
        for b, seq in enumerate(seqs):
            want = plain(w, seq)
            err = (logits[b].double() - want).abs().max() / want.abs().max()
            assert err <= tol, f"request {b}, step {step}: {err.item():.3g} of the largest logit, {tol:.3g} allowed"
        nxt = toks(4)
        seqs = [torch.cat([q, nxt[b:b + 1]]) for b, q in enumerate(seqs)]
        logits = s.step(nxt)
    assert gdn.read_status("cuda") == gdn.GDN_OK
