"""The bookkeeping of examples/hybrid_serve.py on the host (no GPU): the three operators are stood in for by plain ones, and the
served logits compared with the whole model recomputed in 64 bits.

Tolerance: fp32 throughout, 52 half steps of the largest logit for the roundings of 4 layers, and as many for the sums of up to
512 terms in fp32 within each."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("hybrid_serve_host", os.path.join(ROOT, "examples", "hybrid_serve.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)
TOL = 104 * 2.0 ** -24


class Plain:
    """The operators that the example calls, token by token in 64 bits."""

    @staticmethod
    def gdn_linear_prefill(q, k, v, alpha, cu, *, scale=1.0, S0=None, S0_index=None):
        o, states = torch.empty_like(v), []
        for b in range(len(cu) - 1):
            S = torch.zeros(v.shape[1], v.shape[2], k.shape[2], dtype=torch.float64)
            if S0 is not None:
                S = S0[b if S0_index is None else S0_index[b]].double()
            for t in range(cu[b], cu[b + 1]):
                S = alpha.double()[:, None, None] * S + v[t].double()[:, :, None] * k[t].double()[:, None, :]
                o[t] = (scale * (S * q[t].double()[:, None, :]).sum(-1)).to(o.dtype)
            states.append(S.float())
        return dict(o=o, S_final=torch.stack(states))

    @staticmethod
    def gdn_linear_step(q, k, v, alpha, states, *, scale=1.0):
        assert len(states) == len(q)
        S = alpha.double()[:, None, None] * states.double() + v.double()[..., :, None] * k.double()[..., None, :]
        states.copy_(S)
        return (scale * (S * q.double()[:, :, None, :]).sum(-1)).to(v.dtype)

    @staticmethod
    def gdn_prefix_attention(q, kp, vp, kt, vt, tail_len):
        B, n, Hq, D = q.shape
        o, of = torch.zeros_like(q), torch.arange(Hq) // (Hq // kp.shape[1])
        for b in range(B):
            L = int(tail_len[b])
            keys, vals = torch.cat([kp, kt[b, :L]])[:, of].double(), torch.cat([vp, vt[b, :L]])[:, of].double()
            for i in range(n):
                end = len(kp) + max(L - n + i + 1, 0)
                if end:
                    p = torch.softmax(torch.einsum("hd,khd->hk", q[b, i].double(), keys[:end]) * D ** -0.5, -1)
                    o[b, i] = torch.einsum("hk,khd->hd", p, vals[:end]).to(o.dtype)
        return dict(o=o)


def whole(w, tokens):
    """Logits of the last token, the whole sequence in 64 bits."""
    x, n = w["embed"][tokens].double(), len(tokens)
    gap = torch.arange(n)[:, None] - torch.arange(n)[None, :]
    for ly in w["layers"]:
        h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        q, k, v = ((h @ ly[c].double().T).unflatten(-1, (-1, ex.D_HEAD)).transpose(0, 1) for c in "qkv")
        s = q @ k.repeat_interleave(ex.HEADS // k.shape[0], 0).transpose(1, 2) * ex.D_HEAD ** -0.5
        if ly["kind"] == "linear":
            s = torch.where(gap >= 0, s * w["alpha"].double()[:, None, None] ** gap.clamp(min=0), 0.0)
        else:
            s = torch.softmax(s.masked_fill(gap < 0, float("-inf")), -1)
        x = x + (s @ v.repeat_interleave(ex.HEADS // v.shape[0], 0)).transpose(0, 1).flatten(1) @ ly["o"].double().T
    x = x[-1]
    return (x * torch.rsqrt(x.square().mean() + 1e-6)) @ w["embed"].double().T / 16


@pytest.fixture
def server(monkeypatch):
    monkeypatch.setattr(ex, "gdn", Plain)
    w = ex.weights(torch.float32, seed=3, device="cpu")
    g = torch.Generator().manual_seed(5)

    def tokens(n):
        return torch.randint(ex.VOCAB, (n,), generator=g)

    prefix = tokens(21)
    return w, prefix, tokens, lambda capacity: ex.Server(w, prefix, 3, capacity)


def check(w, logits, seqs):
    for b, seq in enumerate(seqs):
        want = whole(w, seq)
        err = ((logits[b].double() - want).abs().max() / want.abs().max()).item()
        assert err <= TOL, f"request {b}: {err:.3g} of the largest logit"


def test_turns_and_steps_follow_one_another(server):
    """Turn, steps, turn, step, turn: every request keeps its own state and tail."""
    w, prefix, tokens, make = server
    s, seqs = make(40), [prefix] * 3
    for lens in ((1, 7, 4), None, None, (5, 1, 3), None, (2, 2, 6)):
        new = [tokens(n) for n in (lens or (1, 1, 1))]
        seqs = [torch.cat(x) for x in zip(seqs, new)]
        check(w, s.turn(new) if lens else s.step(torch.cat(new)), seqs)


def test_tails_past_their_capacity_are_refused(server):
    """On the host and before anything changes: an index past a buffer would reach the GPU otherwise."""
    w, prefix, tokens, make = server
    s, first = make(8), [tokens(6), tokens(1), tokens(3)]
    with pytest.raises(ValueError, match="capacity"):
        s.turn([tokens(1), tokens(9), tokens(1)])
    check(w, s.turn(first), [torch.cat([prefix, t]) for t in first])
    with pytest.raises(ValueError, match="capacity"):
        s.turn([tokens(3), tokens(1), tokens(1)])
    seqs = [torch.cat([prefix, t]) for t in first]
    for _ in range(2):
        new = tokens(3)
        seqs = [torch.cat([q, new[b:b + 1]]) for b, q in enumerate(seqs)]
        check(w, s.step(new), seqs)
    with pytest.raises(ValueError, match="capacity"):
        s.step(tokens(3))
    assert s.lens.tolist() == [8, 3, 5]


@pytest.mark.parametrize("lens", [(0, 2, 3), (2, 0, 3), (2, 3, 0), (0, 0, 0), (2, 3), (2, 3, 1, 1)])
def test_turns_without_a_token_for_each_request_are_refused(server, lens):
    """A request without a token has no last token whose logits the turn could return (it would get another's)."""
    w, _, tokens, make = server
    s = make(8)
    with pytest.raises(ValueError, match="prompt"):
        s.turn([tokens(n) for n in lens])
    assert s.lens.tolist() == [0, 0, 0]
