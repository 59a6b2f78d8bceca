"""A small hybrid model served on a shared prefix: linear-attention layers and full-attention layers in turn.

The prefix is prefilled once.  Every request then forks from it: its linear layers start from the prefix's final state
(S0_index), its attention layers read the prefix's keys and values beside the request's own tail.  A ragged turn of new
tokens is prefilled for all requests at once, and tokens are decoded greedily, one a request and step, with the states
updated in place.  Weights are random: the point is how the three operators fit together.

    python examples/hybrid_serve.py [--requests 8] [--prefix 2000] [--tokens 16] [--dtype bf16|f32]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hybrid_model_recurrent_gb300 as gdn  # noqa: E402

VOCAB, D_MODEL, HEADS, KV_HEADS, D_HEAD, LAYERS = 512, 256, 4, 2, 64, 4   # even layers linear, odd ones attention


def weights(dtype, seed: int = 0, device: str = "cuda"):
    g = torch.Generator().manual_seed(seed)

    def w(*shape):
        return (torch.randn(*shape, generator=g) / math.sqrt(shape[-1])).to(device, dtype)

    kinds = ["linear" if i % 2 == 0 else "attention" for i in range(LAYERS)]
    return dict(embed=w(VOCAB, D_MODEL) * 16, layers=[
        dict(kind=k, q=w(HEADS * D_HEAD, D_MODEL), o=w(D_MODEL, HEADS * D_HEAD),
             k=w((HEADS if k == "linear" else KV_HEADS) * D_HEAD, D_MODEL),
             v=w((HEADS if k == "linear" else KV_HEADS) * D_HEAD, D_MODEL)) for k in kinds],
        alpha=(1.0 - 2.0 ** -torch.arange(2.0, 2.0 + HEADS)).to(device))


def norm(x):
    x = x.float() if x.dtype == torch.bfloat16 else x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def heads(x, w, dtype):
    y = norm(x).to(dtype) @ w.T
    return y.unflatten(-1, (-1, D_HEAD))


class Server:
    """One shared prefix and a batch of requests on it."""

    def __init__(self, w, prefix, requests: int, capacity: int):
        self.w, self.B, self.cap = w, requests, capacity
        self.dtype = w["embed"].dtype
        dev = w["embed"].device
        self.lens = torch.zeros(requests, dtype=torch.int32, device=dev)   # tokens in each request's tail
        self.used = [0] * requests    # the same, for checks on the host
        self.forks = [0] * requests   # the state that each request's linear layers go on from: at first the prefix's
        self.state = []
        x = w["embed"][prefix].float()
        P = len(prefix)
        for ly in w["layers"]:
            q, k, v = (heads(x, ly[n], self.dtype) for n in "qkv")
            if ly["kind"] == "linear":
                r = gdn.gdn_linear_prefill(q, k, v, w["alpha"], [0, P], scale=D_HEAD ** -0.5)
                self.state.append(r["S_final"])
                y = r["o"]
            else:
                # the prefix itself: one request whose tail is the prefix, every token a query
                y = gdn.gdn_prefix_attention(q[None], k[:0], v[:0], k[None], v[None],
                                             torch.full((1,), P, dtype=torch.int32, device=dev))["o"][0]
                tails = [torch.zeros(requests, capacity, KV_HEADS, D_HEAD, dtype=self.dtype, device=dev) for _ in "kv"]
                self.state.append((k, v, *tails))
            x = x + (y.flatten(-2) @ ly["o"].T).float()

    def grow(self, n):
        """Room for n[b] more tokens in request b's tail."""
        used = [u + m for u, m in zip(self.used, n)]
        if max(used) > self.cap:
            raise ValueError(f"a tail of {max(used)} tokens is past the capacity of {self.cap}")
        self.used = used

    def turn(self, prompts):
        """Prefill a ragged turn (a list of token tensors, one a request) after what each request has; returns the logits of each
        request's last token."""
        n = [len(p) for p in prompts]
        if len(n) != self.B or min(n) < 1:
            raise ValueError("a turn takes a prompt of at least one token for each request")
        self.grow(n)
        top, cu = max(n), [0]
        for m in n:
            cu.append(cu[-1] + m)
        dev = self.lens.device
        had = self.lens.long()
        self.lens += torch.tensor(n, dtype=torch.int32, device=dev)
        x = self.w["embed"][torch.cat(prompts)].float()
        # attention takes the last `top` tokens of every tail: rows of shorter turns are padded in front
        row = torch.cat([torch.arange(m, device=dev) + b * top + top - m for b, m in enumerate(n)])
        req = torch.repeat_interleave(torch.arange(self.B, device=dev), torch.tensor(n, device=dev))
        pos = torch.cat([torch.arange(m, device=dev) for m in n]) + had[req]
        for i, ly in enumerate(self.w["layers"]):
            q, k, v = (heads(x, ly[c], self.dtype) for c in "qkv")
            if ly["kind"] == "linear":
                r = gdn.gdn_linear_prefill(q, k, v, self.w["alpha"], cu, scale=D_HEAD ** -0.5, S0=self.state[i],
                                           S0_index=self.forks)
                self.state[i], y = r["S_final"], r["o"]
            else:
                kp, vp, kt, vt = self.state[i]
                kt[req, pos], vt[req, pos] = k, v
                qp = torch.zeros(self.B * top, HEADS, D_HEAD, dtype=self.dtype, device=dev)
                qp[row] = q
                y = gdn.gdn_prefix_attention(qp.unflatten(0, (self.B, top)), kp, vp, kt, vt, self.lens)["o"].flatten(0, 1)[row]
            x = x + (y.flatten(-2) @ ly["o"].T).float()
        self.forks = list(range(self.B))   # from now on its own
        return self.logits(x[torch.tensor(cu[1:], device=dev) - 1])

    def step(self, tokens):
        """One token a request; returns its logits."""
        self.grow([1] * self.B)
        x = self.w["embed"][tokens].float()
        at = self.lens.long()
        every = torch.arange(self.B, device=tokens.device)
        self.lens += 1
        for i, ly in enumerate(self.w["layers"]):
            q, k, v = (heads(x, ly[c], self.dtype) for c in "qkv")
            if ly["kind"] == "linear":
                y = gdn.gdn_linear_step(q, k, v, self.w["alpha"], self.state[i], scale=D_HEAD ** -0.5)
            else:
                kp, vp, kt, vt = self.state[i]
                kt[every, at], vt[every, at] = k, v
                y = gdn.gdn_prefix_attention(q[:, None], kp, vp, kt, vt, self.lens)["o"][:, 0]
            x = x + (y.flatten(-2) @ ly["o"].T).float()
        return self.logits(x)

    def logits(self, x):
        return norm(x).to(self.dtype).float() @ self.w["embed"].float().T / 16


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prefix", type=int, default=2000)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    a = ap.parse_args()
    gdn.build()
    g = torch.Generator().manual_seed(1)
    w = weights(torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    prefix = torch.randint(VOCAB, (a.prefix,), generator=g).cuda()
    turns = [torch.randint(VOCAB, (int(torch.randint(1, 40, (1,), generator=g)),), generator=g).cuda()
             for _ in range(a.requests)]
    s = Server(w, prefix, a.requests, 40 + a.tokens)
    tokens = s.turn(turns).argmax(-1)
    out = [tokens]
    for _ in range(a.tokens - 1):
        tokens = s.step(tokens).argmax(-1)
        out.append(tokens)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    for b, row in enumerate(torch.stack(out, 1).tolist()):
        print(f"request {b} ({len(turns[b])} new tokens on {a.prefix} shared): {row}")


if __name__ == "__main__":
    main()
