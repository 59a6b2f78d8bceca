"""Cases for the serving operators of a hybrid model's other layers: linear attention with a decay for
each head (prompts and single tokens) and attention for a batch that shares a long prefix.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) or, where
``own`` is true, through the package's entry points.  ``exact`` evaluates the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 128  # tokens of a chunk of the plain chunked form


def listed():
    return [
        # the serving framework's prefill workload (8 prompts, 16 heads, a checkpoint every 512 tokens)
        # on a linear-attention layer
        dict(name="prefill_8x16x8192", op="prefill", lens="equal", B=8, T=8192, H=16, Hk=16, dk=128, dv=128,
             dtype="bf16", ckpt=512, fork=False),
        # one very long document: few scans, so the work has to be split along the tokens
        dict(name="prefill_long_1x32x131072", op="prefill", lens="equal", B=1, T=131072, H=32, Hk=32, dk=128, dv=128,
             dtype="bf16", ckpt=16384, fork=False),
        # a batch of ragged new turns that all continue from one cached prefix state, with queries and keys
        # shared by groups of four heads
        dict(name="prefill_ragged_32x16", op="prefill", lens="ragged", B=32, T=1999, H=16, Hk=4, dk=128, dv=128,
             dtype="bf16", ckpt=0, fork=True),
        # smallest: two narrow heads in full precision, a checkpoint every 64 tokens
        dict(name="prefill_f32_1x2x256", op="prefill", lens="equal", B=1, T=256, H=2, Hk=2, dk=32, dv=32,
             dtype="f32", ckpt=64, fork=False),
        # an interactive user's next token: latency
        dict(name="step_b1", op="step", B=1, H=16, Hk=16, dk=128, dv=128, dtype="bf16", extra=3, pad=0),
        # a full decode batch over a scattered pool of states, three of its rows padding
        dict(name="step_b67", op="step", B=67, H=32, Hk=32, dk=128, dv=128, dtype="bf16", extra=61, pad=3),
        # a large decode batch of narrow heads in full precision, queries and keys shared by pairs of heads
        dict(name="step_f32_b256_d64", op="step", B=256, H=32, Hk=16, dk=64, dv=64, dtype="f32", extra=0, pad=0),
        # a few requests on a short common system prompt: latency
        dict(name="prefix_small_b4", op="prefix", B=4, n=1, Hq=16, Hkv=2, D=128, P=1000, cap=96, dtype="bf16"),
        # a decode batch on one long shared document, four query heads a key/value head
        dict(name="prefix_decode_b64", op="prefix", B=64, n=1, Hq=32, Hkv=8, D=128, P=32768, cap=1024, dtype="bf16"),
        # four drafted tokens of each request checked at once, every head with its own narrow keys and values
        dict(name="prefix_draft_b32_d64", op="prefix", B=32, n=4, Hq=16, Hkv=16, D=64, P=8191, cap=500, dtype="bf16"),
        # new turns of 256 tokens on a shared prefix: bound by the products
        dict(name="prefix_turns_b16", op="prefix", B=16, n=256, Hq=32, Hkv=4, D=128, P=16384, cap=700, dtype="bf16"),
        # full precision, odd sizes
        dict(name="prefix_f32_b7", op="prefix", B=7, n=1, Hq=8, Hkv=8, D=64, P=2047, cap=77, dtype="f32"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "step", "prefix"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "prefill":
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (32, 32), (64, 128), (128, 64)])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 4])
        B = _log_uniform(rng, 1, 32)
        T = _log_uniform(rng, 1, max(2, min(65536, 2 ** 24 // (8 * B * H))))
        return dict(op=op, lens=rng.choice(["equal", "ragged"]), B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype,
                    ckpt=rng.choice([0, 0, 100, 512, 1024]), fork=rng.random() < 0.5)
    if op == "step":
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (32, 32), (64, 128), (128, 32)])
        Hk = rng.choice([1, 2, 4, 5, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 4])
        B = _log_uniform(rng, 1, 256)
        return dict(op=op, B=B, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, extra=rng.randint(0, 20),
                    pad=rng.randint(0, B // 4))
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    n = rng.choice([1, 1, 2, 4, 7, 33, 128])
    B = _log_uniform(rng, 1, 128)
    if dtype == "f32":
        n, B = min(n, 2), min(B, 16)
    D = rng.choice([64, 128, 128])
    rows = B * n * Hq
    P = min(_log_uniform(rng, 1, 65536), max(1, 2 ** 31 // rows))
    cap = max(n, min(_log_uniform(rng, 1, 4096), 2 ** 31 // rows, 2 ** 22 // B))
    return dict(op=op, B=B, n=n, Hq=Hq, Hkv=Hkv, D=D, P=P, cap=cap, dtype=dtype)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=torch.float32, unit=False):
    x = torch.empty(shape, dtype=dtype if not unit else torch.float32, device="cuda").normal_(generator=g)
    if unit:
        x = x / x.norm(dim=-1, keepdim=True)
    return x.to(dtype)


def _alpha(H):
    # decays with half lives from about one token to a few hundred over the heads
    h = torch.arange(1, H + 1, dtype=torch.float64)
    return torch.exp(-torch.pow(2.0, -8.0 * h / H)).float().cuda()


def _lens(case):
    # a ragged batch's lengths go with the case, not with the seed: other inputs have the same shapes
    if case["lens"] == "equal":
        return [case["T"]] * case["B"]
    g = torch.Generator()
    g.manual_seed(1000 * case["B"] + case["T"])
    return [int(x) for x in torch.randint(1, case["T"] + 1, (case["B"],), generator=g)]


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "prefill":
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        lens = _lens(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        T = cu[-1]
        s.update(cu=cu, q=_normal(g, (T, Hk, dk), dt, True), k=_normal(g, (T, Hk, dk), dt, True),
                 v=_normal(g, (T, H, dv), dt), alpha=_alpha(H), S0=None, S0_index=None, ckpt=None, scale=1.0)
        if case["fork"]:
            # every sequence starts from one cached state in a pool of four
            s["S0"] = _normal(g, (4, H, dv, dk)) * 0.3
            s["S0_index"] = [2] * len(lens)
        if case["ckpt"]:
            s["ckpt"] = [list(range(case["ckpt"], n + 1, case["ckpt"])) for n in lens]
    elif case["op"] == "step":
        B, H, Hk, dk, dv = case["B"], case["H"], case["Hk"], case["dk"], case["dv"]
        N = B + case["extra"]
        perm = torch.randperm(N, generator=g, device="cuda")[:B].to(torch.int32)
        if case["pad"]:
            perm[B - case["pad"]:] = -1
        s.update(q=_normal(g, (B, Hk, dk), dt, True), k=_normal(g, (B, Hk, dk), dt, True), v=_normal(g, (B, H, dv), dt),
                 alpha=_alpha(H), states=_normal(g, (N, H, dv, dk)) * 0.3, slots=perm, scale=1.0)
    else:
        B, n, Hq, Hkv, D, P, cap = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "P", "cap"))
        tail = torch.randint(min(n, cap), cap + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s.update(q=_normal(g, (B, n, Hq, D), dt), k_prefix=_normal(g, (P, Hkv, D), dt),
                 v_prefix=_normal(g, (P, Hkv, D), dt), k_tail=_normal(g, (B, cap, Hkv, D), dt),
                 v_tail=_normal(g, (B, cap, Hkv, D), dt), tail_len=tail, scale=D ** -0.5)
    return s


def _present(**outputs):
    # a prefill without checkpoints has no checkpoint states
    return {name: x for name, x in outputs.items() if x is not None}


def _plain_prefill(s):
    q, k, v, alpha, cu = s["q"].float(), s["k"].float(), s["v"].float(), s["alpha"], s["cu"]
    H, dv, dk = v.shape[1], v.shape[2], k.shape[2]
    rep = H // k.shape[1]
    o = torch.empty_like(v)
    final, dumps = [], []
    la = torch.log(alpha.double())
    i = torch.arange(CHUNK, device=q.device)
    diff = (i[:, None] - i[None, :])
    D = torch.where(diff >= 0, torch.exp(la[:, None, None] * diff.clamp(min=0)), 0.0).float()   # a^(t-s), [H, C, C]
    up = torch.exp(la[:, None] * (i + 1)).float()                                               # a^(t+1), [H, C]
    for b in range(len(cu) - 1):
        lo, hi = cu[b], cu[b + 1]
        S = torch.zeros(H, dv, dk, device=q.device) if s["S0"] is None else s["S0"][s["S0_index"][b]].clone()
        stops = sorted(set(range(CHUNK, hi - lo, CHUNK)) | set(s["ckpt"][b] if s["ckpt"] else []) | {hi - lo})
        marks = set(s["ckpt"][b]) if s["ckpt"] else set()
        at = 0
        for e in stops:
            n = e - at
            qc = q[lo + at:lo + e].transpose(0, 1).repeat_interleave(rep, 0)     # [H, n, dk]
            kc = k[lo + at:lo + e].transpose(0, 1).repeat_interleave(rep, 0)
            vc = v[lo + at:lo + e].transpose(0, 1)
            inter = torch.matmul(qc * up[:, :n, None], S.transpose(1, 2))
            intra = torch.matmul(torch.matmul(qc, kc.transpose(1, 2)) * D[:, :n, :n], vc)
            o[lo + at:lo + e] = ((inter + intra) * s["scale"]).transpose(0, 1)
            S = S * up[:, n - 1, None, None] + torch.matmul((vc * D[:, n - 1, :n, None]).transpose(1, 2), kc)
            at = e
            if e in marks:
                dumps.append(S)
        final.append(S)
    return _present(o=o.to(s["q"].dtype), S_final=torch.stack(final), ckpt_states=torch.stack(dumps) if dumps else None)


def _plain_step(s):
    q, k, v, alpha, states = s["q"].float(), s["k"].float(), s["v"].float(), s["alpha"], s["states"]
    rep = v.shape[1] // k.shape[1]
    live = s["slots"] >= 0
    idx = s["slots"].long().clamp(min=0)
    kk, qq = k.repeat_interleave(rep, 1), q.repeat_interleave(rep, 1)
    S = states[idx] * alpha[None, :, None, None] + v[..., :, None] * kk[..., None, :]
    o = (S * qq[..., None, :]).sum(-1) * s["scale"]
    # a padding row (slot -1) gives zeros and leaves the pool alone
    pad = torch.full_like(idx, states.shape[0])
    grown = torch.cat([states, states[:1]])
    grown[torch.where(live, idx, pad)] = S
    states.copy_(grown[:-1])
    return dict(o=torch.where(live[:, None, None], o, 0.0).to(s["q"].dtype), states=states)


def _plain_prefix(s):
    q, kt, vt, tail = s["q"], s["k_tail"], s["v_tail"], s["tail_len"]
    B, n, Hq, D = q.shape
    P, Hkv = s["k_prefix"].shape[:2]
    G, cap = Hq // Hkv, kt.shape[1]
    o = torch.empty(B, n, Hq, D, device=q.device)
    lse = torch.empty(B, n, Hq, device=q.device)
    j = torch.arange(cap, device=q.device)
    pos = tail[:, None] - n + torch.arange(n, device=q.device)                        # position of query i in the tail
    hide = (j[None, None, :] > pos[:, :, None]) | (j[None, None, :] >= tail[:, None, None])
    for h in range(Hkv):
        qh = q[:, :, h * G:(h + 1) * G].float() * s["scale"]                          # [B, n, G, D]
        a = torch.matmul(qh.reshape(-1, D), s["k_prefix"][:, h].float().T).reshape(B, n, G, P)
        c = torch.matmul(qh.reshape(B, n * G, D), kt[:, :, h].float().transpose(1, 2)).reshape(B, n, G, cap)
        c = c.masked_fill(hide[:, :, None, :], -math.inf)
        top = torch.maximum(a.amax(-1), c.amax(-1))
        a, c = torch.exp(a - top[..., None]), torch.exp(c - top[..., None])
        den = a.sum(-1) + c.sum(-1)
        num = torch.matmul(a.reshape(-1, P), s["v_prefix"][:, h].float()).reshape(B, n, G, D)
        num = num + torch.matmul(c.reshape(B, n * G, cap), vt[:, :, h].float()).reshape(B, n, G, D)
        o[:, :, h * G:(h + 1) * G] = num / den[..., None]
        lse[:, :, h * G:(h + 1) * G] = top + torch.log(den)
    return dict(o=o.to(q.dtype), lse=lse)


def run(s):
    op = s["case"]["op"]
    if own:
        import hybrid_model_recurrent_gb300 as gdn
        if op == "prefill":
            return _present(**gdn.gdn_linear_prefill(s["q"], s["k"], s["v"], s["alpha"], s["cu"], scale=s["scale"],
                                                     S0=s["S0"], S0_index=s["S0_index"], ckpt_pos=s["ckpt"]))
        if op == "step":
            o = gdn.gdn_linear_step(s["q"], s["k"], s["v"], s["alpha"], s["states"], slots=s["slots"],
                                    scale=s["scale"])
            return dict(o=o, states=s["states"])
        return gdn.gdn_prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], s["k_tail"], s["v_tail"], s["tail_len"],
                                        scale=s["scale"])
    return {"prefill": _plain_prefill, "step": _plain_step, "prefix": _plain_prefix}[op](s)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "prefill":
        H, Hk, dk, dv, B = case["H"], case["Hk"], case["dk"], case["dv"], case["B"]
        lens = _lens(case)
        T = sum(lens)
        dumps = sum(n // case["ckpt"] for n in lens) if case["ckpt"] else 0
        states = (B + dumps + (1 if case["fork"] else 0)) * H * dv * dk * 4
        # per token and head: the state's update and readout
        return dict(bytes=T * (2 * Hk * dk + 2 * H * dv) * size + states + 4 * H, flops=T * H * 4 * dk * dv)
    if case["op"] == "step":
        B, H, Hk, dk, dv = case["B"] - case["pad"], case["H"], case["Hk"], case["dk"], case["dv"]
        return dict(bytes=B * (2 * H * dk * dv * 4 + (2 * Hk * dk + 2 * H * dv) * size) + 4 * H + 4 * case["B"],
                    flops=B * H * 5 * dk * dv)
    B, n, Hq, Hkv, D, P, cap = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "P", "cap"))
    tail = (min(n, cap) + cap) / 2                                                     # the mean tail
    seen = tail - (n - 1) / 2 if tail >= n else tail / 2                               # and what a query sees of it
    return dict(bytes=int(2 * (P + B * tail) * Hkv * D * size + B * n * Hq * (2 * D * size + 4) + 4 * B),
                flops=int(4 * B * n * Hq * D * (P + seen)))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill":
        return _exact_prefill(s)
    if case["op"] == "step":
        live = [(i, j) for i, j in enumerate(s["slots"].tolist()) if j >= 0]
        H, Hk = s["v"].shape[1], s["k"].shape[1]
        of = torch.arange(H, device="cuda") // (H // Hk)
        o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
        states = s["states"].double()
        for i, j in live:
            new = s["alpha"].double()[:, None, None] * states[j] + torch.einsum(
                "hv,hk->hvk", s["v"][i].double(), s["k"][i].double()[of])
            states[j] = new
            o[i] = torch.einsum("hvk,hk->hv", new, s["q"][i].double()[of]) * s["scale"]
        return dict(o=o, states=states)
    B, n, Hq, Hkv, D, P, cap = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "P", "cap"))
    if 4 * B * n * Hq * D * (P + cap) > 4e12:
        return None
    G = Hq // Hkv
    o = torch.zeros(B, n, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, n, Hq, dtype=torch.float64, device="cuda")
    lens = s["tail_len"].tolist()
    for h in range(Hkv):
        kp, vp = s["k_prefix"][:, h].double(), s["v_prefix"][:, h].double()
        for b in range(B):
            keys = torch.cat([kp, s["k_tail"][b, :lens[b], h].double()])
            vals = torch.cat([vp, s["v_tail"][b, :lens[b], h].double()])
            qs = s["q"][b, :, h * G:(h + 1) * G].double()                              # [n, G, D]
            x = torch.einsum("igd,kd->igk", qs, keys) * s["scale"]
            ends = P + lens[b] - n + torch.arange(n, device="cuda")
            x = x.masked_fill(torch.arange(len(keys), device="cuda")[None, None] > ends[:, None, None], -math.inf)
            lse[b, :, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            o[b, :, h * G:(h + 1) * G] = torch.einsum("igk,kd->igd", torch.softmax(x, -1), vals)
    return dict(o=o, lse=lse)


def _exact_prefill(s):
    """The recurrence token by token, the sequences side by side (a sequence that has ended stands still)."""
    cu = s["cu"]
    B, lens = len(cu) - 1, [b - a for a, b in zip(cu, cu[1:])]
    H, dv, dk = s["v"].shape[1], s["v"].shape[2], s["k"].shape[2]
    order = sorted(range(B), key=lambda b: -lens[b])                                   # longest first
    of = torch.arange(H, device="cuda") // (H // s["k"].shape[1])
    alpha = s["alpha"].double()[:, None, None]
    S = torch.zeros(B, H, dv, dk, dtype=torch.float64, device="cuda")
    if s["S0"] is not None:
        S += s["S0"].double()[torch.tensor(s["S0_index"], device="cuda")]
    marks = {}
    total = 0
    for b in range(B):
        for c in (s["ckpt"][b] if s["ckpt"] else []):
            marks.setdefault(c, []).append((order.index(b), total))
            total += 1
    dumps = torch.empty(total, H, dv, dk, dtype=torch.float64, device="cuda")
    o = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
    first = torch.tensor([cu[b] for b in order], device="cuda")
    sorted_lens = [lens[b] for b in order]
    live = B
    for t in range(max(lens)):
        while sorted_lens[live - 1] <= t:
            live -= 1
        at = first[:live] + t
        qt, kt, vt = s["q"][at].double()[:, of], s["k"][at].double()[:, of], s["v"][at].double()
        Sl = S[:live]
        Sl.mul_(alpha).addcmul_(vt[..., :, None], kt[..., None, :])
        o[at] = torch.matmul(Sl, qt[..., None])[..., 0] * s["scale"]
        for row, slot in marks.get(t + 1, []):
            dumps[slot] = S[row]
    final = torch.empty_like(S)
    final[torch.tensor(order, device="cuda")] = S
    return _present(o=o, S_final=final, ckpt_states=dumps if total else None)
