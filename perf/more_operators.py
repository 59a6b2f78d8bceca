"""Cases for the operators around a paged cache in 8 bits: queries and keys prepared (norm of each head and
position rotation in one pass), keys and values appended to the cache, attention over it, and the upkeep of
its pages (forks of a prefix, growth, freeing, compaction).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) or, where ``own`` is
true, through the package's entry points.  ``exact`` evaluates the definition in 64 bits.

The cache: pages [L, N, 2, Hkv, page, D] in e4m3 (L layers, N pages, keys and values), scales [L, N, 2, Hkv] in
fp32, powers of two, one for each block (the tokens of a page for one head); table [R, W] holds each row's
pages in order, lens [R] its tokens, refs [N] how many rows hold a page (0: free).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decode step of a batch: narrow heads in full precision, pairs side by side, half of a head rotated
        dict(name="rotate_step_f32_67", op="rotate", T=67, Hq=16, Hk=16, D=64, rd=32, layout="interleaved", norm=True,
             stretch=1.0, far=100000, dtype="f32"),
        # the prompts of the serving workload (8 of 8192 tokens), positions stretched for a long context
        dict(name="rotate_prompts_8x8192", op="rotate", T=65536, Hq=32, Hk=8, D=128, rd=128, layout="half", norm=True,
             stretch=4.0, far=131072, dtype="bf16"),
        # one token of each request of a decode batch, three rows padding
        dict(name="append_step_67", op="append", B=67, new=1, had=2000, pad=3, Hkv=8, D=128, page=64, dtype="bf16"),
        # ragged new turns behind what each request already has, page ends inside them
        dict(name="append_turns_32x1999", op="append", B=32, new=1999, had=700, pad=0, Hkv=8, D=128, page=64, dtype="bf16"),
        # a few requests on short contexts: latency
        dict(name="attend_small_b4", op="attend", B=4, new=1, had=1096, pad=0, Hq=16, Hkv=2, D=128, page=16, dtype="bf16"),
        # a decode batch on long contexts, four query heads a key/value head
        dict(name="attend_decode_b64", op="attend", B=64, new=1, had=33792, pad=0, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16"),
        # new turns of up to 256 tokens on long contexts: bound by the products
        dict(name="attend_turns_b16", op="attend", B=16, new=256, had=17084, pad=0, Hq=32, Hkv=4, D=128, page=64,
             dtype="bf16"),
        # drafted tokens checked at once, in full precision, odd sizes, narrow heads
        dict(name="attend_draft_f32_b7", op="attend", B=7, new=4, had=2124, pad=0, Hq=8, Hkv=8, D=64, page=32,
             dtype="f32"),
        # a turn begins: a few rows forked from a prefix that ends with a page, room for their tokens
        dict(name="update_small_4", op="update", L=1, R=5, prefix=1024, grow=40, Hkv=2, D=128, page=16, free=20),
        # a batch forked from a prefix that ends inside a page: every row gets a copy of that page in every layer
        dict(name="update_fork_128", op="update", L=8, R=129, prefix=8191, grow=500, Hkv=8, D=128, page=64, free=300),
        # a small cache: every other row leaves, the rest moves together, the rows come back
        dict(name="compact_small_8", op="compact", L=1, R=8, tokens=300, Hkv=2, D=64, page=16, free=10),
        # the same of a large one
        dict(name="compact_64x2000", op="compact", L=8, R=64, tokens=2000, Hkv=8, D=128, page=64, free=100),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend", "update", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([32, 64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotate":
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4, 5])
        most = 65536 * 40 * 128 * 2 // ((Hq + Hk) * D * (2 if dtype == "bf16" else 4))
        return dict(op=op, T=_log_uniform(rng, 1, max(2, min(65536, most))), Hq=Hq, Hk=Hk, D=D,
                    rd=16 * rng.randint(0, D // 16), layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.7,
                    stretch=rng.choice([1.0, 1.0, 2.5, 8.0]), far=_log_uniform(rng, 100, 2 ** 22), dtype=dtype)
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "append":
        B = _log_uniform(rng, 1, 128)
        return dict(op=op, B=B, new=_log_uniform(rng, 1, max(2, 2 ** 22 // (B * Hkv * 8))), had=_log_uniform(rng, 1, 4000),
                    pad=rng.randint(0, B // 4), Hkv=Hkv, D=D, page=page, dtype=dtype)
    if op == "attend":
        G = rng.choice([1, 2, 4, 5, 8])
        new = rng.choice([1, 1, 1, 2, 4, 7, 33, 128, 300])
        B = _log_uniform(rng, 1, 64)
        if dtype == "f32":
            new, B = min(new, 33), min(B, 16)
        rows = B * new * Hkv * G
        had = _log_uniform(rng, 1, max(2, min(65536, 2 ** 30 // rows, 2 ** 23 // (B * Hkv))))
        return dict(op=op, B=B, new=new, had=had, pad=rng.randint(0, B // 4), Hq=Hkv * G, Hkv=Hkv, D=D, page=page,
                    dtype=dtype)
    L = rng.choice([1, 2, 4, 8])
    if op == "update":
        return dict(op=op, L=L, R=_log_uniform(rng, 2, 160), prefix=_log_uniform(rng, 1, 8000), grow=_log_uniform(rng, 1, 400),
                    Hkv=min(Hkv, 8), D=D, page=page, free=rng.randint(0, 300))
    R = _log_uniform(rng, 2, 64)
    return dict(op=op, L=L, R=R, tokens=_log_uniform(rng, 1, 2000), Hkv=min(Hkv, 8), D=D, page=page, free=rng.randint(0, 200))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g).to(dtype)


def _ints(case, lo, hi, n, salt):
    # lengths go with the case, not with the seed: other inputs have the same shapes
    r = np.random.RandomState((salt * 7919 + 31 * n + hi) % 2 ** 31)
    return r.randint(lo, hi + 1, n)


def _batch(case):
    """What each request of a batch adds, and the tokens that it has with them."""
    new = _ints(case, max(1, case["new"] // 8), case["new"], case["B"], 1)
    new[0] = case["new"]
    lens = _ints(case, max(1, case["had"] // 2), case["had"], case["B"], 2) + new
    return new, lens


def _channels(g, n, D):
    # some channels of keys are several times as large as the rest
    return 1.0 + 5.0 * (torch.rand(n, D, generator=g, device="cuda") < 0.05)


def _pool(g, L, N, Hkv, page, D):
    """A cache in use: contents in every page, blocks of different sizes."""
    x = torch.empty((L, N, 2, Hkv, page, D), device="cuda").normal_(generator=g)
    bits = x.mul_(64).clamp_(-448, 448).to(E4M3)
    return bits, torch.exp2(torch.randint(-7, -4, (L, N, 2, Hkv), generator=g, device="cuda").float())


def _tables(g, case, lens, spare, shared=0):
    """Rows of whole pages in a random order; the rows after the first begin with its first `shared` pages."""
    page, R = case["page"], len(lens)
    used = [-(-int(n) // page) for n in lens]
    own_pages = [n if r == 0 else n - shared for r, n in enumerate(used)]
    N = sum(own_pages) + spare
    order = torch.randperm(N, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    W = max(used) + 1
    table = np.full((R, W), -1, np.int32)
    refs = np.zeros(N, np.int32)
    at = 0
    for r, n in enumerate(used):
        first = list(table[0, :shared]) if r else []
        table[r, :n] = np.concatenate([np.array(first, np.int32), order[at:at + own_pages[r]]])
        at += own_pages[r]
        np.add.at(refs, table[r, :n], 1)
    return (torch.from_numpy(table).cuda(), torch.tensor([int(n) for n in lens], dtype=torch.int32, device="cuda"),
            torch.from_numpy(refs).cuda())


def _frequencies(rd, stretch):
    f = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / max(rd, 1))
    if stretch != 1.0 and rd:
        # slow pairs are stretched, fast ones are left, those between in part
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        f = f * keep + f / stretch * (1 - keep)
    return f.cuda()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "rotate":
        T, Hq, Hk, D, dt = case["T"], case["Hq"], case["Hk"], case["D"], DTYPES[case["dtype"]]
        # slices of one projection's output, as a model has them
        qkv = _normal(g, (T, (Hq + 2 * Hk) * D), dt)
        s.update(q=qkv[:, :Hq * D].unflatten(1, (Hq, D)), k=qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)),
                 pos=torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32),
                 freq=_frequencies(case["rd"], case["stretch"]), mscale=0.1 * math.log(case["stretch"]) + 1.0,
                 qw=(1 + 0.1 * _normal(g, (D,))).to(dt) if case["norm"] else None,
                 kw=(1 + 0.1 * _normal(g, (D,))).to(dt) if case["norm"] else None, eps=1e-6 if case["norm"] else None)
        return s
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    if op in ("append", "attend"):
        new, lens = _batch(case)
        B, dt = case["B"], DTYPES[case["dtype"]]
        table, lens_d, refs = _tables(g, case, [9] + list(lens), 3)                    # row 0 has no part in the batch
        rows = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
        if case["pad"]:
            rows[B - case["pad"]:] = -1
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pages, scales = _pool(g, 1, refs.shape[0], Hkv, page, D)
        s.update(pages=pages, scales=scales, table=table, lens=lens_d, refs=refs, rows=rows, cu=torch.from_numpy(cu).cuda(),
                 max_new=int(max(new)), max_len=int(max(lens)))
        T = int(cu[-1])
        if op == "append":
            kv = _normal(g, (T, 2 * Hkv, D), dt)
            s.update(k=(kv[:, :Hkv] * _channels(g, Hkv, D)).to(dt), v=kv[:, Hkv:])
        else:
            s.update(q=_normal(g, (T, case["Hq"], D), dt), scale=D ** -0.5)
        return s
    L, R = case["L"], case["R"]
    if op == "update":
        # row 0 is the prefix; the others have forks of it with tokens of their own
        grow = [0] + [int(x) for x in _ints(case, max(1, case["grow"] // 2), case["grow"], R - 1, 3)]
        whole = case["prefix"] // page
        lens = [case["prefix"]] + [case["prefix"] + n for n in grow[1:]]
        need = sum(-(-n // page) + 1 for n in grow)
        table, lens_d, refs = _tables(g, case, lens, case["free"] + need, whole)
        s.update(drop=None, src=torch.zeros(R - 1, dtype=torch.int32, device="cuda"),
                 dst=torch.arange(1, R, dtype=torch.int32, device="cuda"), grow=torch.tensor(grow, dtype=torch.int32, device="cuda"))
    else:
        lens = [int(x) for x in _ints(case, max(1, case["tokens"] // 2), case["tokens"], R, 4)]
        table, lens_d, refs = _tables(g, case, lens, case["free"])
        every = torch.arange(R, dtype=torch.int32, device="cuda")
        s.update(turn=0, halves=[every[i::2].contiguous() for i in (1, 0)],
                 back=[torch.where(every % 2 == i, lens_d, 0).to(torch.int32) for i in (1, 0)])
    pages, scales = _pool(g, L, refs.shape[0], Hkv, page, D)
    s.update(pages=pages, scales=scales, table=table, lens=lens_d, refs=refs)
    return s


# ---- plain forms ---------------------------------------------------------------------------------------


def _plain_rotate(s):
    case = s["case"]
    rd, h = case["rd"], case["rd"] // 2
    a = s["pos"].double()[:, None] * s["freq"][None]                                  # far positions: 64 bits
    a = torch.remainder(a, 2 * math.pi)
    cos, sin = (torch.cos(a) * s["mscale"]).float()[:, None], (torch.sin(a) * s["mscale"]).float()[:, None]

    def one(x, w):
        y = x.float()
        if s["eps"] is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        if case["layout"] == "half":
            u, v = y[..., :h], y[..., h:rd]
            turned = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
        else:
            u, v = y[..., 0:rd:2], y[..., 1:rd:2]
            turned = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
        return torch.cat([turned, y[..., rd:]], -1).to(x.dtype)

    return dict(q=one(s["q"], s["qw"]), k=one(s["k"], s["kw"]))


def _live_rows(s):
    """The batch's rows of the table, their tokens and their new ones (none for padding)."""
    rows = s["rows"].long()
    live = rows >= 0
    at = rows.clamp(min=0)
    n = torch.where(live, s["cu"][1:] - s["cu"][:-1], 0).long()
    return live, at, s["lens"][at].long() * live, n


def _plain_append(s):
    page = s["case"]["page"]
    live, at, lens, n = _live_rows(s)
    start = lens - n
    P = (s["max_new"] + page - 2) // page + 1                                         # pages that a request may touch
    i = start[:, None] // page + torch.arange(P, device="cuda")                        # [B, P] page of the row
    touched = (i * page < lens[:, None]) & (n[:, None] > 0)
    pg = s["table"][at].long().gather(1, i.clamp(max=s["table"].shape[1] - 1))
    pos = i[..., None] * page + torch.arange(page, device="cuda")                      # [B, P, page] position
    fresh = (pos >= start[:, None, None]) & (pos < lens[:, None, None])
    old = pos < start[:, None, None]
    tok = (s["cu"][:-1].long()[:, None, None] + pos - start[:, None, None]).clamp(0, len(s["k"]) - 1)
    x = torch.stack([s["k"], s["v"]], 1)[tok].float()                                  # [B, P, page, 2, H, D]
    x = x.permute(0, 1, 3, 4, 2, 5) * fresh[:, :, None, None, :, None]
    pg_ok = torch.where(touched, pg, 0)
    pages, scales = s["pages"][0], s["scales"][0]
    had = pages.view(torch.uint8)[pg_ok].view(E4M3).float()
    was = scales[pg_ok]
    f, e = torch.frexp(x.abs().amax((-1, -2)))
    e = torch.where(f == 0, -126, e - 8 - (f <= 0.875).to(e.dtype)).clamp(-126, 120)   # 448 = 0.875 * 2^9
    new_scale = torch.exp2(e.double()).float()
    some_old = old.any(-1)[:, :, None, None]
    scale = torch.where(some_old, torch.maximum(new_scale, was), new_scale)
    value = torch.where(old[:, :, None, None, :, None], had * (was / scale)[..., None, None], x / scale[..., None, None])
    keep = ~(fresh | old)[:, :, None, None, :, None]
    value = torch.where(keep, had, value).to(E4M3)
    t = touched.nonzero(as_tuple=True)
    pages.view(torch.uint8)[pg[t]] = value.view(torch.uint8)[t]
    scales[pg[t]] = scale[t]
    return dict(pages=s["pages"], scales=s["scales"])


def _plain_attend(s):
    case = s["case"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    G = Hq // Hkv
    live, at, lens, n = _live_rows(s)
    B, m = len(at), s["max_new"]
    W = -(-s["max_len"] // page)
    pg = s["table"][at, :W].long().clamp(min=0)
    x = s["pages"][0].view(torch.uint8)[pg].view(E4M3).float() * s["scales"][0][pg][..., None, None]  # [B, W, 2, H, page, D]
    k, v = (x[:, :, c].transpose(1, 2).reshape(B, Hkv, W * page, D) for c in (0, 1))
    del x
    i = torch.arange(m, device="cuda")
    tok = (s["cu"][:-1].long()[:, None] + i).clamp(max=len(s["q"]) - 1)                 # [B, m]
    q = s["q"][tok].float().view(B, m, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, m * G, D)
    a = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    last = torch.where(live[:, None], (lens - n)[:, None] + i, -1)                     # last token that a query sees
    a = a.view(B, Hkv, m, G, W * page)
    a.masked_fill_((torch.arange(W * page, device="cuda") > last[..., None])[:, None, :, None], -math.inf)
    top = a.amax(-1, keepdim=True).clamp(min=-3e38)
    a = a.sub_(top).exp_()
    den = a.sum(-1, keepdim=True)
    lse = torch.where(den > 0, top + torch.log(den), -math.inf)[..., 0]                # [B, H, m, G]
    y = torch.matmul(a.view(B, Hkv, m * G, -1), v).view(B, Hkv, m, G, D) / den.clamp(min=1e-38)
    some = i < (s["cu"][1:] - s["cu"][:-1])[:, None]
    o = torch.zeros(s["q"].shape, device="cuda")
    out = torch.zeros(s["q"].shape[:2], device="cuda")
    b, j = some.nonzero(as_tuple=True)
    o[tok[b, j]] = y.permute(0, 2, 1, 3, 4).reshape(B, m, Hq, D)[b, j]
    out[tok[b, j]] = lse.permute(0, 2, 1, 3).reshape(B, m, Hq)[b, j]
    return dict(o=o.to(s["q"].dtype), lse=out)


def _plain_update(s, drop, src, dst, grow):
    page, table, refs = s["case"]["page"], s["table"], s["refs"]
    lens = s["lens"].long()
    R, W = table.shape
    N = len(refs)
    w = torch.arange(W, device="cuda")

    def count(of, by):
        used = w < (-(-lens // page))[:, None]
        refs.index_add_(0, table.long().clamp(0, N - 1).flatten(), (used & of[:, None]).flatten().to(refs.dtype) * by)

    gone = torch.zeros(R, dtype=torch.bool, device="cuda")
    for rows in (drop, dst):
        if rows is not None:
            gone[rows.long()] = True
    count(gone, -1)
    lens[gone] = 0
    if src is not None:
        table[dst.long()] = table[src.long()]
        lens[dst.long()] = lens[src.long()]
        forked = torch.zeros_like(gone)
        forked[dst.long()] = True
        count(forked, 1)
    if grow is not None:
        grow = grow.long()
        have, after = -(-lens // page), lens + grow
        last = table.long().gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0)
        cow = (grow > 0) & (lens % page > 0) & (refs[last] > 1)
        need = torch.where(after <= W * page, -(-after // page) - have + cow, 0)
        free = refs == 0
        cum = need.cumsum(0)
        served = (after <= W * page) & ((need == 0) | (cum <= free.sum()))
        ranks = torch.full((N + 1,), N, dtype=torch.long, device="cuda")
        ranks[torch.where(free, free.long().cumsum(0) - 1, N)] = torch.arange(N, device="cuda")
        first = cum - need
        copied = served & cow
        old = last[copied]
        fresh = ranks[first[copied]]
        refs.index_add_(0, old, torch.full_like(old, -1, dtype=refs.dtype))
        c = copied.nonzero(as_tuple=True)[0]
        table[c, have[c] - 1] = fresh.to(table.dtype)
        s["pages"].view(torch.uint8)[:, fresh] = s["pages"].view(torch.uint8)[:, old]
        s["scales"][:, fresh] = s["scales"][:, old]
        take = first[:, None] + cow[:, None] + w - have[:, None]
        added = served[:, None] & (w >= have[:, None]) & (w < (-(-after // page))[:, None])
        table.copy_(torch.where(added, ranks[take.clamp(0, N)].to(table.dtype), table))
        lens = torch.where(served, after, lens)
        refs[fresh] = 1
        refs[table[added].long()] = 1
        s["lens"].copy_(lens)
        return torch.where(served, grow, -1).to(torch.int32)
    s["lens"].copy_(lens)


def _plain_compact(s):
    refs, table, page = s["refs"], s["table"], s["case"]["page"]
    N = len(refs)
    live = refs > 0
    n = live.sum()
    i = torch.arange(N, device="cuda")
    movers, holes = (live & (i >= n)).nonzero(as_tuple=True)[0], (~live & (i < n)).nonzero(as_tuple=True)[0]
    to = i.clone()
    to[movers] = holes
    s["pages"].view(torch.uint8)[:, holes] = s["pages"].view(torch.uint8)[:, movers]
    s["scales"][:, holes] = s["scales"][:, movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    used = torch.arange(table.shape[1], device="cuda") < (-(-s["lens"].long() // page))[:, None]
    table.copy_(torch.where(used, to[table.long().clamp(0, N - 1)].to(table.dtype), table))
    return n.to(torch.int32).reshape(1)


def _kept(s, **more):
    return dict(pages=s["pages"], scales=s["scales"], table=s["table"], lens=s["lens"], refs=s["refs"], **more)


def run(s):
    op = s["case"]["op"]
    if own:
        import hybrid_model_recurrent_gb300 as gdn
        if op == "rotate":
            q, k = gdn.gdn_qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], layout=s["case"]["layout"], q_weight=s["qw"],
                                        k_weight=s["kw"], eps=s["eps"], mscale=s["mscale"])
            return dict(q=q, k=k)
        c = gdn.PagedCache(s["pages"], s["scales"], s["table"], s["lens"], s["refs"])
        if op == "append":
            gdn.gdn_cache_append(s["k"], s["v"], c, s["cu"], rows=s["rows"], max_new=s["max_new"])
            return dict(pages=s["pages"], scales=s["scales"])
        if op == "attend":
            return gdn.gdn_paged_attention(s["q"], c, s["cu"], rows=s["rows"], max_new=s["max_new"], max_len=s["max_len"],
                                           scale=s["scale"])
        if op == "update":
            return _kept(s, granted=gdn.gdn_cache_update(c, fork_from=s["src"], fork_to=s["dst"], grow=s["grow"]))
        turn = s["turn"]
        s["turn"] = 1 - turn
        gdn.gdn_cache_update(c, drop=s["halves"][turn])
        n = gdn.gdn_cache_compact(c)
        return _kept(s, live=n, granted=gdn.gdn_cache_update(c, grow=s["back"][turn]))
    if op == "update":
        return _kept(s, granted=_plain_update(s, s["drop"], s["src"], s["dst"], s["grow"]))
    if op == "compact":
        # every other row leaves and comes back with as many tokens, the other half the next time
        turn = s["turn"]
        s["turn"] = 1 - turn
        _plain_update(s, s["halves"][turn], None, None, None)
        n = _plain_compact(s)
        return _kept(s, live=n, granted=_plain_update(s, None, None, None, s["back"][turn]))
    return {"rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend}[op](s)


def work(case):
    op, D = case["op"], case["D"]
    if op == "rotate":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["T"] * (case["Hq"] + case["Hk"]) * D
        return dict(bytes=2 * n * size + 4 * case["T"], flops=n * (4 + 3 * (case["rd"] / D)))
    block = case["Hkv"] * case["page"] * D
    if op in ("append", "attend"):
        size = 2 if case["dtype"] == "bf16" else 4
        new, lens = _batch(case)
        B = case["B"]
        live = B - case["pad"]
        new, lens = [int(x) for x in new], [int(x) for x in lens]
        if op == "append":
            T = sum(new[:live])
            return dict(bytes=T * 2 * case["Hkv"] * D * (size + 1) + 8 * B, flops=T * 4 * case["Hkv"] * D)
        seen = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(new[:live], lens))
        T = sum(new)
        tokens = sum(lens[:live])
        pages = sum(-(-k // case["page"]) for k in lens[:live])
        return dict(bytes=2 * tokens * case["Hkv"] * D + 8 * pages * case["Hkv"] + T * case["Hq"] * (2 * D * size + 4),
                    flops=4 * seen * case["Hq"] * D)
    L, R = case["L"], case["R"]
    if op == "update":
        copies = R - 1 if case["prefix"] % case["page"] else 0
        held = -(-case["prefix"] // case["page"])
        return dict(bytes=copies * L * 2 * (2 * block + 8 * case["Hkv"]) + R * held * 4 * 2, flops=0)
    lens = _ints(case, max(1, case["tokens"] // 2), case["tokens"], R, 4)
    held = [-(-int(n) // case["page"]) for n in lens]
    moved = min(sum(held[0::2]), sum(held[1::2]))                                      # from behind those that left
    return dict(bytes=moved * L * 2 * (2 * block + 8 * case["Hkv"]) + sum(held) * 8, flops=0)


# ---- the definitions in 64 bits ------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        return dict(q=_exact_rotate(s, s["q"], s["qw"]), k=_exact_rotate(s, s["k"], s["kw"]))
    if op == "append":
        return _exact_append(s)
    if op == "attend":
        return _exact_attend(s)
    return None                                                                        # whole numbers and copies


def _exact_rotate(s, x, w):
    rd = s["case"]["rd"]
    x = x.double()
    if s["eps"] is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.double()
    half = s["case"]["layout"] == "half"
    y = x.clone()
    if rd:
        p = torch.arange(rd // 2, device="cuda")
        one, two = (p, p + rd // 2) if half else (2 * p, 2 * p + 1)
        turn = torch.polar(torch.full((1,), s["mscale"], dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None, None] * s["freq"])
        z = torch.complex(x[..., one], x[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_append(s):
    page, H = s["case"]["page"], s["case"]["Hkv"]
    pages, scales = s["pages"].double()[0], s["scales"].double()[0]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    step = 448.0

    def e4m3(x):
        # nearest value with three bits behind the first, or a multiple of 2^-9
        _, e = torch.frexp(x)
        unit = torch.exp2((e - 4).clamp(min=-9).double())
        return torch.round(x / unit) * unit                                            # round: ties to even

    for b, r in enumerate(s["rows"].tolist()):
        if r < 0:
            continue
        at, left = lens[r] - (cu[b + 1] - cu[b]), cu[b]
        while at < lens[r]:
            pg, first = table[r][at // page], at % page
            n = min(page - first, lens[r] - at)
            for c, x in ((0, s["k"]), (1, s["v"])):
                x = x[left:left + n].double().transpose(0, 1)                          # [H, n, D]
                top = x.abs().amax((1, 2))
                e = torch.where(top > 0, torch.ceil(torch.log2(top / step)), torch.full_like(top, -126.0)).clamp(-126, 120)
                e = torch.where(top > step * torch.exp2(e), e + 1, e)                  # where the logarithm was rounded
                e = torch.where(top <= step * torch.exp2(e - 1), e - 1, e).clamp(min=-126)
                scale = torch.exp2(e)
                if first:
                    was = scales[pg, c]
                    scale = torch.maximum(scale, was)
                    pages[pg, c, :, :first] = e4m3(pages[pg, c, :, :first] * (was / scale)[:, None, None])
                pages[pg, c, :, first:first + n] = e4m3(x / scale[:, None, None])
                scales[pg, c] = scale
            at, left = at + n, left + n
    return dict(pages=pages[None], scales=scales[None])


def _exact_attend(s):
    case = s["case"]
    if work(case)["flops"] > 4e12:
        return None
    page, Hkv, D, G = case["page"], case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, r in enumerate(s["rows"].tolist()):
        n = cu[b + 1] - cu[b]
        if r < 0 or n == 0:
            continue
        pg = s["table"][r, :-(-lens[r] // page)].long()
        kv = s["pages"][0].view(torch.uint8)[pg].view(E4M3).double() * s["scales"][0][pg].double()[..., None, None]
        ends = lens[r] - n + torch.arange(n, device="cuda")
        hide = torch.arange(lens[r], device="cuda")[None, None] > ends[:, None, None]
        for h in range(Hkv):
            k, v = (kv[:, c, h].reshape(-1, D)[:lens[r]] for c in (0, 1))
            q = s["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()
            x = torch.einsum("igd,kd->igk", q, k) * s["scale"]
            x = x.masked_fill(hide, -math.inf)
            lse[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            o[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("igk,kd->igd", torch.softmax(x, -1), v)
    return dict(o=o, lse=lse)
