"""What the tests of include/gdn_cache.h share: caches with known contents, and the definitions in 64 bits."""
import math

import torch

import hybrid_model_recurrent_gb300 as gdn

E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24
NAN_BYTE = 0x7F


def round_e4m3(x):
    """The nearest e4m3 value of x (64 bits, at most 448 in size), ties to even, from the format alone: three bits behind the
    first, multiples of 2^-9 at least."""
    _, e = torch.frexp(x)
    unit = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / unit) * unit


def block_scale(top):
    """The least power of two with top <= 448 times it, in 2^-126 .. 2^120."""
    return next((2.0 ** e for e in range(-126, 120) if top <= 448 * 2.0 ** e), 2.0 ** 120)


def make_cache(lens, *, N=None, page=16, H=2, D=64, L=1, W=None, seed=0, gain=1.0, poison=True, spread=3):
    """Rows of `lens` tokens in randomly placed pages; what belongs to no row's tokens is NaN, scales of free pages too."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    used = [-(-n // page) for n in lens]
    N = N or sum(used) + 3
    W = W or max(max(used), 1) + 2
    order = torch.randperm(N, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), W), -7, dtype=torch.int32)
    refs = torch.zeros(N, dtype=torch.int32)
    x = torch.randn(L, N, 2, H, page, D, generator=g, device="cuda") * 60
    pages = x.clamp(-448, 448).to(E4M3).view(torch.uint8)
    scales = torch.exp2(torch.randint(-6 - spread, -5 + spread, (L, N, 2, H), generator=g, device="cuda").float()) * gain
    keep = torch.zeros(N, page, dtype=torch.bool)
    for r, n in enumerate(lens):
        for w in range(used[r]):
            pg = order.pop()
            table[r, w], refs[pg] = pg, 1
            keep[pg, :min(page, n - w * page)] = True
    if poison:
        keep = keep.cuda()
        pages = torch.where(keep[None, :, None, None, :, None], pages, NAN_BYTE)
        scales = torch.where(keep.any(1)[None, :, None, None], scales, math.nan)
    return gdn.PagedCache(pages.contiguous().view(E4M3), scales.contiguous(), table.cuda(),
                          torch.tensor(lens, dtype=torch.int32, device="cuda"), refs.cuda())


def row_values(c, r, n, layer=0):
    """Keys and values [n, H, D] of row r's first n tokens, in 64 bits."""
    page = c.page_size
    pg = c.table[r, :-(-n // page)].long()
    x = c.pages.view(torch.uint8)[layer, pg].view(E4M3).double() * c.scales[layer, pg].double()[..., None, None]
    return [x[:, kv].permute(0, 2, 1, 3).reshape(-1, x.shape[2], x.shape[4])[:n] for kv in (0, 1)]   # x [pages, 2, H, page, D]


def check_attention(c, q, cu, *, rows=None, layer=0, scale=None, cut=0.0, lens=None, **kw):
    """The call's outputs against the definition in 64 bits.  Tolerances (u = 2^-24): a score (times log2 e) is a sum of D
    products and three scalings, off by e = (D + 6) u scale sum |q||k| + 6 u |x|, and fp32 queries by 2^-22 of sum |q||k| more;
    a weight by 2 e + 2^-21 and its rounding (half a step: 2^-11 in f16, 2^-22 in two; at least 2^-32 of the largest: half
    of f16's last step where that one is held as 2^7); numerator and denominator add N terms; the output is rounded once.
    `cut`: what blocks far below the largest of their tile may lose, relative to the largest value (tensor cores: 2^-24)."""
    T, Hq, D = q.shape
    H = c.pages.shape[3]
    G = Hq // H
    r = gdn.gdn_paged_attention(q, c, cu, rows=rows, layer=layer, scale=scale, **kw)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    scale = D ** -0.5 if scale is None else scale
    bf = q.dtype == torch.bfloat16
    out_step = 2.0 ** -8 if bf else U
    weight_step = 2.0 ** -11 if bf else 2.0 ** -22
    ends = cu.tolist()
    lens = c.lens.tolist() if lens is None else lens
    at = list(range(len(ends) - 1)) if rows is None else rows.tolist()
    for b, row in enumerate(at):
        n = ends[b + 1] - ends[b]
        if n == 0:
            continue
        o = r["o"][ends[b]:ends[b + 1]].double().reshape(n, H, G, D)
        lse = r["lse"][ends[b]:ends[b + 1]].double().reshape(n, H, G)
        N = lens[row] if 0 <= row < len(lens) else 0
        seen = torch.clamp(N - n + torch.arange(1, n + 1, device="cuda"), min=0)
        empty = seen == 0
        assert not o[empty].any() and (lse[empty] == -math.inf).all(), (b, "a query that sees nothing")
        live = (~empty).nonzero()[:, 0]
        if not len(live):
            continue
        k, v = row_values(c, row, N, layer)
        qs = q[ends[b]:ends[b + 1]].double().reshape(n, H, G, D)[live]
        x = torch.einsum("ihgd,khd->ihgk", qs, k) * scale
        size = torch.einsum("ihgd,khd->ihgk", qs.abs(), k.abs()) * abs(scale)
        hide = (torch.arange(N, device="cuda")[None] >= seen[live][:, None])[:, None, None]
        x, size = x.masked_fill(hide, -math.inf), size.masked_fill(hide, 0.0)
        p = torch.softmax(x, -1)
        e = ((D + 6) * U + (0 if bf else 2.0 ** -22)) * size.amax(-1) + 6 * U * x.masked_fill(hide, 0.0).abs().amax(-1)
        rel = 2 * (2 * e + 2.0 ** -21 + N * U) + weight_step
        vmax = v.abs().amax((0, 2))[None, :, None]
        want = torch.einsum("ihgk,khd->ihgd", p, v)
        tol = rel[..., None] * torch.einsum("ihgk,khd->ihgd", p, v.abs()) + ((N * 2.0 ** -32 + cut) * vmax)[..., None]
        tol = tol + out_step * (want.abs() + tol) + 1e-37
        off = (o[live] - want).abs()
        assert torch.isfinite(o[live]).all(), b
        assert (off <= tol).all(), (b, float((off / tol).max()))
        ref = torch.logsumexp(x, -1)
        tol = 2 * e + 2.0 ** -21 + N * U + 2 * U * (ref.abs() + x.masked_fill(hide, 0.0).abs().amax(-1)) + 1e-37
        off = (lse[live] - ref).abs()
        assert (off <= tol).all(), (b, "lse", float((off / tol).max()))
    return r
