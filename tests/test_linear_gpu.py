"""Linear attention with a decay for each head on the GPU against the recurrence in 64 bits.

Tolerances, from the roundings (u = 2^-24, half a step of fp32; half a step of bf16 is 2^-8):
 * a state element takes at most two fp32 roundings a token of a value bounded by A, the same recurrence over absolute
   values, and, where products run on split operands, 2^-16 of each added term: E_t = alpha (1 + 2^-16) E_{t-1}
   + 2 u A_t + 2^-16 |v||k|;
 * a readout adds E |q|, d_k + 130 additions of A |q|, and, where a chunk's operands are rounded to bf16 (bf16 in and
   out), 2^-8 of every term once for the state's part and once for the tokens' part: both are within A |q|;
 * the output's own rounding."""
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def make(lens, H, Hk, dk, dv, dtype, seed=0, alpha=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)

    def n(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    q, k = n(T, Hk, dk), n(T, Hk, dk)
    q, k = (x / x.norm(dim=-1, keepdim=True).clamp(min=1e-20) for x in (q, k))
    a = torch.tensor(alpha if alpha is not None else [1.0 - 2.0 ** -(1 + i % 9) for i in range(H)], device="cuda")
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return q.to(dtype), k.to(dtype), n(T, H, dv).to(dtype), a.float(), cu, g


def reference(q, k, v, alpha, cu, S0, scale, ckpt, rounded):
    """(o, o_tol, S_final, S_tol, ckpt, ckpt_tol) in 64 bits, token by token."""
    B, H, dv, dk = len(cu) - 1, v.shape[1], v.shape[2], k.shape[2]
    of = torch.arange(H, device="cuda") // (H // k.shape[1])
    al = alpha.double()[:, None, None]
    o = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    ot = torch.zeros_like(o)
    fin, fint, cks, ckts = [], [], [], []
    for b in range(B):
        S = torch.zeros(H, dv, dk, dtype=torch.float64, device="cuda") if S0[b] is None else S0[b].double().clone()
        A, E = S.abs(), torch.zeros_like(S)
        for t in range(cu[b], cu[b + 1]):
            kk, qq, vv = k[t].double()[of], q[t].double()[of], v[t].double()
            w = vv[:, :, None] * kk[:, None, :]
            S = al * S + w
            A = al * A + w.abs()
            E = al * E * (1 + 2.0 ** -16) + 2 * U * A + 2.0 ** -16 * w.abs()
            Aq = (A * qq.abs()[:, None, :]).sum(-1)
            o[t] = (S * qq[:, None, :]).sum(-1) * scale
            ot[t] = abs(scale) * ((E * qq.abs()[:, None, :]).sum(-1) + Aq * ((dk + 130) * U + (2.0 ** -8 if rounded else 0)))
            if ckpt is not None and t + 1 - cu[b] in ckpt[b]:
                cks.append(S)
                ckts.append(E)
        fin.append(S)
        fint.append(E)
    return o, ot, torch.stack(fin), torch.stack(fint), cks, ckts


def close(got, want, tol, what):
    out = 2.0 ** -8 if got.dtype == BF else U
    bound = tol + (want.abs() + tol) * out + 1e-30
    err = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all(), what
    assert (err <= bound).all(), f"{what}: {(err / bound).max().item():.3g} of the tolerance"


def check(lens, H, Hk, dk, dv, dtype, out_dtype=None, *, S0=None, index=None, ckpt=None, scale=1.0, alpha=None, seed=0,
          readout=True, fused=False):
    q, k, v, a, cu, g = make(lens, H, Hk, dk, dv, dtype, seed, alpha)
    if fused:   # slices of one projection's output, with a gap between them
        T = cu[-1]
        width = 2 * Hk * dk + H * dv + 64
        big = torch.full((T, width), float("nan"), dtype=dtype, device="cuda")
        parts, at = [], 0
        for x in (q, k, v):
            n = x.shape[1] * x.shape[2]
            big[:, at:at + n] = x.reshape(T, n)
            parts.append(big[:, at:at + n].unflatten(1, x.shape[1:]))
            at += n + 16
        q, k, v = parts
    pool = None if S0 is None else torch.randn(S0, H, dv, dk, generator=g, device="cuda")
    r = gdn.gdn_linear_prefill(q, k, v, a, cu, scale=scale, S0=pool, S0_index=index, ckpt_pos=ckpt, out_dtype=out_dtype,
                               readout=readout)
    B = len(lens)
    init = [None] * B if pool is None else [None if (index or range(B))[b] < 0 else pool[(index or range(B))[b]] for b in range(B)]
    rounded = dtype == BF and (out_dtype or dtype) == BF
    o, ot, fin, fint, cks, ckts = reference(q, k, v, a, cu, init, scale, ckpt, rounded)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    if readout:
        close(r["o"], o, ot, "o")
    else:
        assert r["o"] is None
    close(r["S_final"], fin, fint, "S_final")
    for i, (c, t) in enumerate(zip(cks, ckts)):
        close(r["ckpt_states"][i], c, t, f"checkpoint {i}")
    return r


DIMS = [(128, 128), (64, 64), (32, 32), (64, 128), (128, 64), (32, 128)]


@pytest.mark.parametrize("dtype, out", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("dk, dv", DIMS)
def test_prefill_sizes(dk, dv, dtype, out):
    check([0, 1, 2, 63, 64, 65, 127, 128, 129, 257], 4, 2, dk, dv, dtype, out, S0=12, scale=0.5,
          index=[3, 3, -1, 0, 11, 5, 3, 3, 1, 2])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk, dv", DIMS[:3])
def test_prefill_checkpoints(dk, dv, dtype):
    """At the first and last token, next to one another, on and beside the tiles' edges."""
    check([300, 0, 131, 1], 3, 3, dk, dv, dtype, S0=4,
          ckpt=[[1, 2, 63, 64, 65, 127, 128, 130, 256, 300], [], [128, 129, 131], [1]])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk, dv", DIMS[:4])
def test_prefill_decays(dk, dv, dtype):
    """No decay, total decay, and decays whose powers leave the fp32 range inside a chunk."""
    check([200, 77], 6, 2, dk, dv, dtype, S0=2, alpha=[1.0, 0.0, 1e-30, 0.5, 0.999, 2.0 ** -126])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk, dv", DIMS[:3])
@pytest.mark.parametrize("readout", [True, False])
def test_prefill_split_scan(dk, dv, dtype, readout):
    """Few long scans, cut into segments: initial states, checkpoints inside and at the ends of segments."""
    lens = [4500, 1, 2049]
    B, H = len(lens), 2
    cu = [0, 4500, 4501, 6550]
    pr = gdn._LinearProblem()
    pr.num_seqs, pr.num_heads, pr.num_qk_heads, pr.d_k, pr.d_v, pr.scale = B, H, 1, dk, dv, 1.0
    c = gdn._i64(cu)
    pr.cu_seqlens, pr.qkv_dtype, pr.out_dtype = gdn._p64(c), gdn._dtype_code(dtype), gdn._dtype_code(dtype)
    import ctypes
    assert gdn.lib().gdn_linear_scratch_bytes(ctypes.byref(pr)) > 0
    check(lens, H, 1, dk, dv, dtype, S0=3, alpha=[1.0, 0.97], ckpt=[[512, 513, 1000, 4500], [1], [2048]], readout=readout)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk, dv", DIMS[:3])
def test_prefill_strided_rows(dk, dv, dtype):
    check([70, 200], 4, 2, dk, dv, dtype, fused=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk, dv", DIMS[:3])
def test_prefill_sequences_do_not_mix(dk, dv, dtype):
    """A neighbour full of infinities and NaN leaves a sequence's results alone, bit for bit."""
    lens, H = [129, 50, 200], 2
    q, k, v, a, cu, _ = make(lens, H, H, dk, dv, dtype)
    ref = gdn.gdn_linear_prefill(q, k, v, a, cu)
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[129:179] = bad
    got = gdn.gdn_linear_prefill(q, k, v, a, cu)
    keep = [i for i in range(cu[-1]) if not 129 <= i < 179]
    assert torch.equal(got["o"][keep], ref["o"][keep])
    assert torch.equal(got["S_final"][[0, 2]], ref["S_final"][[0, 2]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_many_jobs(dtype):
    """More sequences than one launch's job table holds."""
    check([1 + i % 5 for i in range(401)], 2, 1, 64, 64, dtype, S0=2, index=[i % 3 - 1 for i in range(401)])


def test_prefill_on_another_stream():
    q, k, v, a, cu, _ = make([3000], 4, 4, 128, 128, BF)
    ref = gdn.gdn_linear_prefill(q, k, v, a, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = gdn.gdn_linear_prefill(q, k, v, a, cu, stream=s)
    s.synchronize()
    assert torch.equal(got["o"], ref["o"]) and torch.equal(got["S_final"], ref["S_final"])


def test_prefill_continues_and_repeats():
    """The state of a first half continues the second half to the whole (to rounding), and a call repeats bit for bit."""
    q, k, v, a, cu, _ = make([1000], 8, 8, 128, 128, BF)
    whole = check([1000], 8, 8, 128, 128, BF)
    again = gdn.gdn_linear_prefill(q, k, v, a, cu)
    assert torch.equal(again["o"], whole["o"]) and torch.equal(again["S_final"], whole["S_final"])
    first = gdn.gdn_linear_prefill(q[:384], k[:384], v[:384], a, [0, 384])
    second = gdn.gdn_linear_prefill(q[384:], k[384:], v[384:], a, [0, 616], S0=first["S_final"])
    assert (second["S_final"] - whole["S_final"]).abs().max() <= 2.0 ** -14 * whole["S_final"].abs().max()


# ---- one token a request ------------------------------------------------------------------


def step_reference(q, k, v, alpha, states, slots, scale):
    H, dk = v.shape[1], k.shape[2]
    of = torch.arange(H, device="cuda") // (H // k.shape[1])
    new, tol = states.double().clone(), torch.zeros_like(states, dtype=torch.float64)
    o = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    ot = torch.zeros_like(o)
    for b, s in enumerate(slots):
        if 0 <= s < states.shape[0]:
            w = v[b].double()[:, :, None] * k[b].double()[of][:, None, :]
            old = alpha.double()[:, None, None] * new[s]
            new[s] = old + w
            tol[s] = 2 * U * (old.abs() + w.abs())
            qq = q[b].double()[of][:, None, :]
            o[b] = (new[s] * qq).sum(-1) * scale
            ot[b] = abs(scale) * (((old.abs() + w.abs()) * qq.abs()).sum(-1) * (dk + 8) * U)
    return o, ot, new, tol


@pytest.mark.parametrize("dtype, out", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("dk, dv", DIMS)
@pytest.mark.parametrize("B, H, Hk", [(1, 1, 1), (3, 6, 2), (37, 5, 5)])
def test_step(B, H, Hk, dk, dv, dtype, out):
    q, k, v, a, _, g = make([B], H, Hk, dk, dv, dtype, alpha=[(0.0, 1.0, 0.9, 1e-30, 0.5, 0.99)[i] for i in range(H)])
    pool = torch.randn(B + 4, H, dv, dk, generator=g, device="cuda")
    slots = torch.randperm(B + 4, generator=g, device="cuda")[:B].to(torch.int32)
    if B > 4:
        slots[2], slots[B - 1] = -1, B + 4   # padding rows: negative and past the pool
    o_ref, ot, new, tol = step_reference(q, k, v, a, pool, slots.tolist(), 0.25)
    untouched = [i for i in range(B + 4) if i not in slots.tolist()]
    before = pool.clone()
    o = gdn.gdn_linear_step(q, k, v, a, pool, slots=slots, scale=0.25, out_dtype=out)
    close(o, o_ref, ot, "o")
    close(pool, new, tol, "states")
    assert torch.equal(pool[untouched], before[untouched])
    if B > 4:
        assert not o[2].any() and not o[B - 1].any()


def test_step_continues_a_prefill():
    """A prompt's state, then its next tokens one at a time, against the whole prompt."""
    q, k, v, a, cu, _ = make([140], 8, 2, 128, 128, BF)
    first = gdn.gdn_linear_prefill(q[:100], k[:100], v[:100], a, [0, 100])
    states = first["S_final"]
    o, ot, fin, fint, _, _ = reference(q, k, v, a, cu, [None], 1.0, None, True)
    for t in range(100, 140):
        got = gdn.gdn_linear_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], a, states)
        close(got, o[t:t + 1], ot[t:t + 1], f"token {t}")
    close(states, fin, fint, "state")


def test_step_strided_and_in_a_graph():
    B, H, d = 5, 4, 128
    q, k, v, a, _, g = make([B], H, H, d, d, BF)
    big = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
    qs, ks, vs = (x.unflatten(1, (H, d)) for x in big.split(H * d, 1))
    pool = torch.randn(B, H, d, d, generator=g, device="cuda")
    ref_pool = pool.clone()
    ref = [gdn.gdn_linear_step(q, k, v, a, ref_pool).clone() for _ in range(3)]
    o = torch.empty(B, H, d, dtype=BF, device="cuda")
    keep = pool.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gdn.gdn_linear_step(qs, ks, vs, a, pool, o=o)
    torch.cuda.current_stream().wait_stream(s)
    pool.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_linear_step(qs, ks, vs, a, pool, o=o)
    for r in ref:
        graph.replay()
        assert torch.equal(o, r)
    assert torch.equal(pool, ref_pool)
