"""Linear prefills with more checkpoints for a sequence than a launch holds (1536), with scans cut into segments and whole ones,
against the recurrence in 64 bits.

Tolerances.  States: 2^-19 of a state's norm (fp32 sums of at most 512 tokens that count, errors of independent signs).
Readouts, relative to the sum of the terms' absolute values: in bf16 three half steps, 3 * 2^-8 (one on each term's operand, one
on the output, one for all that is smaller); in fp32 2^-14 (a state element's two roundings of 2^-24 a token, over 512 of them,
of one sign)."""
import ctypes

import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def needs_scratch(cu, H, dk, dv, dtype):
    pr = gdn._LinearProblem()
    c = gdn._i64(cu)
    pr.num_seqs, pr.num_heads, pr.num_qk_heads, pr.d_k, pr.d_v, pr.scale = len(cu) - 1, H, H, dk, dv, 1.0
    pr.cu_seqlens, pr.qkv_dtype, pr.out_dtype = gdn._p64(c), gdn._dtype_code(dtype), gdn._dtype_code(dtype)
    return gdn.lib().gdn_linear_scratch_bytes(ctypes.byref(pr)) > 0


@pytest.mark.parametrize("readout", [True, False])
@pytest.mark.parametrize("dtype, d, H, lens, every, cut", [
    (BF, 64, 160, [1601], 1, False),            # whole scans: the second job takes up the state after 1536 tokens
    (BF, 64, 160, [40, 3300, 1], 1, False),     # three jobs in a row, other sequences beside them
    (BF, 128, 16, [3100], 1, True),             # cut scans whose segments hold fewer
    (BF, 64, 64, [8000], 2, True),              # and more than a job
    (F32, 32, 304, [1601, 5], 1, False),
])
def test_more_checkpoints_than_a_launch_holds(dtype, d, H, lens, every, cut, readout):
    g = torch.Generator(device="cuda").manual_seed(H)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, B = cu[-1], len(lens)
    assert needs_scratch(cu, H, d, d, dtype) == cut
    q, k = (torch.randn(T, H, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    v = torch.randn(T, H, d, generator=g, device="cuda").to(dtype)
    alpha = torch.tensor([1 - 2.0 ** -(3 + i % 7) for i in range(H)], device="cuda")
    pool = torch.randn(2, H, d, d, generator=g, device="cuda")
    ckpt = [list(range(every, n + 1, every)) for n in lens]
    assert max(len(c) for c in ckpt) > 1536
    r = gdn.gdn_linear_prefill(q if readout else None, k, v, alpha, cu, S0=pool, S0_index=[1] * B, ckpt_pos=ckpt, readout=readout)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    al = alpha.double()[:, None, None]
    at, worst, worst_o = 0, torch.zeros((), dtype=torch.float64, device="cuda"), torch.zeros((), dtype=torch.float64, device="cuda")
    for b in range(B):
        S = pool[1].double()
        A = S.abs()
        for t in range(cu[b], cu[b + 1]):
            new = v[t].double()[:, :, None] * k[t].double()[:, None, :]
            S = al * S + new
            if readout:
                A = al * A + new.abs()
                qq = q[t].double()[:, None, :]
                off = (r["o"][t].double() - (S * qq).sum(-1)).abs() / (A * qq.abs()).sum(-1)
                worst_o = torch.maximum(worst_o, off.amax())
            if (t + 1 - cu[b]) % every == 0:
                off = (r["ckpt_states"][at].double() - S).flatten(1).norm(dim=1) / S.flatten(1).norm(dim=1)
                worst = torch.maximum(worst, off.amax())
                at += 1
        off = (r["S_final"][b].double() - S).flatten(1).norm(dim=1) / S.flatten(1).norm(dim=1)
        worst = torch.maximum(worst, off.amax())
    assert at == len(r["ckpt_states"])
    assert worst.item() < 2.0 ** -19, f"states off by {worst.item():.3g}"
    if readout:
        tol = 3 * 2.0 ** -8 if dtype == BF else 2.0 ** -14
        assert worst_o.item() < tol, f"outputs off by {worst_o.item():.3g}"
