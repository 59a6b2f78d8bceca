"""The fp32 states of a linear prefill against the recurrence in 64 bits, by their norms.

Tolerance: 2^-19 of a state's norm.  A state adds up about 1 / (1 - alpha) <= 512 tokens, four chunks of 128: with 24 products
a chunk whose sums lose at most 2^-23 each, of independent signs, 2^-23 * sqrt(96) < 2^-19.  Values kept in two bf16 parts,
or a state rounded to fewer bits between chunks, are off by more (2^-18.6 and up)."""
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk, dv", [(128, 128), (64, 64), (64, 128), (128, 64), (32, 32)])
@pytest.mark.parametrize("lens, H, readout", [((1500, 0, 700, 1), 3, True), ((1500, 0, 700, 1), 3, False),
                                              ((257, 129) * 40, 4, True)])
def test_states_are_fp32_sums(lens, H, readout, dk, dv, dtype):
    """Scans cut into segments (few long ones) and whole ones (many), a checkpoint every 128 tokens, so at every segment's
    end, and at odd places."""
    g = torch.Generator(device="cuda").manual_seed(dk + dv)
    T, B = sum(lens), len(lens)
    q, k = (torch.randn(T, H, dk, generator=g, device="cuda").to(dtype) for _ in range(2))
    v = torch.randn(T, H, dv, generator=g, device="cuda").to(dtype)
    alpha = torch.tensor([1 - 2.0 ** -(3 + 2 * i) for i in range(H)], device="cuda")
    pool = torch.randn(2, H, dv, dk, generator=g, device="cuda")
    index = [(0, -1, 1)[b % 3] for b in range(B)]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    ckpt = [sorted({*range(128, n + 1, 128), *(p for p in (1, 127, 333, n) if 1 <= p <= n)}) for n in lens]
    r = gdn.gdn_linear_prefill(q if readout else None, k, v, alpha, cu, S0=pool, S0_index=index, ckpt_pos=ckpt, readout=readout)
    assert gdn.read_status("cuda") == gdn.GDN_OK
    at = 0
    for b, n in enumerate(lens):
        S = torch.zeros(H, dv, dk, dtype=torch.float64, device="cuda") if index[b] < 0 else pool[index[b]].double()
        last = 0
        for p in ckpt[b]:   # from one checkpoint to the next: the sum itself, with every power of the decay
            kk, vv = k[cu[b] + last:cu[b] + p].double(), v[cu[b] + last:cu[b] + p].double()
            w = alpha.double() ** torch.arange(p - last - 1, -1, -1, device="cuda", dtype=torch.float64)[:, None]
            S = (alpha.double() ** (p - last))[:, None, None] * S + torch.einsum("th,thv,thk->hvk", w, vv, kk)
            last = p
            assert off(r["ckpt_states"][at], S) < 2.0 ** -19, (b, p)
            at += 1
        if n == 0 and index[b] < 0:
            assert not r["S_final"][b].any()
        else:
            assert off(r["S_final"][b], S) < 2.0 ** -19, b
