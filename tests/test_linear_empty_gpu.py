"""A linear prefill of a batch that has no tokens: the final states are the initial ones, bit for bit, and nothing else is read."""
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk, dv", [(128, 128), (64, 64), (64, 128), (128, 64), (32, 32)])
@pytest.mark.parametrize("readout", [True, False])
@pytest.mark.parametrize("initial", [True, False])
def test_batch_without_tokens(dtype, dk, dv, readout, initial):
    H, B = 3, 4
    q = k = torch.empty(0, 1, dk, dtype=dtype, device="cuda")
    v = torch.empty(0, H, dv, dtype=dtype, device="cuda")
    pool = torch.randn(2, H, dv, dk, device="cuda") if initial else None
    index = [1, -1, 0, 1] if initial else None
    alpha = torch.tensor([0.0, 0.9, 1.0], device="cuda")
    r = gdn.gdn_linear_prefill(q, k, v, alpha, [0] * (B + 1), S0=pool, S0_index=index, ckpt_pos=[[]] * B, readout=readout)
    torch.cuda.synchronize()
    assert gdn.read_status("cuda") == gdn.GDN_OK
    assert r["ckpt_states"] is None and (r["o"] is None) == (not readout)
    if readout:
        assert r["o"].shape == (0, H, dv)
    for b in range(B):
        if initial and index[b] >= 0:
            assert torch.equal(r["S_final"][b], pool[index[b]])
        else:
            assert not r["S_final"][b].any()
