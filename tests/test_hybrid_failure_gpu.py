"""Bounded waits of the tensor-core kernels of include/gdn_hybrid.h: with the testing hook they stop issuing their input
copies, so their next wait runs out after the (short) limit; they must drain, record the status and return, and the
context must stay usable."""
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _linear(ws, d):
    T = 900
    q, v, a = torch.ones(T, 2, d, dtype=BF, device="cuda") / 16, torch.ones(T, 2, d, dtype=BF, device="cuda"), torch.full(
        (2,), 0.9, device="cuda")
    return lambda: gdn.gdn_linear_prefill(q, q, v, a, [0, 500, T], ws=ws)["o"]


def _prefix(ws, n, D):
    q, k = torch.ones(3, n, 4, D, dtype=BF, device="cuda"), torch.ones(2000, 2, D, dtype=BF, device="cuda")
    kt, tl = torch.ones(3, 700, 2, D, dtype=BF, device="cuda"), torch.full((3,), 600, dtype=torch.int32, device="cuda")
    return lambda: gdn.gdn_prefix_attention(q, k, k, kt, kt, tl, ws=ws)["o"]


# after how many chunks (of a scan) or tiles (of a CTA, which may have a single one) the copies stop
@pytest.mark.parametrize("make, stall", [
    (lambda ws: _linear(ws, 128), 1), (lambda ws: _linear(ws, 64), 2), (lambda ws: _prefix(ws, 1, 128), 0),
    (lambda ws: _prefix(ws, 100, 128), 0), (lambda ws: _prefix(ws, 300, 64), 0)])
def test_wait_limit_expiry_is_reported_and_recoverable(make, stall):
    gdn.build()
    ws = torch.zeros(int(gdn.lib().gdn_workspace_size()), dtype=torch.uint8, device="cuda")
    call = make(ws)
    ref = call()
    torch.cuda.synchronize()
    assert gdn.read_status(ws=ws) == gdn.GDN_OK
    try:
        gdn.set_wait_limit_ns(20_000_000)   # 20 ms
        gdn.debug_stall_after(stall)
        call()
        torch.cuda.synchronize()
        assert gdn.read_status(ws=ws) == gdn.GDN_ERR_DEVICE_TIMEOUT, "an unfed wait must run out and be reported"
    finally:
        gdn.debug_stall_after(-1)
        gdn.set_wait_limit_ns(0)   # back to the default
    gdn.clear_status(ws=ws)
    again = call()
    torch.cuda.synchronize()
    assert gdn.read_status(ws=ws) == gdn.GDN_OK and torch.equal(again, ref)
