"""Which checkpoint lists a linear prefill refuses, on the host: the limits of the header, whatever the plan (no GPU)."""
import ctypes

import pytest

import hybrid_model_recurrent_gb300 as gdn

FAKE = 0x7f0000000000  # never dereferenced: every call here is refused before anything touches CUDA


@pytest.mark.parametrize("H, first, rest, cut", [
    (1, 100000, 1, True),         # one long scan beside 256 short ones, cut into segments that hold fewer checkpoints each
    (16, 100000, 1, True),
    (1, 2000, 2000, False),       # as many whole ones
    (16, 1537, 900, False),
])
def test_long_lists_are_refused_whatever_the_plan(H, first, rest, cut):
    """A sequence with more checkpoints than a job holds, in a call of more than 256 sequences."""
    gdn.build()
    L = gdn.lib()
    B, n_ck = 257, 1537
    pr = gdn._LinearProblem()
    c = gdn._i64([0] + [first + rest * i for i in range(B)])
    pr.num_seqs, pr.num_heads, pr.num_qk_heads, pr.d_k, pr.d_v, pr.scale = B, H, H, 128, 128, 1.0
    pr.cu_seqlens, pr.qkv_dtype, pr.out_dtype = gdn._p64(c), gdn.GDN_BF16, gdn.GDN_BF16
    need = L.gdn_linear_scratch_bytes(ctypes.byref(pr))
    assert (need > 0) == cut
    ck, cu_ck = gdn._i64(range(1, n_ck + 1)), gdn._i64([0] + [n_ck] * B)
    p = ctypes.c_void_p(FAKE)
    rc = L.gdn_linear_prefill(ctypes.byref(pr), p, p, p, p, None, None, 0, p, p, gdn._p64(ck), gdn._p64(cu_ck), p, p, need, p,
                              256, None)
    assert rc == gdn.GDN_ERR_UNSUPPORTED
