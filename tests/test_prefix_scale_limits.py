"""Scales of the prefix attention that leave the range of fp32 once multiplied by log2 e are refused on the host (no GPU)."""
import ctypes

import pytest

import hybrid_model_recurrent_gb300 as gdn

FAKE = 0x7f0000000000  # never dereferenced: the calls are refused before anything touches CUDA


@pytest.mark.parametrize("scale", [3e38, -3e38, 3.4028234e38, 2.36e38])
@pytest.mark.parametrize("dtype", [gdn.GDN_F32, gdn.GDN_BF16])
def test_scale_out_of_range(scale, dtype):
    gdn.build()
    pr = gdn._PrefixProblem(2, 1, 8, 2, 64, dtype, 1000, 0, 0, scale)
    p = ctypes.c_void_p(FAKE)
    assert gdn.lib().gdn_prefix_scratch_bytes(ctypes.byref(pr)) == 0
    assert gdn.lib().gdn_prefix_attention(ctypes.byref(pr), p, p, p, None, None, None, p, p, p, 1 << 40, p, 256,
                                          None) == gdn.GDN_ERR_INVALID_ARG


def test_largest_scale_is_accepted():
    """The largest float whose product with log2 e is one still has a plan."""
    gdn.build()
    pr = gdn._PrefixProblem(2, 1, 8, 2, 64, gdn.GDN_BF16, 1000, 0, 0, 2.35e38)
    assert gdn.lib().gdn_prefix_scratch_bytes(ctypes.byref(pr)) > 0
