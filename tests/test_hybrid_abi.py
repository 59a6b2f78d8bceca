"""The operators of include/gdn_hybrid.h on the host (no GPU): every bad call returns its status before anything
touches CUDA, scratch sizes, and the binding's own checks of shapes and strides."""
import ctypes

import numpy as np
import pytest
import torch

import hybrid_model_recurrent_gb300 as gdn

FAKE = 0x7f0000000000  # never dereferenced: validation must fail first


@pytest.fixture(scope="module")
def L():
    gdn.build()
    return gdn.lib()


def _vp(off=0):
    return ctypes.c_void_p(FAKE + off)


def _lin(B=2, H=4, Hk=2, dk=64, dv=128, cu=(0, 10, 30), qkv=gdn.GDN_BF16, out=gdn.GDN_BF16, scale=1.0, strides=(0, 0, 0)):
    pr = gdn._LinearProblem()
    pr.num_seqs, pr.num_heads, pr.num_qk_heads, pr.d_k, pr.d_v = B, H, Hk, dk, dv
    if cu is not None:
        arr = np.ascontiguousarray(np.asarray(cu, dtype=np.int64))
        pr.cu_seqlens = arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))
        pr._keep = arr
    pr.qkv_dtype, pr.out_dtype, pr.scale = qkv, out, scale
    pr.q_stride, pr.k_stride, pr.v_stride = strides
    return pr


def _prefill(L, pr, *, q=0, k=0, v=0, alpha=0, S0=None, index=None, slots=0, o=0, S_final=0, ck=None, cu_ck=None,
             ckpt=None, scratch=None, nscratch=0, ws=0, nws=256):
    def ptr(x):
        return None if x is None else _vp(x)

    ix = None if index is None else (ctypes.c_int32 * len(index))(*index)
    c = None if ck is None else (ctypes.c_int64 * max(len(ck), 1))(*ck)
    cc = None if cu_ck is None else (ctypes.c_int64 * len(cu_ck))(*cu_ck)
    return L.gdn_linear_prefill(ctypes.byref(pr) if pr is not None else None, ptr(q), ptr(k), ptr(v), ptr(alpha), ptr(S0),
                                ix, slots, ptr(o), ptr(S_final), c, cc, ptr(ckpt), ptr(scratch), nscratch, ptr(ws), nws,
                                None)


INV, UNS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("prob, want", [
    (dict(B=0), INV), (dict(H=0), INV), (dict(H=4, Hk=3), INV), (dict(Hk=0), INV), (dict(dk=0), INV), (dict(dk=96), UNS),
    (dict(dv=256), UNS), (dict(qkv=7), INV), (dict(out=2), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(strides=(127, 0, 0)), INV), (dict(strides=(0, 64, 0)), INV),
    (dict(strides=(0, 0, 513)), INV), (dict(strides=(-256, 0, 0)), INV), (dict(cu=None), INV), (dict(cu=(1, 10, 30)), INV),
    (dict(cu=(0, 10, 9)), INV), (dict(cu=(0, 10, 2 ** 31)), UNS), (dict(H=2 ** 17, Hk=1), UNS),
])
def test_linear_problem_refusals(L, prob, want):
    pr = _lin(**prob)
    assert _prefill(L, pr) == want
    assert L.gdn_linear_scratch_bytes(ctypes.byref(pr)) == 0
    if "cu" not in prob:
        assert L.gdn_linear_step(ctypes.byref(pr), _vp(), _vp(), _vp(), _vp(), _vp(), 4, None, _vp(), None) == want


@pytest.mark.parametrize("call", [
    dict(q=None), dict(k=None), dict(v=None), dict(alpha=None), dict(S_final=None), dict(ws=None), dict(nws=128),
    dict(q=2), dict(k=8), dict(v=4), dict(alpha=2), dict(S_final=8), dict(o=2), dict(ws=8), dict(S0=8, slots=2),
    dict(S0=0, slots=1), dict(S0=0, slots=3, index=[0, 3]), dict(S0=0, slots=3, index=[-2, 0]),
    dict(ck=[5], cu_ck=[1, 1, 1], ckpt=0), dict(ck=[5, 6], cu_ck=[0, 2, 1], ckpt=0), dict(ck=[0], cu_ck=[0, 1, 1], ckpt=0),
    dict(ck=[11], cu_ck=[0, 1, 1], ckpt=0), dict(ck=[5, 5], cu_ck=[0, 2, 2], ckpt=0), dict(ck=[5], cu_ck=[0, 1, 1]),
    dict(ck=None, cu_ck=[0, 1, 1], ckpt=0), dict(ck=[5], cu_ck=[0, 1, 1], ckpt=4),
])
def test_linear_prefill_refusals(L, call):
    assert _prefill(L, _lin(), **call) == INV


def test_linear_scratch(L):
    """A call whose few long scans are split needs scratch, and says so; many scans need none."""
    long = _lin(B=1, H=2, Hk=2, dk=128, dv=128, cu=(0, 50000))
    need = L.gdn_linear_scratch_bytes(ctypes.byref(long))
    assert need > 0 and need % (2 * 128 * 128 * 4) == 0
    assert _prefill(L, long) == INV
    assert _prefill(L, long, scratch=0, nscratch=need - 1) == INV
    assert _prefill(L, long, scratch=8, nscratch=need) == INV
    many = _lin(B=64, H=16, Hk=16, dk=128, dv=128, cu=[i * 500 for i in range(65)])
    assert L.gdn_linear_scratch_bytes(ctypes.byref(many)) == 0
    assert _prefill(L, None) == INV and L.gdn_linear_scratch_bytes(None) == 0


def test_linear_prefill_too_many_checkpoints(L):
    """More checkpoints in one scan than a launch holds: refused before anything is enqueued."""
    pr = _lin(B=300, H=1, Hk=1, cu=[0] + [2000 * (i + 1) for i in range(300)])
    assert L.gdn_linear_scratch_bytes(ctypes.byref(pr)) == 0
    assert _prefill(L, pr, ck=list(range(1, 2000)), cu_ck=[0] + [1999] * 300, ckpt=0) == UNS


@pytest.mark.parametrize("bad", [0, 1, 2, 3, 4, 5, "slots", "count", "align"])
def test_linear_step_refusals(L, bad):
    a = [_vp(), _vp(), _vp(), _vp(), _vp()]   # q, k, v, alpha, states
    o, slots, count = _vp(), None, 2
    if bad == 5:
        o = None
    elif bad == "slots":
        count = 1          # slot b of 2 requests in a pool of 1
    elif bad == "count":
        count = -1
    elif bad == "align":
        slots = _vp(2)
    else:
        a[bad] = None
    assert L.gdn_linear_step(ctypes.byref(_lin(cu=None)), *a, count, slots, o, None) == INV


def _pre(**kw):
    pr = gdn._PrefixProblem()
    d = dict(batch=2, num_queries=1, num_q_heads=8, num_kv_heads=2, head_dim=128, dtype=gdn.GDN_BF16, prefix_len=1000,
             tail_cap=64, max_tail=64, softmax_scale=0.1)
    d.update(kw)
    for n, x in d.items():
        setattr(pr, n, x)
    return pr


def _attend(L, pr, *, q=0, kp=0, vp=0, kt=0, vt=0, tail=0, o=0, lse=0, scratch=0, nscratch=1 << 40, ws=0, nws=256):
    args = [None if x is None else _vp(x) for x in (q, kp, vp, kt, vt, tail, o, lse, scratch)]
    return L.gdn_prefix_attention(None if pr is None else ctypes.byref(pr), *args, nscratch, None if ws is None else _vp(ws),
                                  nws, None)


@pytest.mark.parametrize("prob, want", [
    (dict(batch=0), INV), (dict(num_queries=0), INV), (dict(num_q_heads=0), INV), (dict(num_kv_heads=3), INV),
    (dict(num_kv_heads=0), INV), (dict(head_dim=0), INV), (dict(head_dim=96), UNS), (dict(head_dim=256), UNS),
    (dict(dtype=5), INV), (dict(prefix_len=-1), INV), (dict(tail_cap=-1, max_tail=0), INV), (dict(max_tail=65), INV),
    (dict(max_tail=-1), INV), (dict(softmax_scale=float("inf")), INV), (dict(prefix_len=2 ** 31), UNS),
    (dict(tail_cap=2 ** 31), UNS), (dict(batch=2 ** 30), UNS), (dict(q_stride_h=129), INV), (dict(kp_stride_t=-8), INV),
    (dict(vt_stride_b=4), INV), (dict(kt_stride_t=2 ** 37), UNS), (dict(num_q_heads=2 ** 17), UNS),
])
def test_prefix_problem_refusals(L, prob, want):
    pr = _pre(**prob)
    assert _attend(L, pr) == want
    assert L.gdn_prefix_scratch_bytes(ctypes.byref(pr)) == 0


@pytest.mark.parametrize("call", [
    dict(q=None), dict(kp=None), dict(vp=None), dict(kt=None), dict(vt=None), dict(tail=None), dict(o=None), dict(ws=None),
    dict(nws=255), dict(scratch=None), dict(nscratch=0), dict(q=8), dict(kp=2), dict(vp=4), dict(kt=8), dict(vt=8),
    dict(tail=2), dict(o=8), dict(lse=2), dict(scratch=8), dict(scratch=16), dict(ws=8),
])
def test_prefix_attention_refusals(L, call):
    assert _attend(L, _pre(), **call) == INV


def test_prefix_null_and_scratch(L):
    assert _attend(L, None) == INV and L.gdn_prefix_scratch_bytes(None) == 0
    pr = _pre()
    need = L.gdn_prefix_scratch_bytes(ctypes.byref(pr))
    assert need > 0 and _attend(L, pr, nscratch=need - 1) == INV
    # nothing to attend to: no parts
    assert L.gdn_prefix_scratch_bytes(ctypes.byref(_pre(prefix_len=0, tail_cap=0, max_tail=0))) == 0


def test_binding_checks_shapes_and_strides(L):
    bf = torch.bfloat16
    q, k, v, a = torch.zeros(5, 2, 64, dtype=bf), torch.zeros(5, 2, 64, dtype=bf), torch.zeros(5, 4, 64, dtype=bf), torch.ones(4)
    ok = dict(S_final=torch.zeros(1, 4, 64, 64), o=torch.zeros(5, 4, 64, dtype=bf), ws=torch.zeros(256, dtype=torch.uint8))
    for bad in (dict(q=q[:4]), dict(v=v.float()), dict(alpha=a[:3]), dict(alpha=a.double()), dict(cu=[0, 4]),
                dict(k=k.transpose(0, 1)), dict(v=v[:, :1].expand(5, 4, 64)), dict(k=k[:, :, ::2]), dict(q=None),
                dict(S0_index=[0]), dict(S0=torch.zeros(1, 4, 64, 32)), dict(S0=torch.zeros(1, 4, 64, 64), S0_index=[0, 0]),
                dict(o=torch.zeros(5, 4, 64)), dict(S_final=torch.zeros(2, 4, 64, 64)), dict(ckpt_pos=[[1], [2]])):
        args = dict(q=q, k=k, v=v, alpha=a, cu=[0, 5])
        kw = dict(ok)
        for n, x in bad.items():
            (args if n in args else kw)[n] = x
        with pytest.raises(ValueError):
            gdn.gdn_linear_prefill(args["q"], args["k"], args["v"], args["alpha"], args["cu"], **kw)
    st = torch.zeros(5, 4, 64, 64)
    for bad in (dict(states=st[0]), dict(states=st.transpose(2, 3)), dict(states=st.double()),
                dict(slots=torch.zeros(5, dtype=torch.int64)), dict(slots=torch.zeros(4, dtype=torch.int32)),
                dict(o=torch.zeros(5, 4, 64))):
        kw = dict(states=st)
        kw.update(bad)
        with pytest.raises(ValueError):
            gdn.gdn_linear_step(q, k, v, a, kw.pop("states"), **kw)
    pq, pk = torch.zeros(2, 1, 8, 64, dtype=bf), torch.zeros(10, 2, 64, dtype=bf)
    kt, tl = torch.zeros(2, 4, 2, 64, dtype=bf), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(q=pq[0]), dict(v_prefix=pk[:9]), dict(k_prefix=pk[:, :, :32], v_prefix=pk[:, :, :32]),
                dict(k_tail=kt), dict(k_tail=kt, v_tail=kt, tail_len=tl.long()), dict(k_tail=kt[:1], v_tail=kt[:1], tail_len=tl),
                dict(tail_len=tl), dict(k_prefix=pk.float(), v_prefix=pk.float()),
                dict(k_prefix=pk[:1].expand(10, 2, 64), v_prefix=pk), dict(q=pq.transpose(2, 3)),
                dict(o=torch.zeros(2, 1, 8, 64)), dict(lse=torch.zeros(2, 8))):
        kw = dict(q=pq, k_prefix=pk, v_prefix=pk)
        kw.update(bad)
        with pytest.raises(ValueError):
            gdn.gdn_prefix_attention(kw.pop("q"), kw.pop("k_prefix"), kw.pop("v_prefix"), **kw)
