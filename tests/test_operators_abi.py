"""Refusals of the router and MXFP4 entry points, on the host, before anything is launched (no
GPU needed)."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_amd as m

FAKE = 1 << 40  # an aligned, never-dereferenced address: every call below fails first


@pytest.fixture(scope="module")
def lib():
    return m.load_library()


def vp(a):
    return None if a is None else ctypes.c_void_p(a)


def router(**kw):
    d = dict(T=8, E=16, K=2, logits_stride=16, logits_dtype=m.F32, ids_dtype=m.I32, score=0,
             renormalize=1, groups=1, topk_groups=1, group_top=1, scale=1.0)
    d.update(kw)
    return m.Router(*[d[n] for n, _ in m.Router._fields_])


BAD_ROUTERS = [
    (dict(T=-1), 2), (dict(E=0, K=1), 2), (dict(E=1025, logits_stride=1025), 2), (dict(K=0), 2),
    (dict(K=33, E=64, logits_stride=64), 2), (dict(K=17), 2), (dict(T=1 << 30, K=8), 2),
    (dict(logits_stride=15), 2), (dict(score=2), 2), (dict(renormalize=2), 2), (dict(groups=0), 2),
    (dict(groups=3), 2), (dict(groups=128, E=128, logits_stride=128, topk_groups=4), 2),
    (dict(groups=4, topk_groups=5), 2), (dict(groups=4, topk_groups=0), 2),
    (dict(groups=8, topk_groups=1, K=3), 2), (dict(group_top=3), 2), (dict(group_top=0), 2),
    (dict(groups=16, topk_groups=4, group_top=2), 2), (dict(scale=float("nan")), 2),
    (dict(scale=float("inf")), 2), (dict(logits_dtype=m.I32), 3), (dict(ids_dtype=m.F32), 3),
]


@pytest.mark.parametrize("bad,code", BAD_ROUTERS)
def test_router_rejects(lib, bad, code):
    r = router(**bad)
    assert lib.moe_ffn_router_fwd(ctypes.byref(r), vp(FAKE), None, vp(FAKE), vp(FAKE), None) == code
    assert lib.moe_ffn_last_error()
    assert lib.moe_ffn_router_bwd(ctypes.byref(r), vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE),
                                  None) == code


def test_router_pointers(lib):
    r = router()
    fwd = lambda l=FAKE, b=None, i=FAKE, w=FAKE, r=r: lib.moe_ffn_router_fwd(
        ctypes.byref(r), vp(l), vp(b), vp(i), vp(w), None)
    assert fwd(l=None) == 1 and fwd(i=None) == 1 and fwd(w=None) == 1
    assert fwd(l=FAKE + 2) == 4 and fwd(b=FAKE + 1) == 4 and fwd(i=FAKE + 2) == 4
    assert fwd(i=FAKE + 4, r=router(ids_dtype=m.I64)) == 4
    assert fwd(l=FAKE + 1, r=router(logits_dtype=m.BF16)) == 4
    assert lib.moe_ffn_router_fwd(None, vp(FAKE), None, vp(FAKE), vp(FAKE), None) == 1
    bwd = lambda d=FAKE, l=FAKE, i=FAKE, o=FAKE: lib.moe_ffn_router_bwd(
        ctypes.byref(r), vp(d), vp(l), vp(i), vp(o), None)
    assert bwd(d=None) == 1 and bwd(l=None) == 1 and bwd(i=None) == 1 and bwd(o=None) == 1
    assert bwd(o=FAKE + 2) == 4 and bwd(d=FAKE + 2) == 4
    # no tokens: nothing to do
    r0 = router(T=0)
    assert lib.moe_ffn_router_fwd(ctypes.byref(r0), None, None, None, None, None) == 0
    assert lib.moe_ffn_router_bwd(ctypes.byref(r0), None, None, None, None, None) == 0


BAD_STACKS = [(dict(E=0), 2), (dict(E=1025), 2), (dict(Kd=0), 2), (dict(Kd=12), 2),
              (dict(N=24, panels=2), 2), (dict(N=4), 2), (dict(panels=3), 2), (dict(panels=0), 2),
              (dict(Kd=1 << 16, N=1 << 15), 2), (dict(dtype=m.I32), 3)]


def stack(**kw):
    d = dict(E=2, Kd=64, N=64, panels=1, dtype=m.BF16)
    d.update(kw)
    return m.MXFP4Stack(d["E"], d["Kd"], d["N"], d["panels"], d["dtype"])


@pytest.mark.parametrize("bad,code", BAD_STACKS)
def test_weight_stack_rejects(lib, bad, code):
    w, n = stack(**bad), ctypes.c_size_t()
    assert lib.moe_ffn_mxfp4_weight_size(ctypes.byref(w), ctypes.byref(n)) == code
    assert lib.moe_ffn_mxfp4_quantize(ctypes.byref(w), vp(FAKE), vp(FAKE), 1 << 40, None) == code
    assert lib.moe_ffn_mxfp4_dequantize(ctypes.byref(w), vp(FAKE), 1 << 40, vp(FAKE), None) == code


def test_weight_size_and_buffers(lib):
    w, n = stack(E=3, Kd=2048, N=2816, panels=2), ctypes.c_size_t()
    assert lib.moe_ffn_mxfp4_weight_size(ctypes.byref(w), ctypes.byref(n)) == 0
    assert n.value == 3 * 2048 * 2816 * 17 // 32  # whole tiles: 17 bits for 4 values
    assert lib.moe_ffn_mxfp4_weight_size(ctypes.byref(w), None) == 1
    q = lambda a=FAKE, p=FAKE, b=n.value: lib.moe_ffn_mxfp4_quantize(ctypes.byref(w), vp(a), vp(p),
                                                                     b, None)
    assert q(a=None) == 1 and q(p=None) == 1 and q(a=FAKE + 8) == 4 and q(p=FAKE + 8) == 4
    assert q(b=n.value - 1) == 5


def prob(**kw):
    d = dict(T=64, H=256, I=128, E=8, K=2, dtype=m.BF16, ids_dtype=m.I32, Is=0)
    d.update(kw)
    return m.Problem(*[d[n] for n, _ in m.Problem._fields_])


@pytest.mark.parametrize("bad,act,flags,code", [
    (dict(H=12), 4, 0, 2), (dict(K=0), 4, 0, 2), (dict(dtype=m.F32), 4, 0, 3), (dict(), 3, 0, 3),
    (dict(), 6, 0, 3), (dict(Is=128), 4, 0, 2), (dict(), 4, m.PIPELINE, 2), (dict(), 5, m.BULK, 2),
    (dict(), 4, 0x100, 2), (dict(T=1 << 22, H=2048), 4, 0, 2), (dict(T=(1 << 21) + 1, H=4000), 5, 0, 2),
    (dict(T=1 << 24, H=8), 4, 0, 2),
    (dict(T=1, H=(1 << 27) - 8, I=8), 4, 0, 2), (dict(T=1, H=8, I=(1 << 27) - 8), 4, 0, 2),
])
def test_forward_rejects(lib, bad, act, flags, code):
    p, n = prob(**bad), ctypes.c_size_t()
    assert lib.moe_ffn_mxfp4_workspace_size(ctypes.byref(p), act, flags, ctypes.byref(n)) == code
    a = [vp(FAKE)] * 7
    assert lib.moe_ffn_mxfp4_fwd(ctypes.byref(p), act, *a, 1 << 40, flags, None) == code


def test_forward_pointers_and_workspace(lib):
    p = prob()
    need = m.mxfp4_workspace_size(p)
    assert m.mxfp4_workspace_size(p, "mxfp6") > need

    def call(bad=None, value=None, ws_bytes=need, p=p):
        a = [FAKE] * 7  # x, ids, gates, up, down, y, ws
        if bad is not None:
            a[bad] = value
        return lib.moe_ffn_mxfp4_fwd(ctypes.byref(p), 4, *[vp(v) for v in a], ws_bytes, 0, None)

    for i in range(7):
        assert call(i, None) == 1
        assert call(i, FAKE + 2) == 4
    assert call(1, FAKE + 4, p=prob(ids_dtype=m.I64)) == 4
    assert call(ws_bytes=need - 1) == 5
    p0 = prob(T=0)
    assert lib.moe_ffn_mxfp4_fwd(ctypes.byref(p0), 4, *[None] * 7, 0, 0, None) == 0


def test_python_refuses_cpu_tensors_and_bad_arguments():
    l = torch.zeros(4, 8)
    with pytest.raises(m.MoEFFNError):
        m.moe_ffn_router_fwd(l, 2)
    with pytest.raises(m.MoEFFNError):
        m.moe_ffn_router_fwd(l, 2, ids_dtype=torch.int16)
    with pytest.raises(m.MoEFFNError):
        m.moe_ffn_router_bwd(torch.zeros(4, 2), l, torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(m.MoEFFNError):
        m.moe_ffn_mxfp4_quantize(torch.zeros(1, 32, 32))
    with pytest.raises(m.MoEFFNError):
        m.mxfp4_workspace_size(prob(), act="fp4")
    w = m.MXFP4Weight(torch.zeros(16, dtype=torch.uint8), 1, 32, 32, 1, torch.bfloat16)
    with pytest.raises(m.MoEFFNError):
        m.moe_ffn_mxfp4_dequantize(w)
    with pytest.raises(m.MoEFFNError):
        m.moe_ffn_mxfp4_fwd(torch.zeros(4, 32, dtype=torch.bfloat16),
                            torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 1), w, w)
