"""Refusals of the grouped and int8 products, on the host, before anything is launched (no GPU
needed)."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_amd as m

FAKE = 1 << 40  # an aligned, never-dereferenced address: every call below fails first
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    return m.load_library()


def vp(a):
    return None if a is None else ctypes.c_void_p(a)


def filled(cls, defaults, kw):
    d = {**defaults, **kw}
    return cls(*[d[n] for n, _ in cls._fields_])


def grouped(**kw):
    return filled(m.Grouped, dict(M=64, E=4, Kd=32, N=48, x_stride=32, dtype=m.BF16,
                                  offsets_dtype=m.I32, transposed=0), kw)


def stack(**kw):
    return filled(m.Int8Stack, dict(E=4, Kd=32, N=48, panels=1, dtype=m.BF16), kw)


def product(w=None, **kw):
    d = {**dict(M=64, offsets_dtype=m.I32, out_dtype=m.BF16), **kw}
    return m.Int8Product(w or stack(), d["M"], d["offsets_dtype"], d["out_dtype"])


# ---- grouped products ------------------------------------------------------------------

BAD_GROUPED = [
    (dict(M=-1), 2), (dict(M=(1 << 30) + 1), 2), (dict(E=0), 2), (dict(E=1025), 2), (dict(Kd=0), 2),
    (dict(Kd=12, x_stride=16), 2), (dict(N=4), 2), (dict(N=1 << 27), 2), (dict(Kd=1 << 31, x_stride=1 << 31), 2),
    (dict(x_stride=24), 2), (dict(x_stride=36), 2), (dict(x_stride=1 << 31), 2), (dict(transposed=2), 2),
    (dict(M=1 << 30, Kd=8, N=1 << 20), 2), (dict(dtype=m.I32), 3), (dict(offsets_dtype=m.BF16), 3),
]


@pytest.mark.parametrize("bad,code", BAD_GROUPED, ids=str)
def test_grouped_rejects(lib, bad, code):
    g = grouped(**bad)
    n = ctypes.c_size_t()
    p = ctypes.byref(g)
    assert lib.moe_ffn_grouped_workspace_size(p, ctypes.byref(n)) == code
    assert lib.moe_ffn_last_error()
    assert lib.moe_ffn_grouped_mm(p, vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE), BIG, None) == code
    assert lib.moe_ffn_grouped_mm_bwd(p, *[vp(FAKE)] * 7, BIG, None) == code


def test_grouped_pointers_and_workspace(lib):
    g = grouped()
    need = m.grouped_workspace_size(g)
    fwd = lambda x=FAKE, w=FAKE, o=FAKE, y=FAKE, s=FAKE, n=BIG, g=g: lib.moe_ffn_grouped_mm(
        ctypes.byref(g), vp(x), vp(w), vp(o), vp(y), vp(s), n, None)
    for kw in (dict(x=None), dict(w=None), dict(o=None), dict(y=None), dict(s=None)):
        assert fwd(**kw) == 1
    # fp32 forms up to 64 groups by itself
    assert m.grouped_workspace_size(grouped(dtype=m.F32, E=64)) == 0
    assert fwd(s=None, g=grouped(dtype=m.F32, E=65), n=0) == 1
    for kw in (dict(x=FAKE + 8), dict(w=FAKE + 2), dict(o=FAKE + 2), dict(y=FAKE + 4), dict(s=FAKE + 8),
               dict(o=FAKE + 4, g=grouped(offsets_dtype=m.I64))):
        assert fwd(**kw) == 4
    assert fwd(n=need - 1) == 5
    assert lib.moe_ffn_grouped_mm(None, *[vp(FAKE)] * 5, BIG, None) == 1
    assert lib.moe_ffn_grouped_workspace_size(ctypes.byref(g), None) == 1
    bwd = lambda dy=FAKE, x=FAKE, w=FAKE, o=FAKE, dx=FAKE, dw=FAKE, s=FAKE, n=BIG: lib.moe_ffn_grouped_mm_bwd(
        ctypes.byref(g), vp(dy), vp(x), vp(w), vp(o), vp(dx), vp(dw), vp(s), n, None)
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(o=None), dict(s=None),
               dict(x=None, dx=None), dict(w=None, dw=None)):
        assert bwd(**kw) == 1
    for kw in (dict(dy=FAKE + 8), dict(x=FAKE + 2), dict(dx=FAKE + 8), dict(dw=FAKE + 8)):
        assert bwd(**kw) == 4
    assert bwd(n=need - 1) == 5


def test_grouped_tensors():
    x, w = torch.zeros(8, 32), torch.zeros(2, 32, 16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (m.moe_ffn_grouped_mm_fwd, m.moe_ffn_grouped_mm):
        with pytest.raises(m.MoEFFNError, match="GPU") as ei:
            call(x, w, off)
        assert ei.value.status == 1
    with pytest.raises(m.MoEFFNError, match="GPU"):
        m.moe_ffn_grouped_mm_bwd(torch.zeros(8, 16), x, w, off)


# ---- int8 --------------------------------------------------------------------------------

BAD_STACKS = [
    (dict(E=0), 2), (dict(E=1025), 2), (dict(Kd=0), 2), (dict(Kd=12), 2), (dict(Kd=131080), 2),
    (dict(N=4), 2), (dict(N=40, panels=2), 2), (dict(panels=0), 2), (dict(panels=3), 2),
    (dict(Kd=1 << 16, N=1 << 15), 2), (dict(dtype=m.I32), 3),
]


@pytest.mark.parametrize("bad,code", BAD_STACKS, ids=str)
def test_int8_weights_reject(lib, bad, code):
    w = stack(**bad)
    p, n = ctypes.byref(w), ctypes.c_size_t()
    assert lib.moe_ffn_int8_weight_size(p, ctypes.byref(n)) == code
    assert lib.moe_ffn_int8_quantize(p, vp(FAKE), vp(FAKE), BIG, None) == code
    assert lib.moe_ffn_int8_pack(p, vp(FAKE), vp(FAKE), vp(FAKE), BIG, None) == code
    assert lib.moe_ffn_int8_dequantize(p, vp(FAKE), BIG, vp(FAKE), None) == code
    if "dtype" not in bad:
        q = product(w)
        assert lib.moe_ffn_int8_mm_workspace_size(ctypes.byref(q), ctypes.byref(n)) == code


def test_int8_weight_pointers(lib):
    w = stack()
    p, n = ctypes.byref(w), ctypes.c_size_t()
    assert lib.moe_ffn_int8_weight_size(p, ctypes.byref(n)) == 0
    # 64 of Kd, 48 columns in two tiles of 32: codes, and a scale for each of the 64 columns
    assert n.value == 4 * 64 * 64 + 4 * 64 * 4
    need = n.value
    assert lib.moe_ffn_int8_weight_size(p, None) == 1
    assert lib.moe_ffn_int8_weight_size(None, ctypes.byref(n)) == 1
    for entry in (lambda a=FAKE, b=FAKE, n=BIG: lib.moe_ffn_int8_quantize(p, vp(a), vp(b), n, None),
                  lambda a=FAKE, b=FAKE, n=BIG: lib.moe_ffn_int8_pack(p, vp(a), vp(FAKE), vp(b), n, None),
                  lambda a=FAKE, b=FAKE, n=BIG: lib.moe_ffn_int8_dequantize(p, vp(b), n, vp(a), None)):
        assert entry(a=None) == 1 and entry(b=None) == 1
        assert entry(a=FAKE + 8) == 4 and entry(b=FAKE + 4) == 4
        assert entry(n=need - 1) == 5
    assert lib.moe_ffn_int8_pack(p, vp(FAKE), None, vp(FAKE), BIG, None) == 1
    assert lib.moe_ffn_int8_pack(p, vp(FAKE), vp(FAKE + 2), vp(FAKE), BIG, None) == 4


def test_int8_rows_reject(lib):
    row = ctypes.c_int64()
    for kd, want in ((8, 64), (64, 64), (72, 128), (131072, 131072)):
        assert lib.moe_ffn_int8_row_bytes(kd, ctypes.byref(row)) == 0 and row.value == want
    for kd in (0, 4, 20, 131080):
        assert lib.moe_ffn_int8_row_bytes(kd, ctypes.byref(row)) == 2
    assert lib.moe_ffn_int8_row_bytes(8, None) == 1

    def rows(M=8, Kd=32, stride=32, dtype=m.BF16, x=FAKE, c=FAKE, s=FAKE):
        r = m.Int8RowsShape(M, Kd, stride, dtype)
        return lib.moe_ffn_int8_quantize_rows(ctypes.byref(r), vp(x), vp(c), vp(s), None)

    for kw in (dict(M=-1), dict(M=(1 << 30) + 1), dict(Kd=12), dict(Kd=131080, stride=131080), dict(stride=24),
               dict(stride=36)):
        assert rows(**kw) == 2
    assert rows(dtype=m.I32) == 3
    assert rows(x=None) == 1 and rows(c=None) == 1 and rows(s=None) == 1
    assert rows(x=FAKE + 8) == 4 and rows(c=FAKE + 8) == 4 and rows(s=FAKE + 2) == 4
    assert rows(M=0, x=None, c=None, s=None) == 0
    assert lib.moe_ffn_int8_quantize_rows(None, vp(FAKE), vp(FAKE), vp(FAKE), None) == 1


def test_int8_product_rejects(lib):
    n = ctypes.c_size_t()

    def mm(p=None, c=FAKE, s=FAKE, w=FAKE, wn=BIG, o=FAKE, y=FAKE, ws=FAKE, wsn=BIG):
        p = p or product()
        return lib.moe_ffn_int8_mm(ctypes.byref(p), vp(c), vp(s), vp(w), wn, vp(o), vp(y), vp(ws), wsn, None)

    for kw, code in ((dict(M=-1), 2), (dict(M=(1 << 30) + 1), 2), (dict(offsets_dtype=m.F32), 3),
                     (dict(out_dtype=m.I32), 3)):
        p = product(**kw)
        assert lib.moe_ffn_int8_mm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
        assert mm(p) == code
    # 8 values of Kd take 64 bytes: 2^26 columns are 4 GiB
    assert mm(product(stack(E=1, Kd=8, N=1 << 26))) == 2
    assert mm(product(stack(E=1, Kd=8, N=1 << 20), M=1 << 30)) == 2  # tiles
    # (2^23 + 1) blocks of 32 rows by 2^8 of 32 columns, counted for each panel
    for p in (product(stack(E=1, Kd=8, N=1 << 13), M=1 << 28), product(stack(E=1, Kd=8, N=1 << 13, panels=2), M=1 << 28),
              product(stack(E=1, Kd=8, N=16, panels=2), M=(1 << 30))):
        few = p.weight.N == 16
        assert lib.moe_ffn_int8_mm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == (0 if few else 2)
        assert few or mm(p) == 2
    assert mm(c=None) == 1 and mm(s=None) == 1 and mm(w=None) == 1 and mm(y=None) == 1
    assert mm(o=None) == 1  # four matrices need offsets
    assert mm(c=FAKE + 8) == 4 and mm(s=FAKE + 2) == 4 and mm(w=FAKE + 8) == 4 and mm(o=FAKE + 2) == 4
    assert mm(y=FAKE + 8) == 4
    assert mm(product(offsets_dtype=m.I64), o=FAKE + 4) == 4
    p = product(stack(E=65))
    assert lib.moe_ffn_int8_mm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
    assert mm(p, wsn=n.value - 1) == 5 and mm(p, ws=None) == 1 and mm(p, ws=FAKE + 8) == 4
    p = product(stack(E=64))
    assert lib.moe_ffn_int8_mm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
    assert n.value == 0  # up to 64 groups are formed by the product itself
    assert lib.moe_ffn_int8_weight_size(ctypes.byref(product().weight), ctypes.byref(n)) == 0
    assert mm(wn=n.value - 1) == 5
    assert mm(product(M=0), c=None, s=None, w=None, y=None, ws=None) == 0


def problem(**kw):
    return filled(m.Problem, dict(T=16, H=32, I=24, E=4, K=2, dtype=m.BF16, ids_dtype=m.I32, Is=0), kw)


@pytest.mark.parametrize("bad,flags,code", [
    (dict(dtype=m.F32), 0, 3), (dict(Is=24), 0, 2), (dict(H=131080, I=8), 0, 2), (dict(H=8, I=131080), 0, 2),
    (dict(T=1 << 24, H=8), 0, 2), (dict(T=1 << 20, H=4096, I=8), 0, 2), (dict(K=33), 0, 2), (dict(), m.PIPELINE, 2),
    (dict(T=1 << 23, H=128, I=8192, K=32), 0, 2), (dict(T=1 << 23, H=128, I=4096, K=32), 0, 2),
    (dict(), m.BULK, 2), (dict(T=-1), 0, 2)], ids=str)
def test_int8_forward_rejects(lib, bad, flags, code):
    p, n = problem(**bad), ctypes.c_size_t()
    assert lib.moe_ffn_int8_workspace_size(ctypes.byref(p), flags, ctypes.byref(n)) == code
    assert lib.moe_ffn_int8_fwd(ctypes.byref(p), *[vp(FAKE)] * 7, BIG, flags, None) == code
    assert lib.moe_ffn_last_error()


def test_int8_forward_pointers(lib):
    p, n = problem(), ctypes.c_size_t()
    assert lib.moe_ffn_int8_workspace_size(ctypes.byref(p), 0, ctypes.byref(n)) == 0
    for i in range(7):
        a = [vp(FAKE)] * 7
        a[i] = None
        assert lib.moe_ffn_int8_fwd(ctypes.byref(p), *a, BIG, 0, None) == 1
        a[i] = vp(FAKE + 2)
        assert lib.moe_ffn_int8_fwd(ctypes.byref(p), *a, BIG, 0, None) == 4
    assert lib.moe_ffn_int8_fwd(ctypes.byref(p), *[vp(FAKE)] * 7, n.value - 1, 0, None) == 5
    assert lib.moe_ffn_int8_fwd(None, *[vp(FAKE)] * 7, BIG, 0, None) == 1
    empty = problem(T=0)
    assert lib.moe_ffn_int8_fwd(ctypes.byref(empty), *[None] * 7, 0, 0, None) == 0


def int8_weight(E=1, Kd=32, N=32, panels=1, dtype=torch.bfloat16):
    return m.Int8Weight(torch.zeros(1 << 14, dtype=torch.uint8), E, Kd, N, panels, dtype)


def test_int8_tensors():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    w = int8_weight()
    for call in (lambda: m.moe_ffn_int8_quantize(torch.zeros(1, 32, 32)), lambda: m.moe_ffn_int8_dequantize(w),
                 lambda: m.moe_ffn_int8_pack(torch.zeros(32, 32, dtype=torch.int8), torch.zeros(32)),
                 lambda: m.moe_ffn_int8_quantize_rows(x), lambda: m.moe_ffn_int8_mm(x, w)):
        with pytest.raises(m.MoEFFNError, match="GPU") as ei:
            call()
        assert ei.value.status == 1


@pytest.mark.parametrize("dtype", [torch.float16, torch.int8, None])
def test_packed_weights_of_another_dtype(dtype):
    w = int8_weight(dtype=dtype)
    for call in (lambda: m.moe_ffn_int8_dequantize(w), lambda: w.nbytes):
        with pytest.raises(m.MoEFFNError) as ei:
            call()
        assert ei.value.status == 3


def test_the_size_of_packed_weights_follows_their_sizes():
    w = int8_weight(Kd=128)
    assert w.nbytes == 128 * 32 + 256  # 32 scales, rounded up to 256 bytes
    w.E, w.N = 3, 64
    assert w.nbytes == 3 * 128 * 64 + 768


@pytest.mark.parametrize("x_grad,gate_grad", [(True, False), (False, True)])
def test_int8_inputs_that_require_a_gradient(x_grad, gate_grad):
    x = torch.ones(4, 32, dtype=torch.bfloat16, requires_grad=x_grad)
    gates = torch.ones(4, 1, requires_grad=gate_grad)
    ids = torch.zeros(4, 1, dtype=torch.int32)
    call = lambda: m.moe_ffn_int8_fwd(x, ids, gates, int8_weight(), int8_weight())
    with pytest.raises(m.MoEFFNError, match="no gradient") as ei:
        call()
    assert ei.value.status == 3
    with torch.no_grad(), pytest.raises(m.MoEFFNError) as ei:
        call()
    assert ei.value.status == 1
