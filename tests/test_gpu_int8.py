"""int8 weights and rows on the GPU: codes and scales bit for bit against the 64-bit numpy
reference, the product within its three fp32 roundings and the output's, and the layer within the
tolerance that the reference derives per output."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import products as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def as_f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rounded(v, dtype):
    """fp64 values code * scale (exact in fp64) rounded to fp32 and then to dtype, as fp64."""
    with np.errstate(over="ignore", invalid="ignore"):
        return as_f64(torch.from_numpy(v.astype(np.float32)).to(DT[dtype]))


# ---- weights -----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,panels", [
    ((1, 8, 8), 1), ((2, 8, 16), 2), ((1, 32, 32), 1), ((3, 64, 64), 2), ((2, 40, 72), 1),
    ((2, 264, 400), 2), ((1, 200, 264), 1), ((2, 512, 96), 2), ((1, 1000, 40), 1),
    ((5, 96, 1024), 2), ((1, 72, 4096), 1), ((1024, 8, 8), 1), ((1, 131072, 8), 1)], ids=str)
def test_quantize_weights(gpu_lib, shape, panels, dtype):
    say(f"[int8] quantize {shape} panels={panels} {dtype}")
    rng = np.random.default_rng(list(shape))
    w = rng.standard_normal(shape) * np.exp(3 * rng.standard_normal((shape[0], 1, shape[2])))
    t = torch.from_numpy(w.astype(np.float32)).to(DT[dtype]).cuda()
    p = gpu_lib.moe_ffn_int8_quantize(t, panels=panels)
    back = gpu_lib.moe_ffn_int8_dequantize(p)
    torch.cuda.synchronize()
    q, s = ref.int8_codes(as_f64(t), 1)
    assert back.dtype == t.dtype and back.shape == t.shape
    np.testing.assert_array_equal(as_f64(back), rounded(q * s[:, None], dtype))
    # the same codes and scales packed give the same bytes, padding and all
    again = gpu_lib.moe_ffn_int8_pack(torch.from_numpy(q.astype(np.int8)).cuda(),
                                      torch.from_numpy(s.astype(np.float32)).cuda(), panels, t.dtype)
    tail = 4 * shape[0] * -(-(shape[2] // panels) // 32) * 32 * panels  # bytes of scales
    used = p.nbytes - (-tail % 256)
    assert again.nbytes == p.nbytes and torch.equal(again.data[:used], p.data[:used])


def special(n=64):
    """Vectors (columns) of n values: ties, steps beside ties, zeros, subnormals, huge, non-finite."""
    rng = np.random.default_rng(2)
    c = np.zeros((n, 32), np.float32)
    c[:, 0] = np.tile([127, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 125.5], n // 8)
    c[:, 1] = np.tile([254, 1, 3, 5, -1, -3, 253, -251], n // 8)
    c[:, 2] = np.nextafter(c[:, 0], np.float32(1e9))
    c[0, 2] = 127
    c[:, 3] = np.nextafter(c[:, 0], np.float32(-1e9))
    c[0, 3] = 127
    c[:, 4] = -0.0
    c[:, 5] = rng.standard_normal(n) * 2.0 ** -130
    c[:, 6] = rng.standard_normal(n) * 2.0 ** 124
    c[3, 7], c[40, 8], c[41, 9] = np.nan, np.inf, -np.inf
    c[5, 7:10] = 3
    c[:, 10] = np.float32(2.0 ** -149) * rng.integers(-200, 200, n)
    c[:, 11] = np.float32(2.0 ** -149)
    c[:, 12] = np.float32(3.3895314e38)  # bf16's largest value
    c[:, 13] = 2.0 ** rng.integers(-40, 0, n)
    c[7, 14] = -5.0
    c[:, 15:] = rng.standard_normal((n, 17)) * 2.0 ** np.linspace(-120, 120, 17)
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_special_values(gpu_lib, dtype):
    say(f"[int8] special values {dtype}")
    t = torch.from_numpy(special()).to(DT[dtype]).cuda()
    back = gpu_lib.moe_ffn_int8_dequantize(gpu_lib.moe_ffn_int8_quantize(t))[0]
    rows = gpu_lib.moe_ffn_int8_quantize_rows(t.t().contiguous())
    torch.cuda.synchronize()
    q, s = ref.int8_codes(as_f64(t), 0)
    np.testing.assert_array_equal(as_f64(back), rounded(q * s, dtype))
    np.testing.assert_array_equal(rows.codes.cpu().numpy(), q.T)
    np.testing.assert_array_equal(as_f64(rows.scales), s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_quotient_near_a_tie(gpu_lib, dtype):
    """For many scales, the values around each middle of two codes."""
    say(f"[int8] ties {dtype}")
    rng = np.random.default_rng(6)
    top = torch.from_numpy((rng.random(512) + 0.5).astype(np.float32)).to(DT[dtype]).float().numpy()
    s = (top.astype(np.float64) / 127).astype(np.float32)
    mid = ((np.arange(-127, 127) + 0.5) * s[:, None].astype(np.float64)).astype(np.float32)
    v = np.concatenate([top[:, None], mid, np.nextafter(mid, np.float32(9)), np.nextafter(mid, np.float32(-9)),
                        np.zeros((512, 5), np.float32)], 1)
    v = np.clip(v, -top[:, None], top[:, None])
    t = torch.from_numpy(v).to(DT[dtype]).cuda()
    rows = gpu_lib.moe_ffn_int8_quantize_rows(t)
    q, sc = ref.int8_codes(as_f64(t), 1)
    np.testing.assert_array_equal(rows.codes[:, :v.shape[1]].cpu().numpy(), q)
    np.testing.assert_array_equal(as_f64(rows.scales), sc)


def test_quantize_past_32_bit_offsets(gpu_lib):
    E, Kd, N = 40, 4096, 16384  # 2.7e9 values
    say(f"[int8] quantize {E}x{Kd}x{N}")
    w = torch.empty(E, Kd, N, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e].normal_()
    back = gpu_lib.moe_ffn_int8_dequantize(gpu_lib.moe_ffn_int8_quantize(w, panels=2))
    for e in (0, 31, 39):
        one = gpu_lib.moe_ffn_int8_quantize(w[e], panels=2)
        assert torch.equal(gpu_lib.moe_ffn_int8_dequantize(one)[0], back[e])
    assert not torch.equal(back[31], back[39])


# ---- rows --------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,Kd", [(1, 8), (1, 7168), (3, 72), (5, 1024), (4, 1032), (33, 264), (130, 2048),
                                  (2, 131072), (20000, 24), (17000, 1040)])
def test_quantize_rows(gpu_lib, M, Kd, dtype):
    say(f"[int8] rows {M}x{Kd} {dtype}")
    rng = np.random.default_rng([M, Kd])
    v = rng.standard_normal((M, Kd)).astype(np.float32) * np.exp(2 * rng.standard_normal((M, 1))).astype(np.float32)
    t = torch.from_numpy(v).to(DT[dtype]).cuda()
    r = gpu_lib.moe_ffn_int8_quantize_rows(t)
    assert r.Kd == Kd and r.dtype == t.dtype and r.codes.shape == (M, -(-Kd // 64) * 64)
    q, s = ref.int8_codes(as_f64(t), 1)
    np.testing.assert_array_equal(r.codes[:, :Kd].cpu().numpy(), q)
    assert not r.codes[:, Kd:].any()
    np.testing.assert_array_equal(as_f64(r.scales), s)
    wide = torch.full((M, Kd + 48), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, 16:16 + Kd] = t
    v = gpu_lib.moe_ffn_int8_quantize_rows(wide[:, 16:16 + Kd])
    assert torch.equal(v.codes, r.codes) and torch.equal(v.scales, r.scales)


# ---- product -------------------------------------------------------------------------------

def make(M, Kd, N, E, dtype, seed=0):
    rng = np.random.default_rng([seed, M, Kd, N, E])
    x = rng.standard_normal((M, Kd)) * np.exp(rng.standard_normal((M, 1)))
    w = rng.standard_normal((E, Kd, N)) / np.sqrt(Kd)
    return (torch.from_numpy(x.astype(np.float32)).to(DT[dtype]),
            torch.from_numpy(w.astype(np.float32)).to(DT[dtype]))


def check(m, x, w, off, out, panels=1, rows=None):
    """The whole product, or of large ones the given rows."""
    pw = m.moe_ffn_int8_quantize(w.cuda(), panels=panels)
    xr = m.moe_ffn_int8_quantize_rows(x.cuda())
    o = None if off is None else off.cuda()
    p = m.Int8Product(pw._stack(), x.shape[0], m.I32 if off is None else m._ids_code(off), m._dtype_code_of(DT[out]))
    ws = torch.full((max(m.int8_mm_workspace_size(p), 16),), 0xFF, dtype=torch.uint8, device="cuda")
    y = m.moe_ffn_int8_mm(xr, pw, o, out_dtype=DT[out], ws=ws)
    torch.cuda.synchronize()
    assert y.dtype == DT[out] and y.shape == (x.shape[0], w.shape[2])
    q, s = ref.int8_codes(as_f64(x), 1)
    cw, sw = ref.int8_codes(as_f64(w), 1)
    if rows is None:
        want, got = ref.int8_mm(q, s, cw, sw, None if off is None else off.numpy()), as_f64(y)
    else:
        want, got = np.zeros((len(rows), w.shape[2])), as_f64(y[rows])
        for i, r in enumerate(rows):
            for e, (a, b) in enumerate([(0, x.shape[0])] if off is None else ref.groups(off.numpy(), x.shape[0])):
                if a <= r < b:
                    want[i] = (q[r] @ cw[e]) * s[r] * sw[e]
    tol = 3 * 2.0 ** -24 * np.abs(want)
    tol = tol + HALF[out] * (np.abs(want) + tol) + 1e-38
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    assert torch.equal(m.moe_ffn_int8_mm(x.cuda(), pw, o, out_dtype=DT[out]), y)
    return y


def offsets(M, E, seed=0, empty=(), head=0, tail=0, dtype=torch.int32):
    rng = np.random.default_rng([seed, M, E])
    p = rng.random(E) ** 2 + 0.05
    p[list(empty)] = 0
    n = M - head - tail
    c = np.bincount(rng.choice(E, n, p=p / p.sum()), minlength=E) if n else np.zeros(E, int)
    return torch.from_numpy(head + np.concatenate([[0], np.cumsum(c)])).to(dtype)


SIZES = [
    (1, 8, 8, 1), (1, 7168, 136, 1), (2, 40, 24, 3), (31, 264, 200, 1), (32, 64, 64, 1), (33, 72, 40, 1),
    (65, 128, 96, 2), (90, 1032, 520, 5), (300, 512, 256, 8), (601, 264, 200, 6), (50, 64, 48, 300),
    (400, 40, 48, 63), (400, 40, 48, 64), (400, 40, 48, 65),
]
# more 32-row tiles than the waves that split a contraction are used for: 64- and 128-row tiles
TALL = [(700, 72, 2600, 1), (1100, 200, 1504, 1), (900, 64, 3200, 2), (2049, 72, 4136, 1), (2300, 136, 4104, 3),
        (4100, 8, 2104, 1), (3000, 264, 3000, 12)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_product(gpu_lib, size, out):
    M, Kd, N, E = size
    say(f"[int8] product {size} {out}")
    x, w = make(M, Kd, N, E, "bf16" if out == "f32" else "f32")
    check(gpu_lib, x, w, offsets(M, E), out)
    if E == 1:
        check(gpu_lib, x, w, None, out)
    if N % 16 == 0:
        check(gpu_lib, x, w, offsets(M, E, seed=1, tail=M // 3), out, panels=2)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("size", TALL, ids=str)
def test_product_of_tall_tiles(gpu_lib, size, out):
    M, Kd, N, E = size
    say(f"[int8] product {size} {out}")
    x, w = make(M, Kd, N, E, "bf16")
    check(gpu_lib, x, w, offsets(M, E, head=3, tail=17), out)
    if E == 1:
        check(gpu_lib, x, w, None, out)
    if N % 16 == 0:
        check(gpu_lib, x, w, offsets(M, E, seed=1), out, panels=2)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("case", ["all outside", "empty", "int64", "wrong", "1024 groups"])
def test_product_offsets(gpu_lib, case, out):
    say(f"[int8] product {case} {out}")
    M, E = 333, 7
    off = {"all outside": lambda: torch.full((E + 1,), 100, dtype=torch.int32),
           "empty": lambda: offsets(M, E, empty=(0, 3, 4, 6), head=10, tail=11),
           "int64": lambda: offsets(M, E, dtype=torch.int64),
           "wrong": lambda: torch.tensor([-5, 40, 30, 2 ** 40, 7, -2 ** 40, 100, 50]),
           "1024 groups": lambda: offsets(M, 1024)}[case]()
    x, w = make(M, 72, 40, len(off) - 1, "bf16")
    check(gpu_lib, x, w, off, out)


def test_product_sums_are_exact(gpu_lib):
    """The longest contraction with codes of 127 and -128 throughout: 2.13e9 below 2^31."""
    say("[int8] exact sums")
    K = 131072
    codes = torch.full((K, 8), -128, dtype=torch.int8)
    codes[:, 1], codes[:, 2] = 127, 1
    codes[::2, 3] = 127
    w = gpu_lib.moe_ffn_int8_pack(codes.cuda(), torch.ones(8, device="cuda"), dtype=torch.float32)
    x = torch.full((40, K), 127.0)
    x[1] = -127.0
    y = gpu_lib.moe_ffn_int8_mm(x.cuda(), w, out_dtype=torch.float32)
    sums = 127 * codes.double().sum(0)
    want = sums.float()  # converted once
    assert torch.equal(y[0].cpu(), want) and torch.equal(y[1].cpu(), -want) and torch.equal(y[39].cpu(), want)


def test_product_non_finite(gpu_lib):
    say("[int8] non-finite")
    x, w = make(70, 64, 96, 2, "f32")
    off = torch.tensor([0, 40, 70], dtype=torch.int32)
    pw = gpu_lib.moe_ffn_int8_quantize(w.cuda())
    clean = gpu_lib.moe_ffn_int8_mm(x.cuda(), pw, off.cuda())
    x[5, 3], x[50, 0], w[1, 7, 33] = float("nan"), -float("inf"), float("inf")
    y = gpu_lib.moe_ffn_int8_mm(x.cuda(), gpu_lib.moe_ffn_int8_quantize(w.cuda()), off.cuda())
    bad = torch.zeros(70, 96, dtype=torch.bool)
    bad[5], bad[50] = True, True
    bad[40:, 33] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert torch.equal(y.cpu()[~bad], clean.cpu()[~bad])


def test_product_of_no_rows(gpu_lib):
    say("[int8] no rows")
    _, w = make(1, 64, 96, 2, "f32")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = gpu_lib.moe_ffn_int8_mm(torch.zeros(0, 64, device="cuda"), gpu_lib.moe_ffn_int8_quantize(w.cuda()), off)
    assert y.shape == (0, 96)


def test_product_past_32_bit_offsets(gpu_lib):
    M, Kd, N = (1 << 19) + 77, 64, 8192  # 8.6 GB of output
    say(f"[int8] product {M}x{Kd}x{N}")
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(M, Kd, generator=gen, device="cuda").bfloat16()
    w = gpu_lib.moe_ffn_int8_quantize(torch.randn(Kd, N, generator=gen, device="cuda"))
    y = gpu_lib.moe_ffn_int8_mm(x, w)
    last = gpu_lib.moe_ffn_int8_mm(x[-300:], w)
    assert torch.equal(y[-300:], last) and y[-300:].any()


# ---- the layer -------------------------------------------------------------------------------

def layer(T, H, I, E, K, seed=0, routing="distinct", empty=()):
    rng = np.random.default_rng([seed, T, H, I, E, K])
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    live = np.setdiff1d(np.arange(E), empty)
    if routing == "distinct":
        ids = np.stack([rng.permutation(live)[:K] for _ in range(T)])
    elif routing == "replace":
        ids = rng.choice(live, size=(T, K))
    else:
        ids = np.full((T, K), E // 2)
    gates = rng.random((T, K)).astype(np.float32) + 0.1
    up = torch.from_numpy((rng.standard_normal((E, H, 2 * I)) / np.sqrt(H)).astype(np.float32))
    down = torch.from_numpy((rng.standard_normal((E, I, H)) / np.sqrt(I)).astype(np.float32))
    return x, ids.astype(np.int32), gates, up.bfloat16(), down.bfloat16()


def run(m, data, ids_dtype=torch.int32, **kw):
    x, ids, gates, up, down = data
    p = m.Problem(x.shape[0], x.shape[1], down.shape[1], down.shape[0], ids.shape[1], m.BF16, m.I32)
    ws = torch.full((m.int8_workspace_size(p),), 0xFF, dtype=torch.uint8, device="cuda")
    y = m.moe_ffn_int8_fwd(x.cuda(), torch.from_numpy(ids).to(ids_dtype).cuda(), torch.from_numpy(gates).cuda(),
                           m.moe_ffn_int8_quantize(up.cuda(), panels=2), m.moe_ffn_int8_quantize(down.cuda()),
                           ws=ws, **kw)
    torch.cuda.synchronize()
    return y


def check_layer(m, data, **kw):
    x, ids, gates, up, down = data
    y = run(m, data, **kw)
    want, tol = ref.int8_ffn(as_f64(x), ids, gates, as_f64(up), as_f64(down))
    assert y.shape == x.shape and y.dtype == torch.bfloat16
    err = np.abs(as_f64(y) - want)
    assert (err <= tol).all(), float(np.nanmax(err / tol))
    # the tolerance is a small part of the output
    assert np.sqrt((err ** 2).mean()) <= 0.01 * np.sqrt((want ** 2).mean()) + 1e-30
    return y


SHAPES = [
    (1, 8, 8, 1, 1), (1, 256, 128, 8, 2), (2, 40, 24, 3, 2), (5, 64, 64, 4, 1),
    (31, 264, 200, 1, 1), (32, 256, 32, 1, 1), (33, 320, 40, 1, 1), (63, 128, 96, 1, 1),
    (65, 72, 136, 1, 1), (127, 192, 72, 1, 1), (129, 264, 264, 1, 1), (257, 96, 80, 2, 1),
    (333, 264, 200, 6, 2), (300, 512, 256, 8, 4), (90, 1032, 520, 5, 3), (700, 256, 192, 16, 8),
    (50, 136, 64, 300, 8), (20, 2048, 64, 4, 2), (20, 64, 2048, 4, 2), (1100, 128, 128, 3, 2),
]
# taller tiles (see test_product_of_tall_tiles)
TALL_LAYERS = [(1050, 520, 72, 2, 2), (900, 72, 1032, 2, 2), (2049, 1032, 40, 1, 1), (1100, 2056, 264, 1, 1),
               (1500, 264, 200, 64, 2), (130, 1032, 72, 16, 8), (4100, 2056, 40, 2, 1), (4033, 40, 2056, 2, 1),
               (3000, 1000, 264, 12, 4)]


@pytest.mark.parametrize("shape", SHAPES + TALL_LAYERS, ids=str)
def test_layer_sizes(gpu_lib, shape):
    say(f"[int8] layer {shape}")
    check_layer(gpu_lib, layer(*shape))


# slots in one block, in several, counted ahead, and more experts than a block's table holds; token
# rows longer than the routing launch takes along
@pytest.mark.parametrize("shape", [(4100, 40, 32, 5, 3), (8200, 72, 24, 9, 5), (650, 64, 32, 1000, 2),
                                   (9, 64, 32, 1024, 5), (20, 8200, 64, 4, 2), (5, 8192, 40, 3, 1)], ids=str)
def test_layer_every_way_of_routing(gpu_lib, shape):
    say(f"[int8] layer {shape}")
    check_layer(gpu_lib, layer(*shape, seed=9))


@pytest.mark.parametrize("routing", ["replace", "one"])
@pytest.mark.parametrize("shape", [(60, 136, 72, 9, 4), (1100, 1032, 136, 9, 4)], ids=str)
def test_layer_routings(gpu_lib, shape, routing):
    say(f"[int8] layer {shape} routing={routing}")
    check_layer(gpu_lib, layer(*shape, seed=11, routing=routing, empty=(0, 3, 8)))


def test_layer_int64_ids_and_repeat(gpu_lib):
    say("[int8] layer int64 ids")
    data = layer(100, 72, 40, 5, 2)
    y = check_layer(gpu_lib, data, ids_dtype=torch.int64)
    assert torch.equal(run(gpu_lib, data), y)


def test_layer_dropped_slots(gpu_lib):
    """Slots with an id out of range contribute nothing; the check names them."""
    say("[int8] layer dropped slots")
    x, ids, gates, up, down = layer(80, 72, 40, 5, 2)
    ids[3, 1], ids[7], ids[79, 0] = -1, 5, 1 << 30
    y = run(gpu_lib, (x, ids, gates, up, down))
    keep, g = np.where((ids < 0) | (ids > 4), 0, ids), np.where((ids < 0) | (ids > 4), 0, gates)
    want, tol = ref.int8_ffn(as_f64(x), keep, g, as_f64(up), as_f64(down))
    assert (np.abs(as_f64(y) - want) <= tol).all() and not y[7].any()
    for kw in (dict(check_ids=True), dict(flags=gpu_lib.CHECK_STATUS)):
        with pytest.raises(gpu_lib.MoEFFNError) as ei:
            run(gpu_lib, (x, ids, gates, up, down), **kw)
        assert ei.value.status == 6


def test_layer_nan_tokens(gpu_lib):
    say("[int8] layer NaN tokens")
    x, ids, gates, up, down = layer(70, 72, 40, 3, 2)
    clean = run(gpu_lib, (x, ids, gates, up, down))
    x[5, 3], x[60, 71] = float("nan"), float("inf")
    y = run(gpu_lib, (x, ids, gates, up, down))
    keep = [t for t in range(70) if t not in (5, 60)]
    assert torch.isnan(y[[5, 60]]).all() and torch.equal(y[keep], clean[keep])


def test_layer_of_no_tokens(gpu_lib):
    say("[int8] layer of no tokens")
    _, _, _, up, down = layer(1, 72, 40, 3, 2)
    y = gpu_lib.moe_ffn_int8_fwd(torch.zeros(0, 72, dtype=torch.bfloat16, device="cuda"),
                                 torch.zeros(0, 2, dtype=torch.int32, device="cuda"),
                                 torch.zeros(0, 2, device="cuda"),
                                 gpu_lib.moe_ffn_int8_quantize(up.cuda(), panels=2),
                                 gpu_lib.moe_ffn_int8_quantize(down.cuda()))
    assert y.shape == (0, 72)


def test_layer_against_its_parts(gpu_lib):
    """The layer as its operators compose it: routing, row quantisation, two products, combine."""
    say("[int8] layer from its parts")
    T, H, I, E, K = 120, 264, 200, 6, 2
    x, ids, gates, up, down = layer(T, H, I, E, K, seed=3)
    y = run(gpu_lib, (x, ids, gates, up, down))
    _, off, slot, pos, _ = gpu_lib.moe_ffn_route(torch.from_numpy(ids).cuda(), E)
    pu, pd = gpu_lib.moe_ffn_int8_quantize(up.cuda(), panels=2), gpu_lib.moe_ffn_int8_quantize(down.cuda())
    h = gpu_lib.moe_ffn_int8_mm(x.cuda()[(slot // K).long()], pu, off, out_dtype=torch.float32)
    act = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
    o = gpu_lib.moe_ffn_int8_mm(act, pd, off, out_dtype=torch.float32)[pos.long()].view(T, K, H)
    want = (torch.from_numpy(gates).cuda().unsqueeze(2) * o).sum(1)
    # the rounding of y to bf16, and an act code now and then that moved by one
    assert float((y.float() - want).abs().max() / want.abs().max()) <= 2.0 ** -6


def test_graph_replays(gpu_lib):
    """Layer and product captured with one workspace each, replayed on other inputs between eager
    calls that use other workspaces."""
    say("[int8] graph")
    T, H, I, E, K = 96, 264, 200, 6, 2
    x, ids, gates, up, down = (t.cuda() if torch.is_tensor(t) else torch.from_numpy(t).cuda()
                               for t in layer(T, H, I, E, K))
    pu, pd = gpu_lib.moe_ffn_int8_quantize(up, panels=2), gpu_lib.moe_ffn_int8_quantize(down)
    off = torch.tensor([0, 10, 10, 40, 60, 80, 90], dtype=torch.int32, device="cuda")

    def step():
        return gpu_lib.moe_ffn_int8_fwd(x, ids, gates, pu, pd), gpu_lib.moe_ffn_int8_mm(x, pu, off)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in range(4):
        x2, ids2, gates2, _, _ = layer(T, H, I, E, K, seed=seed)
        x.copy_(x2), ids.copy_(torch.from_numpy(ids2)), gates.copy_(torch.from_numpy(gates2))
        off[-1] = 90 - seed
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_two_streams(gpu_lib):
    say("[int8] two streams")
    a, b = layer(300, 512, 256, 8, 4), layer(90, 264, 200, 6, 2)
    alone = run(gpu_lib, a), run(gpu_lib, b)

    def put(d):
        x, ids, gates, up, down = d
        return (x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(gates).cuda(),
                gpu_lib.moe_ffn_int8_quantize(up.cuda(), panels=2), gpu_lib.moe_ffn_int8_quantize(down.cuda()))

    a, b = put(a), put(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ya = gpu_lib.moe_ffn_int8_fwd(*a)
        with torch.cuda.stream(s2):
            yb = gpu_lib.moe_ffn_int8_fwd(*b)
        torch.cuda.synchronize()
        assert torch.equal(ya, alone[0]) and torch.equal(yb, alone[1])


def test_tensors_that_are_refused(gpu_lib):
    say("[int8] refusals")
    m, E = gpu_lib, gpu_lib.MoEFFNError
    x, w = (t.cuda() for t in make(16, 32, 48, 2, "bf16"))
    pw, off = m.moe_ffn_int8_quantize(w), torch.tensor([0, 8, 16], dtype=torch.int32, device="cuda")
    r = m.moe_ffn_int8_quantize_rows(x)
    short = m.Int8Weight(pw.data[:64], 2, 32, 48, 1, torch.bfloat16)
    for call in (
            lambda: m.moe_ffn_int8_mm(x, pw), lambda: m.moe_ffn_int8_mm(x[:, :24], pw, off),
            lambda: m.moe_ffn_int8_mm(x.half(), pw, off), lambda: m.moe_ffn_int8_mm(x, pw, off[:2]),
            lambda: m.moe_ffn_int8_mm(x, pw, off.cpu()), lambda: m.moe_ffn_int8_mm(x, pw, off.float()),
            lambda: m.moe_ffn_int8_mm(x, pw, off, out_dtype=torch.float16), lambda: m.moe_ffn_int8_mm(x, short, off),
            lambda: m.moe_ffn_int8_mm(m.Int8Rows(r.codes, r.scales[:8], 32, x.dtype), pw, off),
            lambda: m.moe_ffn_int8_mm(m.Int8Rows(r.codes[:, :32].contiguous(), r.scales, 32, x.dtype), pw, off),
            lambda: m.moe_ffn_int8_mm(m.Int8Rows(r.codes.short(), r.scales, 32, x.dtype), pw, off),
            lambda: m.moe_ffn_int8_quantize_rows(x.t()), lambda: m.moe_ffn_int8_quantize_rows(x[0]),
            lambda: m.moe_ffn_int8_quantize(w.transpose(1, 2)), lambda: m.moe_ffn_int8_quantize(w, panels=4),
            lambda: m.moe_ffn_int8_dequantize(short),
            lambda: m.moe_ffn_int8_pack(w, torch.ones(2, 48, device="cuda")),
            lambda: m.moe_ffn_int8_pack(w.to(torch.int8), torch.ones(48, device="cuda")),
            lambda: m.moe_ffn_int8_fwd(x, torch.zeros(16, 1, dtype=torch.int32, device="cuda"),
                                       torch.ones(16, 1, device="cuda"), pw, pw)):
        with pytest.raises(E):
            call()
