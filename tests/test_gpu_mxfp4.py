"""MXFP4 weights on the GPU: quantisation bit for bit against the 64-bit numpy reference, and the
expert FFN on packed weights within the tolerance that the reference derives per output (rounding
of sums, of act values next to a rounding border, of o and y)."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as ops

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def as_f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ---- quantisation --------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,panels", [
    ((1, 8, 8), 1), ((2, 8, 16), 2), ((1, 32, 32), 1), ((3, 64, 64), 2), ((2, 40, 72), 1),
    ((2, 264, 400), 2), ((1, 200, 264), 1), ((2, 512, 96), 2), ((1, 1000, 40), 1),
    ((5, 96, 1024), 2), ((1, 72, 4096), 1), ((1024, 8, 8), 1)], ids=str)
def test_quantize_round_trip(gpu_lib, shape, panels, dtype):
    say(f"[mxfp4] quantize {shape} panels={panels} {dtype}")
    rng = np.random.default_rng(list(shape))
    w = rng.standard_normal(shape) * np.exp(3 * rng.standard_normal((shape[0], 1, shape[2])))
    t = torch.from_numpy(w.astype(np.float32)).to(DT[dtype]).cuda()
    p = gpu_lib.moe_ffn_mxfp4_quantize(t, panels=panels)
    q = gpu_lib.moe_ffn_mxfp4_dequantize(p)
    torch.cuda.synchronize()
    assert q.dtype == t.dtype and q.shape == t.shape
    np.testing.assert_array_equal(as_f64(q), ops.mx_quantize_columns(as_f64(t)))
    # values on the grid come back as they are
    again = gpu_lib.moe_ffn_mxfp4_dequantize(gpu_lib.moe_ffn_mxfp4_quantize(q, panels=panels))
    assert torch.equal(again, q)


def special_columns():
    """Columns of 64 rows, two blocks: ties, saturation, zeros, subnormals, huge, non-finite."""
    rng = np.random.default_rng(2)
    c = np.zeros((64, 24), np.float32)
    c[:, 0] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0], 8)
    c[:, 1] = np.tile([7.0, 7.999, -6.5, 0.1, 5.001, 4.999, 3.501, 3.499], 8)
    c[:, 2] = -0.0
    c[:, 3] = rng.standard_normal(64) * 2.0 ** -130
    c[:, 4] = rng.standard_normal(64) * 2.0 ** 124
    c[3, 5] = np.nan
    c[40, 6] = np.inf
    c[41, 7] = -np.inf
    c[:, 8] = 2.0 ** -126
    c[:, 9] = np.float32(2.0 ** -149)
    c[:, 10] = np.float32(3.3895314e38)  # bf16's largest value
    c[0, 11] = 1.0
    c[32:, 12] = rng.standard_normal(32)
    c[:, 13] = 2.0 ** rng.integers(-40, 0, 64)
    c[:, 14:] = rng.standard_normal((64, 10)) * 2.0 ** np.arange(-125, -105, 2)
    c[5, 14:19] = 1.0
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_special_values(gpu_lib, dtype):
    say(f"[mxfp4] special values {dtype}")
    t = torch.from_numpy(special_columns()[None]).to(DT[dtype]).cuda()
    q = gpu_lib.moe_ffn_mxfp4_dequantize(gpu_lib.moe_ffn_mxfp4_quantize(t))
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        ref = ops.mx_quantize_columns(as_f64(t))
    np.testing.assert_array_equal(as_f64(q), ref)


@pytest.mark.parametrize("shape,panels", [((1, 1 << 25, 8), 1), ((1, 8, 1 << 25), 2)], ids=str)
def test_quantize_long_and_thin(gpu_lib, shape, panels):
    say(f"[mxfp4] quantize {shape}")
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda",
                        dtype=torch.bfloat16)
    gen = torch.Generator("cuda").manual_seed(7)
    w = grid[torch.randint(0, 15, shape, device="cuda", generator=gen, dtype=torch.int32)]
    w[:, ::8] = 6  # every block's scale is 1, so every value is kept
    q = gpu_lib.moe_ffn_mxfp4_dequantize(gpu_lib.moe_ffn_mxfp4_quantize(w, panels=panels))
    torch.cuda.synchronize()
    assert torch.equal(q, w)


def test_quantize_past_32_bit_offsets(gpu_lib):
    E, Kd, N = 40, 4096, 16384  # 2.7e9 values
    say(f"[mxfp4] quantize {E}x{Kd}x{N}")
    w = torch.empty(E, Kd, N, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e].normal_()
    p = gpu_lib.moe_ffn_mxfp4_quantize(w, panels=2)
    q = gpu_lib.moe_ffn_mxfp4_dequantize(p)
    for e in (0, 31, 39):
        one = gpu_lib.moe_ffn_mxfp4_quantize(w[e:e + 1].contiguous(), panels=2)
        assert torch.equal(gpu_lib.moe_ffn_mxfp4_dequantize(one)[0], q[e])


# ---- expert FFN ------------------------------------------------------------------------

def make(T, H, I, E, K, seed=0, routing="distinct", empty=()):
    rng = np.random.default_rng([seed, T, H, I, E, K])
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    live = np.setdiff1d(np.arange(E), empty)
    if routing == "distinct":
        ids = np.stack([rng.permutation(live)[:K] for _ in range(T)]) if T else np.zeros((0, K))
    elif routing == "replace":
        ids = rng.choice(live, size=(T, K))
    else:
        ids = np.full((T, K), E // 2)
    gates = rng.random((T, K)).astype(np.float32) + 0.1
    up = torch.from_numpy((rng.standard_normal((E, H, 2 * I)) / np.sqrt(H)).astype(np.float32))
    down = torch.from_numpy((rng.standard_normal((E, I, H)) / np.sqrt(I)).astype(np.float32))
    return x, ids.astype(np.int32), gates, up.bfloat16(), down.bfloat16()


def poisoned(m, x, ids, down, act):
    """A workspace full of NaN scale codes."""
    p = m.Problem(x.shape[0], x.shape[1], down.shape[1], down.shape[0], ids.shape[1], m.BF16,
                  m.I32)
    return torch.full((m.mxfp4_workspace_size(p, act),), 0xFF, dtype=torch.uint8, device="cuda")


def run(m, data, act, ids_dtype=torch.int32, **kw):
    x, ids, gates, up, down = data
    pu = m.moe_ffn_mxfp4_quantize(up.cuda(), panels=2)
    pd = m.moe_ffn_mxfp4_quantize(down.cuda())
    y = m.moe_ffn_mxfp4_fwd(x.cuda(), torch.from_numpy(ids).to(ids_dtype).cuda(),
                            torch.from_numpy(gates).cuda(), pu, pd, act=act,
                            ws=poisoned(m, x, ids, down, act), **kw)
    torch.cuda.synchronize()
    return y


def check(m, data, act, **kw):
    x, ids, gates, up, down = data
    y = run(m, data, act, **kw)
    ref, tol = ops.mxfp4_ffn(as_f64(x), ids, gates, as_f64(up), as_f64(down), act)
    assert y.shape == x.shape and y.dtype == torch.bfloat16
    err = np.abs(as_f64(y) - ref)
    assert (err <= tol).all(), float(np.nanmax(err / tol))
    # the tolerance is a small part of the output
    if ref.size:
        assert np.sqrt((err ** 2).mean()) <= 0.01 * np.sqrt((ref ** 2).mean()) + 1e-30
    return y


# (T, H, I, E, K): single tokens, tile edges in tokens (31-33, 63-65, 127-129, 255-257 rows of
# one expert), in columns (multiples of 8, not of 32) and in the contraction (parts of 64 and 256)
SHAPES = [
    (1, 8, 8, 1, 1), (1, 256, 128, 8, 2), (2, 40, 24, 3, 2), (5, 64, 64, 4, 1),
    (31, 264, 200, 1, 1), (32, 256, 32, 1, 1), (33, 320, 40, 1, 1), (63, 128, 96, 1, 1),
    (65, 72, 136, 1, 1), (127, 192, 72, 1, 1), (129, 264, 264, 1, 1), (255, 64, 48, 1, 1),
    (257, 96, 80, 2, 1), (333, 264, 200, 6, 2), (300, 512, 256, 8, 4), (90, 1032, 520, 5, 3),
    (700, 256, 192, 16, 8), (50, 136, 64, 300, 8), (20, 2048, 64, 4, 2), (20, 64, 2048, 4, 2),
    (600, 512, 384, 2, 1), (1100, 128, 128, 3, 2),
]


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_ffn_sizes(gpu_lib, shape, act):
    say(f"[mxfp4] ffn {shape} {act}")
    check(gpu_lib, make(*shape), act)


# more 32-row tiles than the waves that split a contraction are used for: 64-row tiles, and from
# 8192 of them on, and more than 48 rows an expert, 128-row tiles
TALL = [(1050, 520, 72, 2, 2), (900, 72, 1032, 2, 2), (1111, 1000, 200, 5, 2), (2049, 1032, 40, 1, 1),
        (1100, 2056, 1032, 1, 1), (1500, 264, 200, 64, 2), (130, 1032, 72, 16, 8),
        (4100, 2056, 40, 2, 1), (4033, 40, 2056, 2, 1), (3000, 1000, 264, 12, 4),
        (820, 2056, 136, 5, 5), (4097, 2056, 1032, 1, 1), (4200, 2120, 8, 3, 1)]


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("shape", TALL, ids=str)
def test_ffn_sizes_of_tall_tiles(gpu_lib, shape, act):
    say(f"[mxfp4] ffn {shape} {act}")
    check(gpu_lib, make(*shape, seed=10), act)


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("routing", ["replace", "one"])
@pytest.mark.parametrize("shape", [(1100, 1032, 136, 9, 4), (1400, 1544, 136, 9, 4)], ids=str)
def test_ffn_routings_of_tall_tiles(gpu_lib, shape, routing, act):
    say(f"[mxfp4] ffn {shape} routing={routing} {act}")
    check(gpu_lib, make(*shape, seed=11, routing=routing, empty=(0, 3, 8)), act)


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("shape", [(4100, 40, 32, 5, 3), (8200, 72, 24, 9, 5), (650, 64, 32, 1000, 2),
                                   (9, 64, 32, 1024, 5)], ids=str)
def test_ffn_every_way_of_routing(gpu_lib, shape, act):
    """Slots over several blocks, counted ahead, and more experts than a block's table holds."""
    say(f"[mxfp4] routing {shape} {act}")
    check(gpu_lib, make(*shape, seed=9), act)


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("routing", ["replace", "one"])
def test_ffn_routings(gpu_lib, routing, act):
    say(f"[mxfp4] ffn routing={routing} {act}")
    check(gpu_lib, make(210, 264, 136, 9, 4, seed=1, routing=routing, empty=(0, 3, 8)), act,
          ids_dtype=torch.int64)


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
def test_ffn_dropped_slots_and_rows_without_any(gpu_lib, act):
    say(f"[mxfp4] dropped slots {act}")
    x, ids, gates, up, down = make(150, 256, 128, 6, 3, seed=2)
    ids[::7, 1] = -1
    ids[4] = -1
    ids[77] = 6
    ids[149, 2] = 1 << 30
    data = (x, ids, gates, up, down)
    y, ws = run(gpu_lib, data, act, return_ws=True)
    assert gpu_lib.read_status(ws) == gpu_lib.DEV_BAD_ID
    keep = np.where((ids < 0) | (ids >= 6), -1, ids)
    ref, tol = ops.mxfp4_ffn(as_f64(x), keep, gates, as_f64(up), as_f64(down), act)
    assert (np.abs(as_f64(y) - ref) <= tol).all()
    assert (y[4] == 0).all() and (y[77] == 0).all()
    for kw in (dict(check_ids=True), dict(flags=gpu_lib.CHECK_STATUS)):
        with pytest.raises(gpu_lib.MoEFFNError) as ei:
            run(gpu_lib, data, act, **kw)
        assert ei.value.status == 6
    ids[:] = -1
    assert (run(gpu_lib, data, act) == 0).all()


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("shape", [(40, 264, 200, 3, 2), (700, 512, 256, 2, 1)], ids=str)
def test_nan_and_infinity_stay_in_their_token(gpu_lib, shape, act):
    say(f"[mxfp4] NaN tokens {shape} {act}")
    data = make(*shape, seed=3)
    clean = run(gpu_lib, data, act)
    x = data[0].clone()
    x[3, 5] = float("nan")
    x[17, shape[1] - 1] = float("inf")
    x[18] = -float("inf")
    y = run(gpu_lib, (x,) + data[1:], act)
    bad = torch.zeros(shape[0], dtype=torch.bool, device="cuda")
    bad[[3, 17, 18]] = True
    assert y[bad].isnan().all()
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("shape", [(1100, 1032, 72, 2, 1), (4200, 2056, 72, 2, 1)], ids=str)
def test_nan_and_infinity_in_tall_tiles(gpu_lib, shape, act):
    test_nan_and_infinity_stay_in_their_token(gpu_lib, shape, act)


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
def test_ffn_extreme_activations(gpu_lib, act):
    """Zero rows, rows of tiny and of large values: scales at both ends."""
    say(f"[mxfp4] extreme rows {act}")
    x, ids, gates, up, down = make(24, 136, 72, 4, 2, seed=4)
    x = x.float()
    x[0] = 0
    x[1] = -0.0
    x[2] *= 2.0 ** -120
    x[3] *= 2.0 ** 40
    x[4] *= 2.0 ** -20
    x[5, 32:] = 0
    x[6, :32] *= 2.0 ** -126
    check(gpu_lib, (x.bfloat16(), ids, gates, up, down), act)


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
def test_repeats_workspaces_streams_and_graphs(gpu_lib, act):
    say(f"[mxfp4] repeats, streams, graphs {act}")
    m = gpu_lib
    a, b = make(120, 512, 256, 8, 2, seed=5), make(37, 512, 256, 8, 2, seed=6)
    up = m.moe_ffn_mxfp4_quantize(a[3].cuda(), panels=2)
    down = m.moe_ffn_mxfp4_quantize(a[4].cuda())
    dev = [[d[0].cuda(), torch.from_numpy(d[1]).cuda(), torch.from_numpy(d[2]).cuda()]
           for d in (a, b)]
    ws = poisoned(m, a[0], a[1], a[4], act)
    call = lambda i, w=None: m.moe_ffn_mxfp4_fwd(*dev[i], up, down, act=act, ws=w)
    ref = [call(0), call(1)]
    torch.cuda.synchronize()
    # one workspace for calls in turn, the smaller second
    for i in (0, 1, 0, 1):
        assert torch.equal(call(i, ws), ref[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(0)
    mine = call(1)
    torch.cuda.synchronize()
    assert torch.equal(other, ref[0]) and torch.equal(mine, ref[1])
    # two graphs that share a workspace, replayed in turn with eager work between
    graphs, outs = [], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(i, ws))
        graphs.append(g)
    for _ in range(3):
        for i in (0, 1):
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], ref[i])
            call(1 - i, ws)
            torch.cuda.synchronize()


def test_ffn_refusals(gpu_lib):
    say("[mxfp4] refusals")
    m = gpu_lib
    x, ids, gates, up, down = make(8, 64, 32, 4, 2)
    x, ids, gates = x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(gates).cuda()
    pu, pd = m.moe_ffn_mxfp4_quantize(up.cuda(), panels=2), m.moe_ffn_mxfp4_quantize(down.cuda())
    flat = m.moe_ffn_mxfp4_quantize(up.cuda())
    bad = [
        dict(a=(x, ids, gates, flat, pd)), dict(a=(x, ids, gates, pd, pu)),
        dict(a=(x.float(), ids, gates, pu, pd)), dict(a=(x[:, :32].contiguous(), ids, gates, pu, pd)),
        dict(a=(x, ids[:7], gates, pu, pd)), dict(a=(x, ids, gates.double(), pu, pd)),
        dict(a=(x, ids.short(), gates, pu, pd)), dict(a=(x, ids, gates, pu, pd), act="mxfp8"),
        dict(a=(x, ids, gates, pu, pd), ws=torch.empty(64, dtype=torch.uint8, device="cuda")),
        dict(a=(x, ids, gates, pu, pd), flags=m.PIPELINE), dict(a=(x.cpu(), ids, gates, pu, pd)),
        dict(a=(x.t().contiguous().t(), ids, gates, pu, pd)),
    ]
    for kw in bad:
        with pytest.raises(m.MoEFFNError):
            m.moe_ffn_mxfp4_fwd(*kw.pop("a"), **kw)
    assert m.moe_ffn_mxfp4_fwd(x[:0], ids[:0], gates[:0], pu, pd).shape == (0, 64)


def test_short_packed_weights_are_refused(gpu_lib):
    m = gpu_lib
    x, ids, gates, up, down = make(8, 64, 32, 4, 2)
    x, ids, gates = x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(gates).cuda()
    pu, pd = m.moe_ffn_mxfp4_quantize(up.cuda(), panels=2), m.moe_ffn_mxfp4_quantize(down.cuda())
    short = lambda p: m.MXFP4Weight(p.data[:-16], p.E, p.Kd, p.N, p.panels, p.dtype)
    for u, d in ((short(pu), pd), (pu, short(pd))):
        with pytest.raises(m.MoEFFNError):
            m.moe_ffn_mxfp4_fwd(x, ids, gates, u, d)
    with pytest.raises(m.MoEFFNError):
        m.moe_ffn_mxfp4_dequantize(short(pd))


def test_router_into_quantised_layer(gpu_lib):
    """A serving step: logits, router, quantised experts; a padded token and a closed expert."""
    say("[mxfp4] router into the layer")
    m = gpu_lib
    x, _, _, up, down = make(77, 264, 136, 16, 4, seed=8)
    l = torch.randn(77, 16, generator=torch.Generator().manual_seed(9))
    l[:, 5] = -float("inf")
    l[70:] = -float("inf")
    kw = dict(score="sigmoid", groups=4, topk_groups=2, group_top=2, scale=2.5)
    w, ids = m.moe_ffn_router_fwd(l.cuda(), 4, **kw)
    y = m.moe_ffn_mxfp4_fwd(x.cuda(), ids, w, m.moe_ffn_mxfp4_quantize(up.cuda(), panels=2),
                            m.moe_ffn_mxfp4_quantize(down.cuda()), act="mxfp6")
    rw, rid = ops.router(l.numpy(), 4, **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    ref, tol = ops.mxfp4_ffn(as_f64(x), rid, rw, as_f64(up), as_f64(down), "mxfp6")
    # the gates' own half steps (the router's test derives them)
    tol = tol + 32 * 2.0 ** -24 * np.abs(ref).max()
    assert (np.abs(as_f64(y) - ref) <= tol).all()
    assert (y[70:] == 0).all()


def test_close_to_the_bf16_layer_on_grid_weights(gpu_lib):
    """With weights on the grid the only difference to moe_ffn_fwd is the activations' rounding.
    e2m3: at most 2^-4 of the value or of the block's unit, and the unit is about the rms of 32
    normal values, so 2^-4 sqrt(2) at most in either of two places; added up they stay below 2^-2,
    and as random errors (1 / sqrt(3) of their bound) below 2^-3."""
    say("[mxfp4] against the bf16 layer")
    m = gpu_lib
    x, ids, gates, up, down = make(200, 512, 256, 8, 2, seed=10)
    pu, pd = m.moe_ffn_mxfp4_quantize(up.cuda(), panels=2), m.moe_ffn_mxfp4_quantize(down.cuda())
    gu, gd = m.moe_ffn_mxfp4_dequantize(pu), m.moe_ffn_mxfp4_dequantize(pd)
    ids, gates = torch.from_numpy(ids).cuda(), torch.from_numpy(gates).cuda()
    y = m.moe_ffn_mxfp4_fwd(x.cuda(), ids, gates, pu, pd, act="mxfp6").float()
    ref = m.moe_ffn_fwd(x.cuda(), ids, gates, gu, gd).float()
    assert ((y - ref).norm() / ref.norm()).item() < 2.0 ** -3


def test_outputs_past_32_bit_offsets(gpu_lib):
    """o [T K, H] passes 2^31 elements: the last tokens equal the same tokens in a small call."""
    m = gpu_lib
    T, H, I, E, K = 70000, 4096, 32, 4, 8
    say(f"[mxfp4] ffn {(T, H, I, E, K)}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    gates = torch.rand(T, K, generator=g, device="cuda")
    up = (torch.randn(E, H, 2 * I, generator=g, device="cuda") / 64).bfloat16()
    down = (torch.randn(E, I, H, generator=g, device="cuda") / 6).bfloat16()
    pu, pd = m.moe_ffn_mxfp4_quantize(up, panels=2), m.moe_ffn_mxfp4_quantize(down)
    y = m.moe_ffn_mxfp4_fwd(x, ids, gates, pu, pd)
    n = 40
    for at in (0, 35000, T - n):
        sl = slice(at, at + n)
        small = m.moe_ffn_mxfp4_fwd(x[sl].contiguous(), ids[sl].contiguous(),
                                    gates[sl].contiguous(), pu, pd)
        # sums may be taken in another order there, so an act value next to a border may differ
        d = (y[sl].float() - small.float())
        assert (d.norm() / small.float().norm()).item() < 5e-3
