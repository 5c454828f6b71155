"""The grouped products and their gradients on the GPU against the 64-bit numpy reference.

An output may be off by its one rounding (half a step: 2^-8 of a bf16 value, 2^-24 of an fp32
one) and by the roundings of its sum in fp32: at most one a product, each at most a step (the matrix
instruction may cut off), 2^-23 of the sum of the products' magnitudes."""

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


def within(got, want, mag, terms, dtype):
    sums = (np.asarray(terms) + 2) * 2.0 ** -23 * mag
    tol = sums + HALF[dtype] * (np.abs(want) + sums) + 1e-38
    err = np.abs(as_f64(got) - want)
    assert got.dtype == DT[dtype] and tuple(got.shape) == want.shape
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:5].tolist())


def make(M, Kd, N, E, dtype, transposed, sizes, seed=0, offsets_dtype=torch.int32):
    """sizes: rows of each group, behind `first` rows of no group."""
    rng = np.random.default_rng([seed, M, Kd, N, E])
    t = lambda a: torch.from_numpy(a.astype(np.float32)).to(DT[dtype])
    x, dy = t(rng.standard_normal((M, Kd))), t(rng.standard_normal((M, N)))
    w = t(rng.standard_normal((E, N, Kd) if transposed else (E, Kd, N)) / np.sqrt(Kd))
    first, counts = sizes
    off = first + np.concatenate([[0], np.cumsum(counts)])
    return x, w, dy, torch.from_numpy(off).to(offsets_dtype)


def poisoned(m, x, w, off, transposed):
    Kd, N = (w.shape[2], w.shape[1]) if transposed else w.shape[1:]
    g = m.Grouped(x.shape[0], w.shape[0], Kd, N, Kd, m._dtype_code(x), m._ids_code(off), int(transposed))
    return torch.full((max(m.grouped_workspace_size(g), 16),), 0xFF, dtype=torch.uint8, device="cuda")


def check(m, data, dtype, transposed):
    x, w, dy, off = data
    E, M = w.shape[0], x.shape[0]
    dx_, dw_, dy_, do_ = x.cuda(), w.cuda(), dy.cuda(), off.cuda()
    ws = poisoned(m, x, w, off, transposed)
    y = m.moe_ffn_grouped_mm_fwd(dx_, dw_, do_, transposed=transposed, ws=ws)
    ws.fill_(0xFF)
    gx, gw = m.moe_ffn_grouped_mm_bwd(dy_, dx_, dw_, do_, transposed=transposed, ws=ws)
    torch.cuda.synchronize()
    Kd, N = (w.shape[2], w.shape[1]) if transposed else w.shape[1:]
    want, mag = ref.grouped_mm(as_f64(x), as_f64(w), off.numpy(), transposed)
    within(y, want, mag, Kd, dtype)
    (wx, mx), (ww, mw) = ref.grouped_mm_grad(as_f64(dy), as_f64(x), as_f64(w), off.numpy(), transposed)
    within(gx, wx, mx, N, dtype)
    rows = np.array([b - a for a, b in ref.groups(off.numpy(), M)]).reshape(E, 1, 1)
    within(gw, ww, mw, rows, dtype)
    # without group rows exactly zero; a second pass gives the same bits
    again = m.moe_ffn_grouped_mm_bwd(dy_, dx_, dw_, do_, transposed=transposed)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)
    assert torch.equal(m.moe_ffn_grouped_mm_fwd(dx_, dw_, do_, transposed=transposed), y)


def spread(M, E, seed=0, empty=(), head=0, tail=0):
    rng = np.random.default_rng([seed, M, E])
    p = rng.random(E) ** 2 + 0.05
    p[list(empty)] = 0
    n = M - head - tail
    return head, np.bincount(rng.choice(E, n, p=p / p.sum()), minlength=E) if n else np.zeros(E, int)


# (M, Kd, N, E): one row, tile edges in rows, columns and contraction.  In bf16 most of them take the
# kernel for few tiles (taller ones: HEIGHTS below, and test_gpu_grouped_tall.py)
SIZES = [
    (1, 8, 8, 1), (1, 256, 512, 4), (3, 40, 24, 2), (8, 512, 256, 32), (31, 72, 136, 3), (63, 64, 64, 1),
    (64, 264, 200, 1), (65, 136, 264, 1), (127, 128, 256, 1), (129, 256, 128, 1), (255, 264, 8, 2),
    (257, 8, 264, 1), (300, 256, 256, 5), (500, 384, 512, 3), (601, 264, 200, 6), (640, 512, 256, 2),
    (1000, 128, 256, 2), (700, 256, 384, 9), (90, 1032, 520, 5), (200, 64, 48, 300), (1500, 256, 256, 1),
    # columns that end inside a 256-row tile: of dx and of y in the last two
    (900, 160, 264, 2), (1300, 1288, 416, 3), (2100, 288, 2056, 2),
    # as many groups as a wave has lanes, one less, one more
    (400, 40, 48, 63), (400, 40, 48, 64), (400, 40, 48, 65),
]


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(gpu_lib, size, dtype, transposed):
    M, Kd, N, E = size
    say(f"[grouped] {size} {dtype} transposed={transposed}")
    check(gpu_lib, make(M, Kd, N, E, dtype, transposed, spread(M, E)), dtype, transposed)


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", ["head and tail", "all outside", "empty groups", "one group", "int64",
                                  "1024 groups"])
@pytest.mark.parametrize("Kd,N", [(256, 512), (72, 40)])
def test_offsets(gpu_lib, Kd, N, case, dtype, transposed):
    say(f"[grouped] {case} {Kd}x{N} {dtype} transposed={transposed}")
    M, E, kw = 333, 7, {}
    if case == "head and tail":
        sizes = spread(M, E, head=37, tail=61)
    elif case == "all outside":
        sizes = (100, np.zeros(E, int))
    elif case == "empty groups":
        sizes = spread(M, E, empty=(0, 3, 4, 6))
    elif case == "one group":
        sizes = (0, np.array([0, 0, 0, M, 0, 0, 0]))
    elif case == "1024 groups":
        E = 1024
        sizes = spread(M, E, head=3, tail=5)
        Kd, N = (256, 256) if Kd == 256 else (16, 24)
    else:
        sizes, kw = spread(M, E, tail=9), dict(offsets_dtype=torch.int64)
    check(gpu_lib, make(M, Kd, N, E, dtype, transposed, sizes, seed=1, **kw), dtype, transposed)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [[-7, 40, 30, 100, 1000], [500, 3, 2, 1, 0], [0, 2 ** 40, 5, -2 ** 40, 90],
                                 [10, 10, 10, 10, 10], [0, 50, 20, 60, 99]], ids=str)
def test_offsets_that_are_wrong(gpu_lib, off, dtype):
    """Held to the rows, and to their running maximum: never outside."""
    say(f"[grouped] offsets {off} {dtype}")
    x, w, dy, _ = make(99, 128, 256, 4, dtype, False, spread(99, 4))
    check(gpu_lib, (x, w, dy, torch.tensor(off)), dtype, False)


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Kd,N", [(256, 512), (72, 40)])
def test_strided_rows(gpu_lib, Kd, N, dtype, transposed):
    """x as columns of a wider matrix: the same results as its copy, bit for bit or within the sums."""
    say(f"[grouped] strided {Kd}x{N} {dtype} transposed={transposed}")
    x, w, dy, off = (t.cuda() for t in make(200, Kd, N, 3, dtype, transposed, spread(200, 3, tail=4)))
    wide = torch.full((200, Kd + 40), float("nan"), dtype=DT[dtype], device="cuda")
    view = wide[:, 24:24 + Kd]
    view.copy_(x)
    y = gpu_lib.moe_ffn_grouped_mm_fwd(view, w, off, transposed=transposed)
    gx, gw = gpu_lib.moe_ffn_grouped_mm_bwd(dy, view, w, off, transposed=transposed)
    want, mag = ref.grouped_mm(as_f64(x), as_f64(w), off.cpu().numpy(), transposed)
    within(y, want, mag, Kd, dtype)
    rx, rw = gpu_lib.moe_ffn_grouped_mm_bwd(dy, x, w, off, transposed=transposed)
    assert torch.equal(gx, rx) and torch.equal(gw, rw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_no_group_and_empty_groups_are_not_read(gpu_lib, dtype):
    say(f"[grouped] poisoned {dtype}")
    for Kd, N in ((256, 512), (72, 40)):
        x, w, dy, off = make(300, Kd, N, 5, dtype, False, spread(300, 5, empty=(1, 4), head=20, tail=30))
        x[:20], x[270:], dy[:20], dy[270:] = (float("nan"),) * 4
        w[1], w[4] = float("nan"), float("inf")
        x, w, dy, off = x.cuda(), w.cuda(), dy.cuda(), off.cuda()
        y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off)
        gx, gw = gpu_lib.moe_ffn_grouped_mm_bwd(dy, x, w, off)
        for t in (y, gx):
            assert torch.isfinite(t).all() and not t[:20].any() and not t[270:].any() and t[20:270].any()
        assert torch.isfinite(gw).all() and not gw[1].any() and not gw[4].any() and gw[0].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_and_inf_stay_in_their_rows(gpu_lib, dtype):
    say(f"[grouped] non-finite {dtype}")
    x, w, _, off = make(130, 128, 256, 2, dtype, False, (0, np.array([70, 60])))
    clean = gpu_lib.moe_ffn_grouped_mm_fwd(x.cuda(), w.cuda(), off.cuda())
    x[5, 3], x[100, 127] = float("nan"), float("inf")
    y = gpu_lib.moe_ffn_grouped_mm_fwd(x.cuda(), w.cuda(), off.cuda())
    keep = [r for r in range(130) if r not in (5, 100)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[5]).all() and not torch.isfinite(y[100]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_rows(gpu_lib, dtype):
    say(f"[grouped] no rows {dtype}")
    x, w = torch.zeros(0, 64, dtype=DT[dtype], device="cuda"), torch.ones(3, 64, 32, dtype=DT[dtype], device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off).shape == (0, 32)
    gx, gw = gpu_lib.moe_ffn_grouped_mm_bwd(torch.zeros(0, 32, dtype=DT[dtype], device="cuda"), x, w, off)
    assert gx.shape == (0, 64) and gw.shape == w.shape and not gw.any()


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_autograd(gpu_lib, dtype, transposed):
    """Gradients through the wrapper, from a gradient that is a broadcast (stride 0), and for one
    input alone."""
    say(f"[grouped] autograd {dtype} transposed={transposed}")
    x, w, _, off = (t.cuda() for t in make(150, 64, 48, 4, dtype, transposed, spread(150, 4, tail=11)))
    x.requires_grad_(), w.requires_grad_()
    y = gpu_lib.moe_ffn_grouped_mm(x, w, off, transposed=transposed)
    y.sum().backward()
    ones = torch.ones_like(y)
    gx, gw = gpu_lib.moe_ffn_grouped_mm_bwd(ones, x.detach(), w.detach(), off, transposed=transposed)
    assert torch.equal(x.grad, gx) and torch.equal(w.grad, gw)
    only, = torch.autograd.grad(gpu_lib.moe_ffn_grouped_mm(x, w.detach(), off, transposed=transposed).sum(), x)
    assert torch.equal(only, gx)
    only, = torch.autograd.grad(gpu_lib.moe_ffn_grouped_mm(x.detach(), w, off, transposed=transposed).sum(), w)
    assert torch.equal(only, gw)
    assert gpu_lib.moe_ffn_grouped_mm_bwd(ones, x.detach(), w.detach(), off, transposed=transposed,
                                          need_dx=False, need_dw=False) == (None, None)
    with pytest.raises(RuntimeError):  # no second derivative
        g, = torch.autograd.grad((gpu_lib.moe_ffn_grouped_mm(x, w, off, transposed=transposed) ** 2).sum(), x,
                                 create_graph=True)
        g.sum().backward()


def test_gradients_by_differences(gpu_lib):
    """fp32: the loss along a direction against the gradients' product with it."""
    say("[grouped] differences")
    x, w, dy, off = (t.cuda() for t in make(90, 40, 56, 3, "f32", False, spread(90, 3, tail=7)))
    gx, gw = gpu_lib.moe_ffn_grouped_mm_bwd(dy, x, w, off)
    gen = torch.Generator("cuda").manual_seed(1)
    loss = lambda x, w: float((gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off).double() * dy.double()).sum())
    for x_on in (True, False):
        d = torch.randn((x if x_on else w).shape, generator=gen, device="cuda")
        slope = float(((gx if x_on else gw).double() * d.double()).sum())
        # linear in each: a step of 1 has no error of its own; the sums' roundings are 1e-4 of it
        diff = (loss(x + d, w) - loss(x - d, w)) / 2 if x_on else (loss(x, w + d) - loss(x, w - d)) / 2
        assert abs(diff - slope) <= 1e-4 * (abs(slope) + float((dy.abs().sum())))


def test_the_layer_from_its_products(gpu_lib):
    """Routing, grouped products, SwiGLU and combine as a caller writes them give the layer and its
    gradients; ids out of range leave rows behind the last group."""
    say("[grouped] the layer from its products")
    T, H, I, E, K = 200, 256, 128, 6, 2
    rng = np.random.default_rng(3)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
    x, up, down = f(T, H).bfloat16(), (f(E, H, 2 * I) / 16).bfloat16(), (f(E, I, H) / 11).bfloat16()
    ids = torch.from_numpy(rng.integers(0, E, (T, K)).astype(np.int32)).cuda()
    ids[7, 1], ids[50] = -1, E
    gates = torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda()
    counts, offsets, sorted_slot, slot_pos, _ = gpu_lib.moe_ffn_route(ids, E)
    for t in (x, up, down):
        t.requires_grad_()

    live = int(offsets[-1])
    slots = torch.where(torch.arange(T * K, device="cuda") < live, sorted_slot, 0).long()
    h = gpu_lib.moe_ffn_grouped_mm(x[slots // K], up, offsets)
    act = (torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()).bfloat16()
    o = gpu_lib.moe_ffn_grouped_mm(act, down, offsets)
    pos = slot_pos.long()
    y = (torch.where(pos >= 0, gates.flatten(), 0.0).unsqueeze(1) * o[pos.clamp(min=0)].float()).view(T, K, H).sum(1)
    want, saved = gpu_lib.moe_ffn_fwd(x.detach(), ids, gates, up.detach(), down.detach(), save_for_backward=True)
    err = lambda a, b: float((a.detach().float() - b.float()).abs().max() / b.float().abs().max())
    # h is rounded to bf16 here and not in the layer; act, o and y in both: a few steps of 2^-8
    assert err(y, want) <= 2.0 ** -6
    dy = f(T, H).bfloat16()
    y.backward(dy.float())
    gx, gu, gd, _ = gpu_lib.moe_ffn_bwd(dy, x.detach(), ids, gates, up.detach(), down.detach(), saved)
    for a, b in ((x.grad, gx), (up.grad, gu), (down.grad, gd)):
        assert err(a, b) <= 2.0 ** -5
    assert not y[50].any() and not x.grad[50].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graph_replays(gpu_lib, dtype):
    """Captured forward and backward on fresh inputs and offsets, replayed between eager work."""
    say(f"[grouped] graph {dtype}")
    M, Kd, N, E = 260, 256, 512, 4
    x, w, dy, off = (t.cuda() for t in make(M, Kd, N, E, dtype, False, spread(M, E)))

    def step():
        y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off)
        return (y, *gpu_lib.moe_ffn_grouped_mm_bwd(dy, x, w, off))

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
        x2, w2, dy2, off2 = make(M, Kd, N, E, dtype, False, spread(M, E, seed=seed, tail=40 * seed), seed=seed)
        x.copy_(x2), w.copy_(w2), dy.copy_(dy2), off.copy_(off2)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("one,two", [((900, 512, 256, 5), (700, 264, 520, 9)), ((16000, 512, 512, 7), (57000, 128, 256, 1))],
                         ids=["short", "long"])
def test_two_streams(gpu_lib, one, two):
    """Two calls at once, each with its own workspace, give what they give alone."""
    say(f"[grouped] two streams {one} {two}")
    a = [t.cuda() for t in make(*one, "bf16", False, spread(one[0], one[3]))]
    b = [t.cuda() for t in make(*two, "bf16", True, spread(two[0], two[3]), seed=2)]
    run = lambda d, tr: (gpu_lib.moe_ffn_grouped_mm_fwd(d[0], d[1], d[3], transposed=tr),
                         *gpu_lib.moe_ffn_grouped_mm_bwd(d[2], d[0], d[1], d[3], transposed=tr))
    alone = run(a, False), run(b, True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            got_a = run(a, False)
        with torch.cuda.stream(s2):
            got_b = run(b, True)
        torch.cuda.synchronize()
        for want, got in zip(alone, (got_a, got_b)):
            assert all(torch.equal(p, q) for p, q in zip(want, got))


# few rows: 16- and 32-row tiles of every width, contractions that end inside a step or leave waves
# without one, more groups than a wave has lanes
@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 8, 24600, 1), (16, 40, 36872, 1), (5, 200, 25000, 2), (17, 8, 30008, 1), (40, 72, 9000, 3),
                                  (150, 104, 9608, 2), (33, 2056, 72, 1), (7, 4104, 16, 5), (64, 1096, 1544, 3),
                                  (8, 40, 48, 100), (30, 136, 264, 70), (100, 520, 8, 2),
                                  (1, 520, 512, 1), (64, 264, 1000, 1), (70, 1032, 520, 5), (600, 72, 136, 66)], ids=str)
def test_few_rows(gpu_lib, size, dtype, transposed):
    M, Kd, N, E = size
    say(f"[grouped] few rows {size} {dtype} transposed={transposed}")
    check(gpu_lib, make(M, Kd, N, E, dtype, transposed, spread(M, E, head=M // 5, tail=M // 7)), dtype, transposed)


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
def test_few_rows_of_a_matrix_of_4_gib(gpu_lib, transposed):
    M, Kd, N = 3, 65544, 32760
    say(f"[grouped] {M}x{Kd}x{N} transposed={transposed}")
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(M, Kd, generator=gen, device="cuda").bfloat16()
    w = torch.randn(*((1, N, Kd) if transposed else (1, Kd, N)), generator=gen, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, M], device="cuda")
    y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off, transposed=transposed)
    for c in (slice(0, 8), slice(N - 200, N)):
        wc = (w[0, c].double().t() if transposed else w[0, :, c].double()).contiguous()
        want, mag = x.double() @ wc, x.double().abs() @ wc.abs()
        sums = (Kd + 2) * 2.0 ** -23 * mag
        assert bool(((y[:, c].double() - want).abs() <= sums + HALF["bf16"] * (want.abs() + sums)).all())
        # far above what rounding gives, a step left out or taken twice is too
        assert float((y[:, c].double() - want).abs().max()) < 0.01 * Kd ** 0.5


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("Kd,N", [(32768, 32768), (32760, 32768)], ids=["past 4 GiB", "below"])
def test_few_rows_of_a_large_matrix_in_fp32(gpu_lib, Kd, N, transposed):
    M = 3
    say(f"[grouped] {M}x{Kd}x{N} fp32 transposed={transposed}")
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(M, Kd, generator=gen, device="cuda")
    w = torch.randn(*((1, N, Kd) if transposed else (1, Kd, N)), generator=gen, device="cuda")
    y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, torch.tensor([0, M], device="cuda"), transposed=transposed)
    for c in (slice(0, 8), slice(N - 200, N)):
        wc = (w[0, c].double().t() if transposed else w[0, :, c].double()).contiguous()
        want, mag = x.double() @ wc, x.double().abs() @ wc.abs()
        sums = (Kd + 2) * 2.0 ** -23 * mag
        assert bool(((y[:, c].double() - want).abs() <= sums + HALF["f32"] * (want.abs() + sums)).all())
        assert float((y[:, c].double() - want).abs().max()) < 1e-4 * Kd ** 0.5


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dtype,Kd,N,E", [("bf16", 40, 24, 3), ("f32", 200, 1000, 3)])
def test_few_rows_keep_infinities_apart(gpu_lib, dtype, Kd, N, E, transposed):
    """Values past K, N and a group's rows are not multiplied: what is infinite there stays there."""
    say(f"[grouped] infinities {dtype} transposed={transposed}")
    M = 5
    x, w, dy, off = (t.cuda() for t in make(M, Kd, N, E, dtype, transposed, (0, np.array([2, 0, 3]))))
    clean = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off, transposed=transposed)
    w2 = w.clone()
    w2[1] = float("inf")
    assert torch.equal(gpu_lib.moe_ffn_grouped_mm_fwd(x, w2, off, transposed=transposed), clean)
    wide = torch.full((M, Kd + 8), float("inf"), dtype=x.dtype, device="cuda")
    wide[:, :Kd] = x
    assert torch.equal(gpu_lib.moe_ffn_grouped_mm_fwd(wide[:, :Kd], w, off, transposed=transposed), clean)
    w3 = w.clone()
    (w3[0][3] if transposed else w3[0][:, 3]).fill_(float("inf"))
    y = gpu_lib.moe_ffn_grouped_mm_fwd(x.abs() + 1, w3, off, transposed=transposed)
    assert bool(torch.isinf(y[:2, 3]).all()) and bool(torch.isfinite(y[2:]).all())


# more tiles than the kernel for few rows takes: tiles of 64, 128 and 256 rows, whole or not in columns
# and contraction
HEIGHTS = [(150, 512, 512, 100), (150, 520, 552, 100), (2600, 512, 512, 20), (2600, 520, 552, 20), (5000, 512, 512, 8),
           (5000, 544, 552, 8), (57000, 128, 256, 1), (57000, 160, 264, 2), (30000, 128, 512, 3)]


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("size", HEIGHTS, ids=str)
def test_every_height(gpu_lib, size, transposed):
    M, Kd, N, E = size
    say(f"[grouped] height {size} transposed={transposed}")
    check(gpu_lib, make(M, Kd, N, E, "bf16", transposed, spread(M, E, head=M // 50, tail=M // 40)), "bf16", transposed)


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("M,Kd,N,E", [(150, 512, 512, 100), (2600, 512, 512, 20), (5000, 544, 552, 8), (57000, 160, 264, 1),
                                      (20, 256, 512, 2), (1500, 256, 512, 2), (1500, 288, 264, 1), (300, 256, 512, 2)])
def test_strided_rows_of_every_height(gpu_lib, M, Kd, N, E, transposed):
    say(f"[grouped] strided {M}x{Kd}x{N}/{E} transposed={transposed}")
    x, w, dy, off = (t.cuda() for t in make(M, Kd, N, E, "bf16", transposed, spread(M, E, tail=9)))
    wide = torch.full((M, Kd + 24), float("nan"), dtype=x.dtype, device="cuda")
    rows = wide[:, 8:8 + Kd]
    rows.copy_(x)
    want = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off, transposed=transposed)
    assert torch.equal(gpu_lib.moe_ffn_grouped_mm_fwd(rows, w, off, transposed=transposed), want)
    for p, q in zip(gpu_lib.moe_ffn_grouped_mm_bwd(dy, x, w, off, transposed=transposed),
                    gpu_lib.moe_ffn_grouped_mm_bwd(dy, rows, w, off, transposed=transposed)):
        assert torch.equal(p, q)


def test_graph_of_a_long_product(gpu_lib):
    """The routed rows decide the kernel at each replay."""
    say("[grouped] long graph")
    M, Kd, N, E = 16384, 2048, 2048, 8
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(M, Kd, generator=gen, device="cuda").bfloat16()
    w = torch.randn(E, Kd, N, generator=gen, device="cuda").bfloat16()
    even = torch.arange(0, M + 1, M // E, device="cuda")
    off = even.clone()
    gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off)
    skewed = torch.tensor([0, 40, 90, 150, 15000, 15200, 15700, 16000, 16384], device="cuda")
    for o in (even, skewed, skewed - 8, even):
        off.copy_(o)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, gpu_lib.moe_ffn_grouped_mm_fwd(x, w, o))
        for e in (0, 3, 7):
            a, b = int(o[e].clamp(0)), int(o[e + 1])
            want = x[a:b].double() @ w[e].double()
            mag = x[a:b].double().abs() @ w[e].double().abs()
            sums = (Kd + 2) * 2.0 ** -23 * mag
            assert bool(((out[a:b].double() - want).abs() <= sums + HALF["bf16"] * (want.abs() + sums)).all())


def test_tensors_that_are_refused(gpu_lib):
    say("[grouped] refusals")
    x, w, dy, off = (t.cuda() for t in make(16, 32, 48, 2, "bf16", False, (0, np.array([8, 8]))))
    E = gpu_lib.MoEFFNError
    for bad in (dict(x=x.float()), dict(x=x[:, :24]), dict(x=x.t()), dict(w=w[0]), dict(w=w.transpose(1, 2)),
                dict(off=off[:2]), dict(off=off.float()), dict(off=off.cpu()), dict(x=x.half(), w=w.half()),
                dict(x=torch.zeros(16, 37, dtype=x.dtype, device="cuda")[:, 5:]),
                dict(x=torch.zeros(16, 40, dtype=x.dtype, device="cuda")[:, 4:36]),
                dict(ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        a = {**dict(x=x, w=w, off=off, ws=None), **bad}
        with pytest.raises(E):
            gpu_lib.moe_ffn_grouped_mm_fwd(a["x"], a["w"], a["off"], ws=a["ws"])
    for bad in (dy[:, :40], dy.float(), dy[:8], dy.t().contiguous().t()):
        with pytest.raises(E):
            gpu_lib.moe_ffn_grouped_mm_bwd(bad, x, w, off)


# long products, for which the routed rows decide the kernel: rows split evenly and by Zipf's law,
# with empty groups and rows of no group
@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("routing", ["even", "zipf"])
@pytest.mark.parametrize("M,Kd,N,E", [(16384, 2048, 2048, 8), (20000, 1056, 3208, 24), (24576, 1408, 2048, 64)])
def test_long_products(gpu_lib, M, Kd, N, E, routing, transposed):
    say(f"[grouped] {M}x{Kd}x{N}/{E} {routing} transposed={transposed}")
    gen = torch.Generator("cuda").manual_seed(3)
    p = torch.ones(E, device="cuda")
    if routing == "zipf":
        rank = torch.randperm(E, generator=gen, device="cuda")
        p = (1.0 + rank) ** -1.2 * (rank < E - 2)
    counts = torch.bincount(torch.multinomial(p, M - 500, replacement=True, generator=gen), minlength=E)
    off = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)) + 123
    x = torch.randn(M, Kd, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(*((E, N, Kd) if transposed else (E, Kd, N)), generator=gen, device="cuda") / Kd ** 0.5).bfloat16()
    y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off, transposed=transposed)
    dx, dw = gpu_lib.moe_ffn_grouped_mm_bwd(y, x, w, off, transposed=transposed)

    def near(got, a, b, terms):
        want, mag = a @ b, a.abs() @ b.abs()
        sums = (terms + 2) * 2.0 ** -23 * mag
        return bool(((got.double() - want).abs() <= sums + HALF["bf16"] * (want.abs() + sums) + 1e-38).all())

    for e, (a, b) in enumerate(ref.groups(off.cpu().numpy(), M)):
        we = w[e].double().t().contiguous() if transposed else w[e].double()
        xe, ye = x[a:b].double(), y[a:b].double()
        assert near(y[a:b], xe, we, Kd), e
        assert near(dx[a:b], ye, we.t().contiguous(), N), e
        g = dw[e].t() if transposed else dw[e]
        assert near(g, xe.t().contiguous(), ye, b - a), e
    for t in (y, dx):
        assert not t[:123].any() and not t[M - 377:].any()


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
def test_past_32_bit_offsets(gpu_lib, transposed):
    """Outputs of more than 2^32 bytes: the last rows against the same rows alone."""
    M, Kd, N = (1 << 19) + 77, 128, 8192
    say(f"[grouped] {M}x{Kd}x{N} transposed={transposed}")
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(M, Kd, generator=gen, device="cuda").bfloat16()
    w = torch.randn(*((2, N, Kd) if transposed else (2, Kd, N)), generator=gen, device="cuda").bfloat16()
    off = torch.tensor([0, M - 300, M], dtype=torch.int32, device="cuda")
    y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off, transposed=transposed)
    last = gpu_lib.moe_ffn_grouped_mm_fwd(x[-300:].contiguous(), w,
                                          torch.tensor([0, 0, 300], dtype=torch.int32, device="cuda"),
                                          transposed=transposed)
    assert torch.equal(y[-300:], last)
    gx, gw = gpu_lib.moe_ffn_grouped_mm_bwd(y, x, w, off, transposed=transposed)
    lx, lw = gpu_lib.moe_ffn_grouped_mm_bwd(last, x[-300:].contiguous(), w,
                                            torch.tensor([0, 0, 300], dtype=torch.int32, device="cuda"),
                                            transposed=transposed)
    assert torch.equal(gw[1], lw[1])
    # 300 rows alone take another kernel, which sums in another order: both are near the formula
    we = (w[1] if transposed else w[1].t()).double()
    want, mag = last.double() @ we, last.double().abs() @ we.abs()
    sums = (N + 2) * 2.0 ** -23 * mag
    for got in (gx[-300:], lx):
        assert bool(((got.double() - want).abs() <= sums + HALF["bf16"] * (want.abs() + sums)).all())
