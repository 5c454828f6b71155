"""Offsets that are wrong, rows of no group, empty groups and values that are not finite, on the
kernels of 64-, 128- and 256-row tiles, which walk the tables that the set-up launch builds.

bf16 products come there with more than 160 tiles of 32 rows and 256 columns."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import products as ref
from test_gpu_grouped import HALF, check, make, spread

pytestmark = pytest.mark.gpu

# 64-, 128- and 256-row tiles, whole or not in columns and contraction
SIZES = [(150, 512, 512, 100), (150, 520, 552, 100), (2600, 512, 512, 20), (2600, 520, 552, 20), (5000, 512, 512, 8),
         (5000, 544, 552, 8), (57000, 160, 264, 2)]
both = pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])


def is_tall(M, Kd, N, E):
    tiles = (M + min(M, E) * 31) // 32
    return all(tiles * -(-n // 256) > 160 for n in (Kd, N))


def test_the_sizes_are_tall():
    assert all(is_tall(*s) for s in SIZES)


def wrong(M, E, kind):
    """Offsets that descend, lie before the first row or behind the last, or do all of it."""
    off = np.linspace(0, M, E + 1).astype(np.int64)
    if kind == "outside":
        off[0], off[-1] = -7, M + 1000
    elif kind == "descending":
        off = off[::-1].copy()
        off[0] = M // 2
    elif kind == "far":
        off[E // 2], off[-1] = -2 ** 40, 2 ** 40
    elif kind == "jumps":
        off[1::2] //= 3
        off[E // 2] += M // 4
    else:
        off[:] = M // 3
    return torch.from_numpy(off)


@both
@pytest.mark.parametrize("kind", ["outside", "descending", "far", "jumps", "equal"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_offsets_that_are_wrong(gpu_lib, size, kind, transposed):
    M, Kd, N, E = size
    say(f"[grouped] tall {size} offsets {kind} transposed={transposed}")
    x, w, dy, _ = make(M, Kd, N, E, "bf16", transposed, spread(M, E))
    check(gpu_lib, (x, w, dy, wrong(M, E, kind)), "bf16", transposed)


@both
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_rows_of_no_group_and_empty_groups_are_not_read(gpu_lib, size, transposed):
    M, Kd, N, E = size
    say(f"[grouped] tall {size} poisoned transposed={transposed}")
    head, tail = M // 50, M // 40
    empty = (1,) if E == 2 else (1, E - 1)
    x, w, dy, off = make(M, Kd, N, E, "bf16", transposed, spread(M, E, empty=empty, head=head, tail=tail))
    for t in (x, dy):
        t[:head], t[M - tail:] = float("nan"), float("inf")
    for i, e in enumerate(empty):
        w[e] = (float("nan"), float("inf"))[i]
    x, w, dy, off = x.cuda(), w.cuda(), dy.cuda(), off.cuda()
    y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off, transposed=transposed)
    gx, gw = gpu_lib.moe_ffn_grouped_mm_bwd(dy, x, w, off, transposed=transposed)
    for t in (y, gx):
        assert bool(torch.isfinite(t).all()) and not t[:head].any() and not t[M - tail:].any()
        assert bool((t[head:M - tail] != 0).any(1).all())
    assert bool(torch.isfinite(gw).all()) and not any(gw[e].any() for e in empty) and gw[0].any()


@both
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_nan_and_inf_stay_where_they_are(gpu_lib, size, transposed):
    """Of a token's row in its row and its group's weight gradient, of a weight in its group's rows."""
    M, Kd, N, E = size
    say(f"[grouped] tall {size} non-finite transposed={transposed}")
    x, w, dy, off = (t.cuda() for t in make(M, Kd, N, E, "bf16", transposed, spread(M, E)))
    run = lambda x, w, dy: (gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off, transposed=transposed),
                            *gpu_lib.moe_ffn_grouped_mm_bwd(dy, x, w, off, transposed=transposed))
    y, gx, gw = run(x, w, dy)
    group = torch.bucketize(torch.arange(M, device="cuda"), off, right=True) - 1
    rows = torch.tensor([5, M - 3], device="cuda")
    x2, dy2 = x.clone(), dy.clone()
    x2[5, 3], x2[M - 3, Kd - 1] = float("nan"), float("inf")
    dy2[5, N - 1], dy2[M - 3, 0] = -float("inf"), float("nan")
    y2, gx2, gw2 = run(x2, w, dy2)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[rows] = False
    for a, b in ((y, y2), (gx, gx2)):
        assert torch.equal(a[keep], b[keep])
    assert bool(torch.isnan(y2[5]).all()) and not torch.isfinite(y2[M - 3]).any()
    assert not torch.isfinite(gx2[5]).any() and bool(torch.isnan(gx2[M - 3]).all())
    others = [e for e in range(E) if e not in group[rows].tolist()]
    assert torch.equal(gw[others], gw2[others]) and not torch.isfinite(gw2[group[5]]).all()
    e = int(group[M - 3])
    w3 = w.clone()
    w3[e] = float("nan")
    y3, gx3, _ = run(x, w3, dy)
    for a, b in ((y, y3), (gx, gx3)):
        assert torch.equal(a[group != e], b[group != e]) and bool(torch.isnan(b[group == e]).all())


@both
@pytest.mark.parametrize("size", [SIZES[1], SIZES[2], SIZES[5]], ids=str)
def test_graph_replays(gpu_lib, size, transposed):
    """Captured forward and backward on fresh inputs and offsets, wrong ones too, between eager work."""
    M, Kd, N, E = size
    say(f"[grouped] tall {size} graph transposed={transposed}")
    x, w, dy, off = (t.cuda() for t in make(M, Kd, N, E, "bf16", transposed, spread(M, E), offsets_dtype=torch.int64))

    def step():
        y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off, transposed=transposed)
        return (y, *gpu_lib.moe_ffn_grouped_mm_bwd(dy, x, w, off, transposed=transposed))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed, kind in enumerate(("descending", None, "far", None, "outside")):
        x2, w2, dy2, off2 = make(M, Kd, N, E, "bf16", transposed, spread(M, E, seed=seed, tail=9 * seed), seed=seed)
        x.copy_(x2), w.copy_(w2), dy.copy_(dy2), off.copy_(off2 if kind is None else wrong(M, E, kind))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


@both
@pytest.mark.parametrize("kind", ["outside", "descending", "far", "jumps"])
def test_a_long_product_with_wrong_offsets(gpu_lib, kind, transposed):
    """Both tile tables are built, and the routed rows decide which is walked."""
    M, Kd, N, E = 16384, 2048, 2048, 8
    say(f"[grouped] long, offsets {kind} transposed={transposed}")
    gen = torch.Generator("cuda").manual_seed(9)
    x = torch.randn(M, Kd, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(E, Kd, N, generator=gen, device="cuda") / Kd ** 0.5).bfloat16()
    off = wrong(M, E, kind)
    ranges = ref.groups(off.numpy(), M)
    x[:ranges[0][0]], x[ranges[-1][1]:] = float("nan"), float("inf")
    for e, (a, b) in enumerate(ranges):
        if a == b:
            w[e] = float("nan")
    y = gpu_lib.moe_ffn_grouped_mm_fwd(x, w, off.cuda(), transposed=transposed)
    dx, dw = gpu_lib.moe_ffn_grouped_mm_bwd(y, x, w, off.cuda(), transposed=transposed)

    def near(got, a, b, terms):
        want, mag = a @ b, a.abs() @ b.abs()
        sums = (terms + 2) * 2.0 ** -23 * mag
        return bool(((got.double() - want).abs() <= sums + HALF["bf16"] * (want.abs() + sums) + 1e-38).all())

    for e, (a, b) in enumerate(ranges):
        if a == b:
            assert not dw[e].any()
            continue
        we = w[e].double().t().contiguous() if transposed else w[e].double()
        xe, ye = x[a:b].double(), y[a:b].double()
        assert near(y[a:b], xe, we, Kd), e
        assert near(dx[a:b], ye, we.t().contiguous(), N), e
        assert near(dw[e].t() if transposed else dw[e], xe.t().contiguous(), ye, b - a), e
    for t in (y, dx):
        assert not t[:ranges[0][0]].any() and not t[ranges[-1][1]:].any()
