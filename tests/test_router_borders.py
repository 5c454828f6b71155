"""The router's selection where fp32 keys do not order the experts: keys of the type's largest and
lowest value, sums next to each other, and biases that switch experts off by a finite value."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as ops

pytestmark = pytest.mark.gpu

BIG = float(np.finfo(np.float32).max)
INF = float("inf")


def check(m, l, K, bias, **kw):
    l, bias = np.asarray(l, np.float32), np.asarray(bias, np.float32)
    say("[router] borders", l.shape, K, kw)
    w, ids = m.moe_ffn_router_fwd(torch.from_numpy(l).cuda(), K, bias=torch.from_numpy(bias).cuda(),
                                  **kw)
    torch.cuda.synchronize()
    rw, rid = ops.router(l, K, bias=bias, **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    return ids.cpu().numpy()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 256, 192, 512])
def test_groups_of_the_lowest_and_largest_bias(gpu_lib, E, score):
    """Four groups, two kept.  Closed: 0.  All at the lowest value: 1, whose sum of two lies below
    every fp32 number and still above the closed group's.  Numbers: 2.  Closed: 3."""
    rng = np.random.default_rng(E)
    n = E // 4
    l = rng.standard_normal((40, E))
    l[:, :n] = -INF
    l[:, 3 * n:] = -INF
    bias = np.zeros(E)
    bias[n:2 * n] = -BIG
    kw = dict(score=score, groups=4, topk_groups=2, group_top=2)
    ids = check(gpu_lib, l, 6, bias, **kw)
    assert (ids >= 2 * n).all()  # numbers first
    ids = check(gpu_lib, l[:, :2 * n], 6, bias[:2 * n], score=score, groups=2, topk_groups=1,
                group_top=2)
    assert (ids == np.arange(n, n + 6)).all()  # equal keys: the lower ids
    # sums past the largest number: 1.5 and 2 times it
    bias = np.full(E, 0.25)
    bias[[1, n + 1, n + 2]] = BIG
    bias[2] = BIG / 2
    ids = check(gpu_lib, rng.standard_normal((40, E)), 2, bias, score=score, groups=4,
                topk_groups=1, group_top=2)
    assert (ids == [n + 1, n + 2]).all()


def group_sums_in_the_wrong_order(rows, E, seed):
    """Logits [rows, E] and a bias in two groups, the sum of the first group's two keys the larger
    by less than 2^-24, that fp32 arithmetic may put 2^-17 the other way round.

    Keys lie in [16, 18), where fp32's step is G = 2^-19.  A score of the first group lies just
    above (n + 1/2) G: a key of even last place goes down by G / 2 from the halfway point, one of
    odd last place if its score came out a step low.  One of the second group lies just below, and
    goes up likewise.  The sums, in [32, 36) with a step of 2 G, are then odd multiples of G,
    halfway again: the first goes down where it is 1 modulo 4, and the second up.
    """
    rng = np.random.default_rng(seed)
    G, n = 2.0 ** -19, E // 2
    bias = np.zeros(E)
    bias[[0, 1, n, n + 1]] = [17.25, 16.25, 17.0, 16.5]
    sign = np.array([1, 1, -1, -1])
    m = 40 * rows
    a = rng.integers(int(0.29 / G), int(0.36 / G), (m, 2))
    shift = rng.integers(-4000, 4000, m)
    mid = (np.stack([a[:, 0], a[:, 1], a[:, 0] + shift, a[:, 1] - shift], 1) + 0.5) * G
    s = mid + sign * 0.05 * 2.0 ** -24
    four = np.log(s / (1 - s)).astype(np.float32)
    # the fp32 logits' own scores: within 2^-27 of the halfway points, on the right side
    off = sign * (1 / (1 + np.exp(-four.astype(np.float64))) - mid)
    good = ((off > 0) & (off < 2.0 ** -27)).all(1)
    good &= (a.sum(1) + round((bias[0] + bias[1]) / G)) % 4 == 1
    four = four[good]
    l = rng.normal(-3, 0.5, (len(four), E)).astype(np.float32)
    l[:, [0, 1, n, n + 1]] = four
    return l, bias


@pytest.mark.parametrize("E", [16, 18, 64, 512])
def test_group_sums_next_to_each_other(gpu_lib, E):
    """E = 16 and 64: sixteen lanes a row; the others: a wave."""
    l, bias = group_sums_in_the_wrong_order(50000, E, seed=E)
    ids = check(gpu_lib, l, 2, bias, score="sigmoid", groups=2, topk_groups=1, group_top=2)
    assert (ids == [0, 1]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [16.0, 63.9, 300.0, 1e5])
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (160, 8), (512, 16)])
def test_sums_of_large_biases(gpu_lib, E, groups, size, score):
    """Biases far above the scores and a few fp32 steps apart: keys and group sums lie on a coarse
    grid, and the scores decide."""
    rng = np.random.default_rng([E, int(size)])
    step = float(np.spacing(np.float32(size)))
    bias = size + step * rng.integers(-2, 3, E)
    l = rng.standard_normal((200, E))
    for group_top in (1, 2):
        check(gpu_lib, l, 6, bias, score=score, groups=groups, topk_groups=groups // 2,
              group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("off", [-3.0, -1e4, -1e9, -BIG], ids=str)
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (160, 8), (512, 16)])
def test_experts_switched_off_by_a_finite_bias(gpu_lib, E, groups, off, score):
    rng = np.random.default_rng([E, groups])
    l = rng.standard_normal((200, E))
    some = 0.1 * rng.standard_normal(E)
    some[rng.random(E) < 0.2] = off
    whole = some.copy()  # whole groups, and all but one expert of another
    whole[:E // 4] = off
    whole[E // 2:E // 2 + E // groups - 1] = off
    for bias in (some, whole):
        for group_top in (1, 2):
            check(gpu_lib, l, 6, bias, score=score, groups=groups, topk_groups=groups // 2,
                  group_top=group_top)
        check(gpu_lib, l, 6, bias, score=score)
    # fewer experts left than slots: the switched-off ones follow, by their scores where the sum
    # still shows them, else by their ids
    bias = np.full(E, off)
    bias[[3, E - 1]] = 0
    ids = check(gpu_lib, l, 6, bias, score=score)
    assert (np.sort(ids[:, :2], axis=1) == [3, E - 1]).all()


@pytest.mark.parametrize("E", [256, 320])
def test_a_finite_mask_costs_no_more_than_a_closed_expert(gpu_lib, E):
    """A mask of -1e9 or the type's lowest value against one of -inf: about the same time, where
    rows selected again in 64 bits would take several times as long."""
    say("[router] time with masked experts", E)
    l = torch.randn(32768, E, device="cuda")
    times = {}
    biases = {}
    for off in (-INF, -1e9, -BIG):
        biases[off] = 0.1 * torch.randn(E, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        biases[off][::9] = off
    for _ in range(7):
        for off, bias in biases.items():
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            start.record()
            for _ in range(10):
                gpu_lib.moe_ffn_router_fwd(l, 8, bias=bias, score="sigmoid", groups=8, topk_groups=4,
                                           group_top=2)
            end.record()
            end.synchronize()
            times[off] = min(times.get(off, INF), start.elapsed_time(end) * 100)
    say("us:", times)
    assert max(times.values()) < 1.5 * times[-INF]
