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
