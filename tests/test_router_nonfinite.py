"""The router on rows with NaN, infinities and switched-off experts, against values worked out by
hand: which experts are chosen must not depend on what else stands in the row."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as ops

INF, NAN = float("inf"), float("nan")


def oracle(logits, K, **kw):
    bias = kw.pop("bias", None)
    with np.errstate(all="ignore"):
        return ops.router(np.array(logits, np.float32), K,
                          bias=None if bias is None else np.array(bias, np.float32), **kw)


def on_gpu(m, logits, K, bias=None, pad=0, **kw):
    """The kernels' answer, with ``pad`` closed experts behind the row's own: above 256 experts
    one wave takes a row, up to there sixteen lanes."""
    l = torch.tensor(logits, dtype=torch.float32)
    l = torch.nn.functional.pad(l, (0, pad), value=-INF).cuda()
    b = None
    if bias is not None:
        b = torch.nn.functional.pad(torch.tensor(bias, dtype=torch.float32), (0, pad)).cuda()
    w, ids = m.moe_ffn_router_fwd(l, K, bias=b, **kw)
    torch.cuda.synchronize()
    return w.cpu().numpy(), ids.cpu().numpy()


# (score, logits, bias, ids of K = 3, which of the three gates are NaN)
CLOSED = [
    # one NaN makes every softmax score NaN: the open experts in their order, the closed one never
    ("softmax", [NAN, 1, 2, 3], [0, -INF, 0, 0], [0, 2, 3], [1, 1, 1]),
    ("softmax", [0, INF, 1, 2], [-INF, 0, 0, 0], [1, 2, 3], [1, 1, 1]),
    ("softmax", [NAN, 1, 2, 3], [-INF, -INF, -INF, 0], [3, -1, -1], [1, 0, 0]),
    # sigmoid: NaN at 0 is closed, NaN at 2 is open and below every number
    ("sigmoid", [NAN, 1, NAN, 3], [-INF, 0, 0, 0], [3, 1, 2], [0, 0, 1]),
    ("sigmoid", [1, NAN, NAN, 3], [0, -INF, -INF, 0], [3, 0, -1], [0, 0, 0]),
    ("sigmoid", [INF, NAN, 0, -INF], [-INF, 0, 0, 0], [2, 1, -1], [0, 1, 0]),
]


def expect_closed(answer):
    for score, l, bias, ids, nan in CLOSED:
        say("[router] closed by the bias", score, l, bias)
        w, got = answer([l], 3, bias=bias, score=score, renormalize=False)
        assert got.tolist() == [ids], (score, l, bias)
        assert np.isnan(w).tolist() == [[bool(n) for n in nan]], (score, l, bias)
        assert (w[got < 0] == 0).all()


def test_oracle_closed_by_the_bias():
    expect_closed(oracle)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 12, 252, 253, 600])
def test_closed_by_the_bias(gpu_lib, pad):
    expect_closed(lambda l, K, **kw: on_gpu(gpu_lib, l, K, pad=pad, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 1), (64, 8), (256, 8), (160, 8), (512, 1), (512, 16)])
def test_random_rows_with_every_kind_of_value(gpu_lib, E, groups, score):
    """NaN, +inf and -inf strewn over logits and -inf over the bias: ids as the oracle's, and an
    expert whose bias is -inf in no slot."""
    say("[router] strewn", E, groups, score)
    rng = np.random.default_rng([E, groups])
    T, K = 300, 6
    l = rng.standard_normal((T, E)).astype(np.float32)
    for value in (NAN, INF, -INF):
        l[rng.random((T, E)) < 0.3 * rng.random((T, 1)) ** 3] = value
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32)
    bias[rng.random(E) < 0.3] = -INF
    kw = dict(score=score, groups=groups, topk_groups=max(1, groups // 2))
    w, ids = on_gpu(gpu_lib, l, K, bias=bias, **kw)
    rw, rid = oracle(l, K, bias=bias, **kw)
    np.testing.assert_array_equal(ids, rid)
    assert not np.isin(np.nonzero(bias == -INF)[0], ids).any()
    np.testing.assert_array_equal(np.isnan(w), np.isnan(rw))


# (score, logits, bias, groups, ids of K = 2 from the best group by the sum of two)
GROUPS = [
    # every score is NaN: the group that holds open experts, not the closed one before it
    ("softmax", [-INF, -INF, NAN, 1], None, 2, [3, 2]),
    ("softmax", [-INF, -INF, NAN, 1], [0, 0, 0, 0], 2, [2, 3]),
    ("softmax", [-INF, 5, INF, 1], None, 2, [2, 3]),
    # two NaNs are above closed experts, below a NaN and a number, and that below two numbers
    ("sigmoid", [-INF, -INF, NAN, NAN, -INF, -INF], [0] * 6, 3, [2, 3]),
    ("sigmoid", [NAN, NAN, NAN, -9, -INF, -INF], [0] * 6, 3, [3, 2]),
    ("sigmoid", [NAN, 99, -9, -9, NAN, NAN], [0] * 6, 3, [2, 3]),
    # ... however low those are
    ("sigmoid", [NAN, 1, 0, 0], [0, 0, -3e38, -3e38], 2, [2, 3]),
    # +inf beside a closed expert is no sum of two; beside a number it is the largest
    ("sigmoid", [1, -INF, 3, 4], [INF, 0, 0, 0], 2, [3, 2]),
    ("sigmoid", [3, 4, 1, -INF], [0, 0, INF, 0], 2, [1, 0]),
    ("sigmoid", [3, 4, 1, 0], [0, 0, INF, 0], 2, [2, 3]),
    ("sigmoid", [3, 4, 1, NAN], [0, 0, INF, 0], 2, [2, 3]),
    # one open expert: the lowest value, so that the lower of two such groups is kept
    ("sigmoid", [-INF, -INF, 9, -INF], None, 2, [-1, -1]),
    ("sigmoid", [9, -INF, -INF, -INF], None, 2, [0, -1]),
]


def expect_groups(answer, spread=1):
    """``spread`` closed experts follow each of a group's, which changes no sum and scales the ids."""
    for score, l, bias, groups, ids in GROUPS:
        say("[router] groups", score, l, bias)
        wide = lambda v, fill: [x for y in v for x in [y] + [fill] * (spread - 1)]
        w, got = answer([wide(l, -INF)], 2, bias=None if bias is None else wide(bias, 0),
                        score=score, groups=groups, topk_groups=1, group_top=2)
        assert got.tolist() == [[i * spread if i > 0 else i for i in ids]], (score, l, bias)
        if score == "softmax":
            assert np.isnan(w).all()


def test_oracle_groups():
    expect_groups(oracle)
    expect_groups(oracle, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1, 4, 16, 100])
def test_groups(gpu_lib, spread):
    """4 and 16: whole lanes of the sixteen, for the cases of two groups."""
    expect_groups(lambda l, K, **kw: on_gpu(gpu_lib, l, K, **kw), spread)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [True, False], ids=["bias", "plain"])
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (160, 8), (512, 16)])
def test_groups_of_random_rows(gpu_lib, E, groups, with_bias, score):
    say("[router] groups of strewn rows", E, groups, with_bias, score)
    rng = np.random.default_rng([E, groups, 2])
    T, K = 300, 6
    l = rng.standard_normal((T, E)).astype(np.float32)
    for value in (NAN, INF, -INF, -INF):
        l[rng.random((T, E)) < 0.9 * rng.random((T, 1)) ** 3] = value
    bias = None
    if with_bias:
        bias = (0.2 * rng.standard_normal(E)).astype(np.float32)
        bias[rng.random(E) < 0.3] = -INF
        bias[rng.random(E) < 0.02] = INF
    kw = dict(score=score, groups=groups, topk_groups=groups // 4, group_top=2)
    w, ids = on_gpu(gpu_lib, l, K, bias=bias, **kw)
    rw, rid = oracle(l, K, bias=bias, **kw)
    np.testing.assert_array_equal(ids, rid)
    np.testing.assert_array_equal(np.isnan(w), np.isnan(rw))


# plain softmax, K = 2: (logits, ids, d_topk_weights, which gradients are NaN); the others are 0
GRADIENTS = [
    # +inf: the other exponentials underflow to 0, and still depend on it
    ([INF, 0, 1, -INF], [0, 2], [1, 2], [1, 1, 1, 0]),
    ([5, INF, -INF, -200], [0, 3], [1, 2], [1, 1, 0, 1]),
    ([NAN, 0, -300, -INF], [1, 2], [1, 2], [1, 1, 1, 0]),
    # one NaN gate's gradient reaches an expert whose score is 0
    ([0, -400, -INF, 1], [0, 3], [NAN, 2], [1, 1, 0, 1]),
    # no slot: no gradient
    ([INF, NAN, 1, -INF], [-1, -1], [1, 2], [0, 0, 0, 0]),
    ([-INF] * 4, [0, -1], [1, 2], [0, 0, 0, 0]),
]


def expect_gradients(grad):
    for l, ids, dw, nan in GRADIENTS:
        say("[router] gradient", l, ids)
        d = grad(np.array([dw], np.float32), np.array([l], np.float32), np.array([ids]))
        assert np.isnan(d).tolist() == [[bool(n) for n in nan]], (l, ids, d)
        assert (d[~np.isnan(d)] == 0).all()


def test_oracle_gradients():
    def grad(dw, l, ids):
        with np.errstate(all="ignore"):
            return ops.router_grad(dw, l, ids, renormalize=False)[0]
    expect_gradients(grad)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 13, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_gradients(gpu_lib, dtype, pad):
    def grad(dw, l, ids):
        l = np.pad(l, ((0, 0), (0, pad)), constant_values=-INF)
        d = gpu_lib.moe_ffn_router_bwd(torch.from_numpy(dw).cuda(),
                                       torch.from_numpy(l).to(dtype).cuda(),
                                       torch.from_numpy(ids).cuda(), renormalize=False)
        d = d.float().cpu().numpy()
        assert (d[:, l.shape[1] - pad:] == 0).all()
        return d[:, :l.shape[1] - pad]
    expect_gradients(grad)
