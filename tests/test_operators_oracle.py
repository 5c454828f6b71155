"""Pins of the numpy reference of the router and the MXFP4 expert FFN: hand-worked cases, the
definitions by brute force, and the router's gradient against differences."""

import numpy as np
import pytest

from oracle import operators as ops


def test_router_by_hand():
    l = np.log([[1.0, 4.0, 2.0, 1.0]])
    w, ids = ops.router(l, 2)
    assert ids.tolist() == [[1, 2]]
    np.testing.assert_allclose(w, [[2 / 3, 1 / 3]])
    w, ids = ops.router(l, 3, renormalize=False, scale=2.0)
    assert ids.tolist() == [[1, 2, 0]]  # 0 and 3 tie: the lower id
    np.testing.assert_allclose(w, [[1.0, 0.5, 0.25]])
    # a bias moves the selection, not the gates
    w, ids = ops.router(l, 2, bias=[0.0, 0.0, 0.0, 1.0], renormalize=False)
    assert ids.tolist() == [[3, 1]]
    np.testing.assert_allclose(w, [[0.125, 0.5]])


def test_router_groups_by_hand():
    l = np.array([[3.0, -3.0, 2.0, 2.0, 1.9, 1.9]])
    kw = dict(score="sigmoid", groups=3, topk_groups=1)
    assert ops.router(l, 1, group_top=1, **kw)[1].tolist() == [[0]]
    # the sum of two: groups 1 and 2 pass group 0
    assert ops.router(l, 2, group_top=2, **kw)[1].tolist() == [[2, 3]]


def test_router_closed_experts():
    inf = np.inf
    l = np.array([[-inf, 1.0, -inf, 0.0], [-inf] * 4, [np.nan, 1.0, -inf, -inf]])
    w, ids = ops.router(l, 3)
    assert ids.tolist() == [[1, 3, -1], [-1] * 3, [1, 0, -1]]
    assert w[0, 2] == 0 and w[1].tolist() == [0, 0, 0]
    np.testing.assert_allclose(w[0, :2].sum(), 1.0)
    assert np.isnan(w[2, :2]).all() and w[2, 2] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_router_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((3, 9))
    l[1, 4] = -np.inf
    dw = rng.standard_normal((3, 4))
    kw = dict(score=score, renormalize=renormalize, scale=1.7)
    _, ids = ops.router(l, 4, **kw)
    d, mag = ops.router_grad(dw, l, ids, **kw)
    h = 1e-6
    for t in range(3):
        for j in range(9):
            if l[t, j] == -np.inf:
                assert d[t, j] == 0
                continue
            up, dn = l.copy(), l.copy()
            up[t, j] += h
            dn[t, j] -= h
            wu, iu = ops.router(up, 4, **kw)
            wd, idn = ops.router(dn, 4, **kw)
            assert (iu == ids).all() and (idn == ids).all()
            np.testing.assert_allclose(d[t, j], ((wu - wd) * dw).sum() / (2 * h), atol=1e-8)
    assert (np.abs(d) <= mag + 1e-15).all()


def test_formats():
    assert len(ops._E2M3) == 32 and ops._E2M3[-1] == 7.5 and ops._E2M3[1] == 0.125
    # ties to even: .25 -> 0, .75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    v = np.zeros(32)
    v[:9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -6, 4]
    assert ops.mx_quantize(v)[:9].tolist() == [0, 1, 1, 2, 2, 4, 4, -6, 4]
    # the block's maximum 7 saturates at 6; 8 starts the next octave
    v[0] = 7.0
    assert ops.mx_quantize(v)[0] == 6
    v[0] = 8.0
    assert ops.mx_quantize(v)[:4].tolist() == [8, 1, 1, 2]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp6"])
def test_quantisation_is_nearest_idempotent_and_scales(fmt):
    rng = np.random.default_rng(5)
    v = rng.standard_normal((20, 75)) * np.exp(2 * rng.standard_normal((20, 1)))
    q = ops.mx_quantize(v, fmt)
    assert (ops.mx_quantize(q, fmt) == q).all()
    assert (ops.mx_quantize(v * 2.0 ** 9, fmt) == q * 2.0 ** 9).all()
    grid, top = ops._FORMATS[fmt]
    for r in range(20):
        for b in range(0, 75, 32):
            blk = v[r, b:b + 32]
            unit = 2.0 ** (np.floor(np.log2(np.abs(blk).max())) - top)
            near = np.abs(np.abs(blk)[:, None] / unit - grid).min(1)
            np.testing.assert_allclose(np.abs(np.abs(q[r, b:b + 32]) - np.abs(blk)) / unit, near,
                                       atol=1e-12)


def test_special_blocks():
    v = np.ones((4, 64))
    v[0, 3] = np.nan
    v[1, 40] = np.inf
    v[2] = 0
    v[3] *= 2.0 ** -140
    q = ops.mx_quantize(v)
    assert np.isnan(q[0, :32]).all() and (q[0, 32:] == 1).all()
    assert (q[1, :32] == 1).all() and np.isnan(q[1, 32:]).all()
    assert (q[2:] == 0).all()


def test_slack_covers_every_neighbour():
    rng = np.random.default_rng(6)
    v = rng.standard_normal((40, 64))
    s = np.abs(rng.standard_normal((40, 64))) * 0.02
    for fmt in ("mxfp4", "mxfp6"):
        q, off = ops.mx_quantize(v, fmt, slack=s)
        for _ in range(50):
            other = ops.mx_quantize(v + s * rng.uniform(-1, 1, s.shape), fmt)
            assert (np.abs(other - q) <= off + 1e-12).all()


def test_ffn_equals_dense_on_grid_values():
    """K = 1, gate 1 and weights already on the grid: a dense FFN with quantised activations."""
    rng = np.random.default_rng(7)
    x = rng.standard_normal((5, 40))
    up = ops.mx_quantize_columns(rng.standard_normal((1, 40, 48)))
    down = ops.mx_quantize_columns(rng.standard_normal((1, 24, 40)))
    y, tol = ops.mxfp4_ffn(x, np.zeros((5, 1), int), np.ones((5, 1)), up, down)
    h = ops.mx_quantize(x) @ up[0]
    a = h[:, :24] / (1 + np.exp(-h[:, :24])) * h[:, 24:]
    np.testing.assert_allclose(y, ops.mx_quantize(a) @ down[0], rtol=1e-12)
    assert (tol > 0).all() and (tol < 0.5 * np.abs(y).max()).all()
    # an id outside the experts contributes nothing
    y2, _ = ops.mxfp4_ffn(x, np.full((5, 1), -1), np.ones((5, 1)), up, down)
    assert (y2 == 0).all()
