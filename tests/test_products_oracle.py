"""The 64-bit reference of the grouped and int8 products against other ways to the same numbers."""

import numpy as np
import pytest
import torch

from oracle import products as ref


@pytest.mark.parametrize("offsets,want", [
    ([0, 2, 5, 9], [(0, 2), (2, 5), (5, 9)]), ([3, 3, 4, 4], [(3, 3), (3, 4), (4, 4)]),
    ([-5, 20, 3, 9], [(0, 9), (9, 9), (9, 9)]), ([0, 6, 2, 8], [(0, 6), (6, 6), (6, 8)])])
def test_groups(offsets, want):
    assert ref.groups(offsets, 9) == want


@pytest.mark.parametrize("transposed", [False, True])
def test_grouped_against_autograd_and_differences(transposed):
    rng = np.random.default_rng(1)
    off = [1, 4, 4, 9]
    x, w, dy = rng.standard_normal((11, 8)), rng.standard_normal((3, 8, 16)), rng.standard_normal((11, 16))
    if transposed:
        w = w.transpose(0, 2, 1).copy()
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    rows = []
    for m in range(11):
        e = next((e for e in range(3) if off[e] <= m < off[e + 1]), None)
        we = None if e is None else (tw[e].T if transposed else tw[e])
        rows.append(torch.zeros(16, dtype=torch.float64) if e is None else tx[m] @ we)
    y = torch.stack(rows)
    (y * torch.tensor(dy)).sum().backward()
    got, _ = ref.grouped_mm(x, w, off, transposed)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-13, atol=1e-13)
    (dx, _), (dw, _) = ref.grouped_mm_grad(dy, x, w, off, transposed)
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-12, atol=1e-12)
    loss = lambda x, w: (ref.grouped_mm(x, w, off, transposed)[0] * dy).sum()
    for at in ((2, 3), (8, 0), (10, 1), (0, 0)):  # rows 0, 9 and 10 lie in no group
        d = np.zeros_like(x)
        d[at] = 1e-5
        assert abs((loss(x + d, w) - loss(x - d, w)) / 2e-5 - dx[at]) < 1e-6
    for at in ((0, 1, 2), (1, 5, 5), (2, 7, 7)):
        d = np.zeros_like(w)
        d[at] = 1e-5
        assert abs((loss(x, w + d) - loss(x, w - d)) / 2e-5 - dw[at]) < 1e-6


def test_int8_codes_by_search():
    rng = np.random.default_rng(2)
    v = (rng.standard_normal((40, 24)) * np.exp(2 * rng.standard_normal((40, 1)))).astype(np.float32)
    v[3] = 0
    v[4] = np.tile([127, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 125.5], 3)  # scale 1: ties to even
    q, s = ref.int8_codes(v, 1)
    for r in range(40):
        assert s[r] == np.float32(np.abs(v[r]).max().astype(np.float64) / 127)
        for c in range(24):
            cand = np.arange(-127, 128)
            d = np.abs(v[r, c] / s[r] - cand) if s[r] else np.abs(cand)
            best = cand[d == d.min()]
            assert q[r, c] in best and (len(best) == 1 or q[r, c] % 2 == 0)
    assert list(q[4, :8]) == [127, 0, 2, 2, 0, -2, -126, 126]


def test_int8_codes_not_finite():
    v = np.ones((4, 8))
    v[1, 3], v[2, 0] = np.nan, -np.inf
    q, s = ref.int8_codes(v, 1)
    assert (q[[0, 3]] == 127).all() and (q[1:3] == 0).all()
    assert np.isnan(s[1:3]).all() and np.isfinite(s[[0, 3]]).all()


def test_int8_slack_covers_perturbed_values():
    rng = np.random.default_rng(3)
    v = rng.standard_normal((50, 64))
    slack = 1e-3 * np.abs(v)
    q, s, off = ref.int8_codes(v, 1, slack=slack)
    for _ in range(20):
        p = v + slack * rng.uniform(-1, 1, v.shape)
        q2, s2 = ref.int8_codes(p, 1)
        assert (np.abs(q2 * s2[:, None] - q * s[:, None]) <= off + 1e-12).all()


def test_int8_ffn_against_the_layer():
    """The layer's formula on the values that codes and scales stand for, slot by slot."""
    rng = np.random.default_rng(4)
    T, H, I, E, K = 9, 24, 16, 4, 2
    x, up, down = rng.standard_normal((T, H)), rng.standard_normal((E, H, 2 * I)), rng.standard_normal((E, I, H))
    ids, gates = rng.integers(0, E, (T, K)), rng.random((T, K))

    def deq(v, axis):
        q, s = ref.int8_codes(v, axis)
        return q * np.expand_dims(s, axis)

    want = np.zeros((T, H))
    for t in range(T):
        for k in range(K):
            h = deq(x[t], 0) @ deq(up[ids[t, k]], 0)
            act = h[:I] / (1 + np.exp(-h[:I])) * h[I:]
            want[t] += gates[t, k] * (deq(act, 0) @ deq(down[ids[t, k]], 0))
    y, tol = ref.int8_ffn(x, ids, gates, up, down)
    np.testing.assert_allclose(y, want, rtol=1e-12, atol=1e-12)
    assert (tol > 0).all() and np.sqrt((tol ** 2).mean()) < 0.05 * np.sqrt((y ** 2).mean())


def test_int8_mm_rows_and_columns_that_are_nan():
    rng = np.random.default_rng(5)
    c, w = rng.integers(-127, 128, (5, 8)), rng.integers(-127, 128, (2, 8, 8))
    sx, sw = rng.random(5), rng.random((2, 8))
    sx[1], sw[1, 3] = np.nan, np.nan
    y = ref.int8_mm(c, sx, w, sw, [0, 2, 4])
    assert np.isnan(y[1]).all() and np.isnan(y[2:4, 3]).all()
    assert np.isfinite(y[0]).all() and (y[4] == 0).all() and np.isnan(y).sum() == 8 + 2
