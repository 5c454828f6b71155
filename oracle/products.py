"""Plain numpy reference, in 64 bits, of the experts' products on their own: the product of row
groups with its gradients, int8 quantisation, the int8 product and the expert FFN on int8 weights.

Written from the formulas; used only by the tests.
"""

from __future__ import annotations

import numpy as np

__all__ = ["groups", "grouped_mm", "grouped_mm_grad", "int8_codes", "int8_mm", "int8_ffn"]


def groups(offsets, M):
    """Row ranges of the groups: each offset held to [0, M], then their running maximum."""
    o = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, M))
    return [(int(a), int(b)) for a, b in zip(o[:-1], o[1:])]


def grouped_mm(x, w, offsets, transposed=False):
    """(y, mag): rows of group e times w[e] (transposed if so), and the sums of the products'
    magnitudes, by which rounding errors of the sums are counted."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    M, N = x.shape[0], w.shape[1] if transposed else w.shape[2]
    y, mag = np.zeros((M, N)), np.zeros((M, N))
    for e, (a, b) in enumerate(groups(offsets, M)):
        if a < b:
            we = w[e].T if transposed else w[e]
            y[a:b] = x[a:b] @ we
            with np.errstate(invalid="ignore"):
                mag[a:b] = np.abs(x[a:b]) @ np.abs(we)
    return y, mag


def grouped_mm_grad(dy, x, w, offsets, transposed=False):
    """((dx, mag), (dw, mag)) of grouped_mm."""
    dy, x, w = (np.asarray(v, np.float64) for v in (dy, x, w))
    dx = grouped_mm(dy, w, offsets, not transposed)
    dw, mag = np.zeros_like(w), np.zeros_like(w)
    for e, (a, b) in enumerate(groups(offsets, x.shape[0])):
        if a < b:
            g = x[a:b].T @ dy[a:b]
            m = np.abs(x[a:b]).T @ np.abs(dy[a:b])
            dw[e], mag[e] = (g.T, m.T) if transposed else (g, m)
    return dx, (dw, mag)


def _scale(v, axis):
    """max|v| / 127 in fp32 (kept as fp64, with the axis); NaN where v is not finite."""
    bad = ~np.isfinite(v).all(axis, keepdims=True)
    with np.errstate(invalid="ignore"):
        top = np.abs(v).max(axis, keepdims=True, initial=0.0)
    s = (np.where(bad, 0.0, top) / 127.0).astype(np.float32).astype(np.float64)
    return s, bad


def int8_codes(v, axis, slack=None):
    """(codes, scales) of v along axis, both fp64; scales without the axis, NaN where v holds a NaN
    or an infinity (codes 0 then).

    With ``slack`` (>= 0, v's shape: how far an evaluation's values may lie from v) also how far
    its code * scale may lie from this one's."""
    v = np.asarray(v, np.float64)
    s, bad = _scale(v, axis)

    def codes(x, s):
        t = np.where(bad, 0.0, x) / np.where(s > 0, s, 1.0)
        return np.where(s > 0, np.clip(np.rint(t), -127, 127), 0.0)

    q = codes(v, s)
    out = np.where(bad, np.nan, s).squeeze(axis)
    if slack is None:
        return q, out
    off = np.zeros_like(q)
    mag = np.abs(np.where(bad, 0.0, v))
    lo_s, hi_s = (_scale(np.maximum(m, 0.0), axis)[0] for m in (mag - slack, mag + slack))
    # the least and the largest code, each with the least and the largest scale
    for c in (codes(np.maximum(mag - slack, 0.0), hi_s), codes(mag + slack, lo_s)):
        for sc in (lo_s, hi_s):
            off = np.maximum(off, np.abs(c * sc - np.abs(q) * s))
    off = np.where(slack > mag, off + 2 * np.abs(q) * s, off)  # the sign may differ
    return q, out, off


def int8_mm(codes, scales, wcodes, wscales, offsets=None):
    """y of int8 rows (codes [M, Kd], scales [M]) and weights (wcodes [E, Kd, N], wscales [E, N])."""
    codes, wcodes = np.asarray(codes, np.float64), np.asarray(wcodes, np.float64)
    M, (E, _, N) = codes.shape[0], wcodes.shape
    ranges = [(0, M)] if offsets is None else groups(offsets, M)
    y = np.zeros((M, N))
    for e, (a, b) in enumerate(ranges):
        y[a:b] = (codes[a:b] @ wcodes[e]) * np.asarray(scales)[a:b, None] * np.asarray(wscales)[e]
    return y


def int8_ffn(x, ids, gates, up, down):
    """(y, tol): the layer on weights quantised to int8 and activations too, row by row, and how
    far the bf16 output of an evaluation in fp32 (with exact integer sums) may lie from it.

    The tolerance adds up: four half steps of fp32 for h (the sum's conversion, two scales), silu and the
    product (|silu'| <= 1.1; 16 half steps, and |g| of them for the exponential's argument); an act value that
    these may carry to another code, and the change of its row's scale; four half steps for o, gates
    and the sum over K in fp32 (2 K half steps), y rounded to bf16 (half a step is 2^-8 of the value).
    """
    x, gates = np.asarray(x, np.float64), np.asarray(gates, np.float64)
    T, H = x.shape
    E, I = down.shape[0], down.shape[1]
    K = ids.shape[1]
    half = 2.0 ** -24
    xq, sx = int8_codes(x, 1)
    y, tol, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, k = np.nonzero(np.asarray(ids) == e)
        if len(t) == 0:
            continue
        wu, su = int8_codes(up[e], 0)
        wd, sd = int8_codes(down[e], 0)
        with np.errstate(invalid="ignore", over="ignore"):
            h = (xq[t] @ wu) * sx[t, None] * su
            dh = 4 * half * np.abs(h)
            g, u = h[:, :I], h[:, I:]
            sig = 1.0 / (1.0 + np.exp(-g))
            a = g * sig * u
            da = (1.1 * dh[:, :I] * (np.abs(u) + dh[:, I:]) + np.abs(g * sig) * dh[:, I:]
                  + (16 + np.abs(g)) * half * np.abs(a))
            aq, sa, off = int8_codes(a, 1, slack=np.where(np.isfinite(da), da, 0.0))
            o = (aq @ wd) * sa[:, None] * sd
            do = (off @ np.abs(wd)) * sd
            do = do + 4 * half * (np.abs(o) + do)
            w = gates[t, k][:, None]
            np.add.at(y, t, w * o)
            np.add.at(tol, t, np.abs(w) * do)
            np.add.at(mag, t, np.abs(w * o))
    tol = tol + 2 * K * half * mag
    return y, tol + 2.0 ** -8 * (np.abs(y) + tol) + 1e-30
