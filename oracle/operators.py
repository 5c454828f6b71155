"""Plain numpy reference, in 64 bits, of the operators beside the layer: the router and its
gradient, the block-scaled 4- and 6-bit formats, and the expert FFN on MXFP4 weights.

Written from the formulas, row by row where that is plainer; used only by the tests.
"""

from __future__ import annotations

import numpy as np

__all__ = ["router", "router_grad", "mx_quantize", "mx_quantize_columns", "mxfp4_ffn"]


# ---- router -------------------------------------------------------------------------

def _scores(l, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    with np.errstate(invalid="ignore"):
        e = np.exp(l - top)
    return e / e.sum()


# a NaN key: below every fp32 number, as is the sum of two, and above a closed expert's -inf
_NAN_KEY = -1e300


def _best(values, n):
    """Indices of the n largest, descending, ties to the lower index."""
    return np.argsort(-values, kind="stable")[:n]


def router(logits, K, bias=None, score="softmax", renormalize=True, groups=1, topk_groups=1,
           group_top=1, scale=1.0):
    """(weights [T, K] f64, ids [T, K]) of logits [T, E] (any float array)."""
    L = np.asarray(logits, np.float64)
    T, E = L.shape
    ids = np.full((T, K), -1, np.int64)
    w = np.zeros((T, K))
    for t in range(T):
        l = L[t]
        s = _scores(l, score)
        closed = l == -np.inf
        key = l.copy() if bias is None else s + np.asarray(bias, np.float64)
        if bias is not None:
            closed |= np.asarray(bias) == -np.inf
        key = np.where(np.isnan(key), _NAN_KEY, key)
        key[closed] = -np.inf
        if topk_groups < groups:
            rank = key if bias is not None or group_top == 1 else np.where(
                closed, -np.inf, np.where(np.isnan(s), _NAN_KEY, s))
            best = -np.sort(-rank.reshape(groups, -1), axis=1)[:, :group_top]
            few = (best == -np.inf).any(1)  # of +inf and a closed expert there is no sum
            kept = _best(np.where(few, -np.inf, np.where(few[:, None], 0, best).sum(1)), topk_groups)
            mask = np.ones(groups, bool)
            mask[kept] = False
            key[np.repeat(mask, E // groups)] = -np.inf
        pick = _best(key, K)
        pick = pick[key[pick] > -np.inf]
        n = len(pick)
        if n == 0:
            continue
        ids[t, :n] = pick
        if renormalize and score == "softmax":
            with np.errstate(invalid="ignore"):
                e = np.exp(l[pick] - l[pick].max())
            v = e / e.sum()
        elif renormalize:
            # s = e^min(l, 0) / (1 + e^-|l|), with the common factor taken out of the ratio
            low = np.minimum(l[pick], 0.0)
            e = np.exp(low - low.max()) / (1.0 + np.exp(-np.abs(l[pick])))
            v = e / e.sum()
        else:
            v = s[pick]
        if score == "softmax" and (np.isnan(l) | (l == np.inf)).any():
            v = np.full(n, np.nan)
        w[t, :n] = scale * v
    return w, ids


def router_grad(d_weights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    """(d_logits [T, E], magnitude [T, E]): the gradient and the sum of the absolute values of
    the terms that it is added up from."""
    L = np.asarray(logits, np.float64)
    T, E = L.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        l = L[t]
        live = [(k, int(i)) for k, i in enumerate(ids[t]) if 0 <= i < E and l[int(i)] > -np.inf]
        if not live:
            continue
        ks, js = np.array([k for k, _ in live]), np.array([j for _, j in live])
        g = scale * np.asarray(d_weights, np.float64)[t, ks]
        if renormalize:
            low = np.minimum(l[js], 0.0) if score == "sigmoid" else l[js]
            u = np.exp(low - low.max())
            if score == "sigmoid":
                u = u / (1.0 + np.exp(-np.abs(l[js])))
            u = u / u.sum()
            part, size = u * (g - (g * u).sum()), u * (np.abs(g) + (np.abs(g) * u).sum())
            if score == "sigmoid":
                with np.errstate(over="ignore"):
                    part, size = part / (1.0 + np.exp(l[js])), size / (1.0 + np.exp(l[js]))
            np.add.at(d[t], js, part)
            np.add.at(mag[t], js, size)
        elif score == "sigmoid":
            e = np.exp(-np.abs(l[js]))
            part = g * e / (1.0 + e) ** 2
            np.add.at(d[t], js, part)
            np.add.at(mag[t], js, np.abs(part))
        else:
            p = _scores(l, score)
            own, size = np.zeros(E), np.zeros(E)
            np.add.at(own, js, g)
            np.add.at(size, js, np.abs(g))
            d[t] = np.where(l == -np.inf, 0.0, p * (own - (g * p[js]).sum()))
            mag[t] = np.where(l == -np.inf, 0.0, p * (size + (np.abs(g) * p[js]).sum()))
    return d, mag


# ---- block-scaled formats --------------------------------------------------------------

_E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
_E2M3 = np.array([m / 8 for m in range(8)]
                 + [(1 + m / 8) * 2.0 ** e for e in range(3) for m in range(8)])
_FORMATS = {"mxfp4": (_E2M1, 2), "mxfp6": (_E2M3, 2)}


def _round(a, grid):
    """Index of the nearest grid value of a >= 0, ties to the even index, saturating."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, a)
    tie = a == mid[np.minimum(i, len(mid) - 1)]
    return np.where(tie & (i % 2 == 1) & (i < len(mid)), i + 1, i)


def mx_quantize(v, fmt="mxfp4", slack=None):
    """Values that blocks of 32 along the last axis stand for.

    With ``slack`` (an array like v: how far another evaluation's input may lie from v) also
    returns, per value, how far that evaluation's quantised value may lie from this one's: 0
    unless the rounding or the block's scale could go the other way.
    """
    v = np.asarray(v, np.float64)
    grid, top_exp = _FORMATS[fmt]
    n = v.shape[-1]
    pad = [(0, 0)] * (v.ndim - 1) + [(0, -n % 32)]
    b = np.pad(v, pad).reshape(*v.shape[:-1], -1, 32)
    amax = np.abs(b).max(-1, keepdims=True)
    bad = ~np.isfinite(b).all(-1, keepdims=True)

    def unit_of(m):
        m = np.where(bad | (m == 0), 1.0, m)
        e = np.frexp(m)[1] - 1 - top_exp
        return np.ldexp(1.0, np.maximum(e, -127))

    unit = unit_of(amax)
    unit = np.where(amax == 0, 2.0 ** -127, unit)
    with np.errstate(invalid="ignore"):
        a = np.where(bad, 0.0, np.abs(b)) / unit
        q = np.where(bad, np.nan, np.copysign(grid[_round(a, grid)] * unit, b))
    out = q.reshape(*v.shape[:-1], -1)[..., :n]
    if slack is None:
        return out
    sl = np.pad(slack, pad).reshape(b.shape)
    lo = np.maximum(np.abs(b) - sl, 0.0)
    hi = np.abs(b) + sl
    off = np.zeros_like(b)
    m_lo, m_hi = lo.max(-1, keepdims=True), hi.max(-1, keepdims=True)
    for m in (m_lo, m_hi):  # the scale of either end; inside one octave there are no others
        un = unit_of(m)
        for x in (lo, hi):
            with np.errstate(invalid="ignore"):
                r = grid[_round(np.where(bad, 0.0, x) / un, grid)] * un
            off = np.maximum(off, np.abs(r - np.abs(np.where(bad, 0.0, q))))
    crossed = sl > np.abs(b)  # the sign may differ: then both magnitudes count
    off = np.where(crossed, off + 2 * np.abs(np.where(bad, 0.0, q)), off)
    return out, off.reshape(*v.shape[:-1], -1)[..., :n]


def mx_quantize_columns(w, fmt="mxfp4"):
    """The same for weights [..., Kd, N], blocks down the columns."""
    return np.swapaxes(mx_quantize(np.swapaxes(np.asarray(w, np.float64), -1, -2), fmt), -1, -2)


# ---- expert FFN on MXFP4 weights -----------------------------------------------------------

def mxfp4_ffn(x, ids, gates, up, down, act="mxfp4"):
    """(y, tol): the layer on weights quantised to MXFP4 and activations to ``act``, and how far
    the bf16 output of an evaluation with fp32 sums may lie from it.

    The tolerance adds up
    * sums of h: each matrix instruction adds 64 products to an fp32 sum; 2^-22 of the sum of the
      products' magnitudes per instruction (four half steps of fp32) and four more for joining
      partial sums;
    * silu and the product: 16 half steps of fp32;
    * an act value that those errors may carry over a rounding border: the two values' distance
      times the weight's magnitude;
    * sums of o like those of h, o and y each rounded to bf16 (half a step is 2^-8 of the value),
      gates and the sum over K in fp32 (2 K half steps).
    """
    x, gates = np.asarray(x, np.float64), np.asarray(gates, np.float64)
    T, H = x.shape
    E, I = down.shape[0], down.shape[1]
    K = ids.shape[1]
    wu, wd = mx_quantize_columns(up), mx_quantize_columns(down)
    xq = mx_quantize(x, act)
    y, tol, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    e_h = ((H + 63) // 64 + 4) * 2.0 ** -22
    e_o = ((I + 63) // 64 + 4) * 2.0 ** -22
    for e in range(E):
        t, k = np.nonzero(np.asarray(ids) == e)
        if len(t) == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            h = xq[t] @ wu[e]
            dh = e_h * (np.abs(xq[t]) @ np.abs(wu[e]))
            g, u = h[:, :I], h[:, I:]
            dg, du = dh[:, :I], dh[:, I:]
            sig = 1.0 / (1.0 + np.exp(-g))
            a = g * sig * u
            # |silu'| <= 1.1
            da = 1.1 * dg * (np.abs(u) + du) + np.abs(g * sig) * du + 16 * 2.0 ** -24 * np.abs(a)
            aq, off = mx_quantize(a, act, slack=da)
            o = aq @ wd[e]
            do = off @ np.abs(wd[e]) + e_o * ((np.abs(aq) + off) @ np.abs(wd[e]))
            do = do + 2.0 ** -8 * (np.abs(o) + do)
            w = gates[t, k][:, None]
            np.add.at(y, t, w * o)
            np.add.at(tol, t, np.abs(w) * do)
            np.add.at(mag, t, np.abs(w * o))
    tol = tol + 2 * K * 2.0 ** -24 * mag
    return y, tol + 2.0 ** -8 * (np.abs(y) + tol) + 1e-30
