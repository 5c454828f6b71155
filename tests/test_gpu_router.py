"""The router and its gradient on the GPU against the 64-bit numpy reference.

ids must be equal.  Gates: an fp32 exponential, a sum over at most 32 of them, a quotient and the
scale are below 16 half steps (2^-24), and the rounding of an exponent's argument l - max adds
half a step per unit of the row's spread.  Gradients are held to the sum of the absolute values
of their terms: softmax's denominator adds up to 22 roundings (16 experts a lane, six levels),
twice the spread's half steps and the dot product's; 64 covers them.  A bf16 gradient adds half of
its step, 2^-8."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def spread(l):
    f = np.where(np.isfinite(l), l, np.nan)
    if not np.isfinite(f).any():
        return 0.0
    return float(np.nanmax(f) - np.nanmin(f))


def make(T, E, dtype, seed=0, std=1.5, closed=0.0):
    rng = np.random.default_rng([seed, T, E])
    l = (std * rng.standard_normal((T, E))).astype(np.float32)
    if closed:
        l[rng.random((T, E)) < closed] = -np.inf
        l[rng.random(T) < closed] = -np.inf
    t = torch.from_numpy(l).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    return t, t.float().numpy().astype(np.float64), rng


def check(m, t, l, K, rng, bias=None, strided=False, ids_dtype=torch.int32, grad=True, **kw):
    say(f"[router] T,E={tuple(l.shape)} K={K} {t.dtype} bias={bias is not None} {kw}")
    T, E = l.shape
    dev = t.cuda()
    if strided:
        wide = torch.full((T, E + 5), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, 1:E + 1] = dev
        dev = wide[:, 1:E + 1]
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    w, ids = m.moe_ffn_router_fwd(dev, K, bias=b, ids_dtype=ids_dtype, **kw)
    torch.cuda.synchronize()
    assert ids.dtype == ids_dtype and w.dtype == torch.float32
    rw, rid = ops.router(l, K, bias=None if bias is None else bias.astype(np.float32), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    got = w.cpu().numpy().astype(np.float64)
    # below fp32's normal range a gate is off by its absolute step
    np.testing.assert_allclose(got, rw, rtol=(16 + spread(l)) * U, atol=2.0 ** -140)
    if not grad:
        return
    dw = rng.standard_normal((T, K)).astype(np.float32)
    form = {k: v for k, v in kw.items() if k in ("score", "renormalize", "scale")}
    d = m.moe_ffn_router_bwd(torch.from_numpy(dw).cuda(), dev, ids, **form)
    torch.cuda.synchronize()
    assert d.shape == l.shape and d.dtype == t.dtype and d.is_contiguous()
    rd, mag = ops.router_grad(dw, l, rid, **form)
    step = 0.0 if t.dtype == torch.float32 else 2.0 ** -8
    tol = (64 + 2 * spread(l)) * U * mag + step * np.abs(rd) + 2.0 ** -126
    err = np.abs(d.float().cpu().numpy().astype(np.float64) - rd)
    assert (err <= tol).all(), float((err / tol).max())


FORMS = [dict(score=s, renormalize=r) for s in ("softmax", "sigmoid") for r in (True, False)]
IDS = ["softmax-renorm", "softmax", "sigmoid-renorm", "sigmoid"]
SHAPES = [(1, 1, 1), (1, 256, 8), (3, 5, 5), (5, 16, 4), (64, 17, 3), (63, 64, 6), (65, 65, 7),
          (130, 128, 32), (33, 160, 6), (257, 256, 8), (50, 257, 1), (40, 511, 8), (21, 1000, 9),
          (9, 1024, 32)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sizes(gpu_lib, shape, form, dtype):
    T, E, K = shape
    t, l, rng = make(T, E, dtype)
    check(gpu_lib, t, l, K, rng, **form)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("shape", [(70, 24, 4), (33, 130, 6), (257, 256, 8), (20, 1024, 32)], ids=str)
def test_bias_closed_experts_scale_and_strides(gpu_lib, shape, form):
    T, E, K = shape
    t, l, rng = make(T, E, "f32", seed=1, closed=0.2)
    bias = 0.2 * rng.standard_normal(E)
    bias[E // 3] = -np.inf
    check(gpu_lib, t, l, K, rng, bias=bias, strided=True, ids_dtype=torch.int64, scale=2.5, **form)
    t, l, rng = make(T, E, "bf16", seed=2, closed=0.9)
    check(gpu_lib, t, l, K, rng, strided=True, scale=0.5, **form)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("with_bias", [True, False], ids=["bias", "plain"])
@pytest.mark.parametrize("E,groups,topk_groups,group_top,K", [
    (256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (64, 8, 3, 2, 6), (16, 4, 1, 2, 4), (160, 8, 3, 1, 6),
    (128, 64, 5, 2, 10), (1024, 64, 1, 2, 16), (1024, 2, 1, 2, 32), (63, 9, 9, 2, 5),
    (24, 24, 3, 1, 3), (96, 12, 5, 2, 7), (384, 3, 2, 2, 12)])
def test_groups(gpu_lib, E, groups, topk_groups, group_top, K, with_bias, form):
    for dtype, closed in (("f32", 0.0), ("bf16", 0.3)):
        t, l, rng = make(150, E, dtype, seed=3, closed=closed)
        bias = 0.1 * rng.standard_normal(E) if with_bias else None
        check(gpu_lib, t, l, K, rng, bias=bias, groups=groups, topk_groups=topk_groups,
              group_top=group_top, **form)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("with_bias", [True, False], ids=["bias", "plain"])
def test_ties_go_to_the_lower_id(gpu_lib, with_bias, form):
    for E, groups in ((16, 4), (64, 8), (200, 8), (1024, 16)):
        rng = np.random.default_rng(E)
        l = rng.integers(-2, 3, size=(120, E)).astype(np.float32)
        l[7] = 1.0
        t = torch.from_numpy(l)
        bias = rng.integers(0, 2, size=E) * 0.25 if with_bias else None
        for g in (1, groups):
            check(gpu_lib, t, l.astype(np.float64), 8, rng, bias=bias, groups=g,
                  topk_groups=max(1, g // 2), group_top=2 if g > 1 else 1, **form)


def test_scores_next_to_each_other(gpu_lib):
    """Keys that differ by less than fp32's step: ids must follow the 64-bit order."""
    rng = np.random.default_rng(11)
    E, T = 64, 400
    for trial in range(4):
        l = rng.standard_normal((T, E)).astype(np.float32)
        s = 1 / (1 + np.exp(-l[0].astype(np.float64)))
        # biases that bring every expert of row 0 to about the same key; the other rows are
        # row 0 with single last places of the logits changed
        bias = (0.75 - s).astype(np.float32)
        for t in range(T):
            l[t] = l[0]
            j = rng.integers(0, E, 20)
            l[t, j] = np.nextafter(l[t, j], np.float32(rng.choice([-9, 9])))
        check(gpu_lib, torch.from_numpy(l), l.astype(np.float64), 8, rng, bias=bias,
              score="sigmoid")
        check(gpu_lib, torch.from_numpy(l), l.astype(np.float64), 8, rng, bias=bias,
              score="sigmoid", groups=8, topk_groups=3, group_top=2)
        check(gpu_lib, torch.from_numpy(l), l.astype(np.float64), 8, rng, score="softmax",
              groups=8, topk_groups=3, group_top=2)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_extreme_logits(gpu_lib, form):
    big = float(np.finfo(np.float32).max)
    rows = [[-big] * 8, [big] * 8, [-big, 0, 1, 2, big, 3, 4, 5], [80.0, -80, 60, 88, 1, 2, 3, 4],
            [-100.0, -101, -102, -103, -104, -105, -106, -107],
            [200.0, 199, 198, 3, 2, 1, 0, -1], [0.0] * 8, [1e-40, -1e-40, 0, 0, 1e-39, 0, 0, 0]]
    l = np.array(rows, np.float32)
    say("[router] extreme logits", form)
    for K in (1, 3, 8):
        dev = torch.from_numpy(l).cuda()
        w, ids = gpu_lib.moe_ffn_router_fwd(dev, K, **form)
        rw, rid = ops.router(l, K, **form)
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)
        # spreads of single rows: rows 0-2 have gates of 0, 1 and 1/K only
        np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=(16 + 168) * U, atol=2.0 ** -126)
        d = gpu_lib.moe_ffn_router_bwd(torch.ones_like(w), dev, ids, **form)
        rd, mag = ops.router_grad(np.ones_like(rw), l, rid, **form)
        np.testing.assert_array_less(np.abs(d.cpu().numpy() - rd), (64 + 400) * U * mag + 2.0 ** -125)


def test_nan_and_infinity(gpu_lib):
    inf, nan = float("inf"), float("nan")
    l = np.array([[nan, 1, 2, 3], [nan] * 4, [nan, -inf, -inf, 0], [inf, 0, 1, -inf],
                  [-inf] * 4, [0, 1, 2, 3]], np.float32)
    say("[router] NaN and infinity")
    dev = torch.from_numpy(l).cuda()
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            w, ids = gpu_lib.moe_ffn_router_fwd(dev, 3, score=score, renormalize=renormalize)
            w, ids = w.cpu().numpy(), ids.cpu().numpy()
            # NaN is below every number and above the closed experts
            assert ids.tolist() == [[3, 2, 1], [0, 1, 2], [3, 0, -1], [0, 2, 1], [-1] * 3,
                                    [3, 2, 1]]
            assert np.isnan(w[1]).all() and np.isnan(w[2, 1]) and w[2, 2] == 0
            assert (w[4] == 0).all() and np.isfinite(w[5]).all()
            if score == "softmax":
                assert np.isnan(w[0]).all() and np.isnan(w[3]).all()
            else:
                assert np.isfinite(w[0]).all() and np.isfinite(w[3]).all()
            d = gpu_lib.moe_ffn_router_bwd(torch.ones(6, 3, device="cuda"), dev,
                                           torch.from_numpy(ids).cuda(), score=score,
                                           renormalize=renormalize).cpu().numpy()
            assert (d[4] == 0).all() and np.isfinite(d[5]).all()
            assert np.isnan(d[1, :3]).all()


def test_gradient_of_repeated_and_foreign_ids(gpu_lib):
    """The backward takes any ids: a repeated one adds up, one outside [0, E) or of a closed
    expert has no part."""
    rng = np.random.default_rng(17)
    l = rng.standard_normal((40, 20)).astype(np.float32)
    l[:, 7] = -np.inf
    ids = rng.integers(-2, 24, size=(40, 6))
    ids[:5] = 3
    ids[5] = [-1] * 6
    ids[6] = [1 << 40] * 6
    dw = rng.standard_normal((40, 6)).astype(np.float32)
    for form in FORMS:
        say("[router] foreign ids", form)
        d = gpu_lib.moe_ffn_router_bwd(torch.from_numpy(dw).cuda(), torch.from_numpy(l).cuda(),
                                       torch.from_numpy(ids).cuda(), **form).cpu().numpy()
        rd, mag = ops.router_grad(dw, l, ids, **form)
        assert (np.abs(d - rd) <= (64 + 20) * U * mag).all()


def test_no_tokens(gpu_lib):
    say("[router] T=0")
    w, ids = gpu_lib.moe_ffn_router_fwd(torch.zeros(0, 8, device="cuda"), 2)
    assert w.shape == (0, 2) and ids.shape == (0, 2)
    d = gpu_lib.moe_ffn_router_bwd(w, torch.zeros(0, 8, device="cuda"), ids)
    assert d.shape == (0, 8)


def test_refusals(gpu_lib):
    say("[router] refusals")
    l = torch.zeros(4, 8, device="cuda")
    for kw in (dict(K=9), dict(K=0), dict(K=2, groups=3), dict(K=2, score="relu"),
               dict(K=2, bias=torch.zeros(7, device="cuda")), dict(K=2, bias=torch.zeros(8)),
               dict(K=2, bias=torch.zeros(8, device="cuda", dtype=torch.float64))):
        with pytest.raises(gpu_lib.MoEFFNError):
            gpu_lib.moe_ffn_router_fwd(l, **kw)
    with pytest.raises(gpu_lib.MoEFFNError):
        gpu_lib.moe_ffn_router_fwd(l.t(), 2)
    with pytest.raises(gpu_lib.MoEFFNError):
        gpu_lib.moe_ffn_router_fwd(l.half(), 2)
    with pytest.raises(gpu_lib.MoEFFNError):
        gpu_lib.moe_ffn_router_fwd(l[:1].expand(4, 8), 2)
    w, ids = gpu_lib.moe_ffn_router_fwd(l, 2)
    with pytest.raises(gpu_lib.MoEFFNError):
        gpu_lib.moe_ffn_router_bwd(w[:3], l, ids)
    with pytest.raises(gpu_lib.MoEFFNError):
        gpu_lib.moe_ffn_router_bwd(w.double(), l, ids)
    with pytest.raises(gpu_lib.MoEFFNError):
        gpu_lib.moe_ffn_router_bwd(w, l.cpu(), ids)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_autograd_with_the_layer(gpu_lib, form):
    """Router and layer together, as a training step runs them: the gradient of the logits through
    gates and experts equals the router's backward of the layer's d_topk_weights."""
    say("[router] with the layer", form)
    g = torch.Generator().manual_seed(5)
    T, H, I, E, K = 96, 256, 128, 8, 2
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    up = (torch.randn(E, H, 2 * I, generator=g) / 16).bfloat16().cuda()
    down = (torch.randn(E, I, H, generator=g) / 11).bfloat16().cuda()
    dy = torch.randn(T, H, generator=g).bfloat16().cuda()
    l = torch.randn(T, E, generator=g)
    l[5] = -float("inf")  # a padded token
    logits = l.cuda().requires_grad_(True)
    w, ids = gpu_lib.moe_ffn_router(logits, K, scale=1.5, **form)
    assert not ids.requires_grad and w.requires_grad
    y = gpu_lib.moe_ffn(x, ids, w, up, down)
    y.backward(dy)
    torch.cuda.synchronize()
    assert (y[5] == 0).all() and (logits.grad[5] == 0).all()
    _, saved = gpu_lib.moe_ffn_fwd(x, ids, w.detach(), up, down, save_for_backward=True)
    d_topk = gpu_lib.moe_ffn_bwd(dy, x, ids, w.detach(), up, down, saved)[3]
    rd, mag = ops.router_grad(d_topk.cpu().numpy(), l.numpy(), ids.cpu().numpy(), scale=1.5, **form)
    err = np.abs(logits.grad.cpu().numpy() - rd)
    assert (err <= (64 + 2 * spread(l.numpy())) * U * mag).all()


def test_second_derivative_is_refused(gpu_lib):
    l = torch.randn(6, 16, device="cuda", requires_grad=True)
    w, _ = gpu_lib.moe_ffn_router(l, 2)
    g, = torch.autograd.grad((w * w).sum(), l, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_graph_replays_and_other_streams(gpu_lib):
    say("[router] graph and streams")
    l = torch.randn(300, 64, device="cuda")
    dw = torch.randn(300, 6, device="cuda")
    bias = 0.1 * torch.randn(64, device="cuda")

    def step():
        w, ids = gpu_lib.moe_ffn_router_fwd(l, 6, bias=bias, score="sigmoid", groups=8,
                                            topk_groups=4, group_top=2)
        return w, ids, gpu_lib.moe_ffn_router_bwd(dw, l, ids, score="sigmoid")

    ref = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    for a, b in zip(other, ref):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
        step()
        torch.cuda.synchronize()


def test_long_batch_with_rows_past_32_bit_offsets(gpu_lib):
    """Rows whose element offset passes 2^31 (a wide stride): the same results as those rows alone."""
    T, E, stride = 40000, 64, 60000
    say(f"[router] offsets past 2^31: T={T} stride={stride}")
    buf = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    l = buf.view(T, stride)[:, :E]
    l.copy_(torch.randn(T, E, device="cuda"))
    w, ids = gpu_lib.moe_ffn_router_fwd(l, 6)
    dw = torch.randn(T, 6, device="cuda")
    d = gpu_lib.moe_ffn_router_bwd(dw, l, ids, renormalize=False)
    tail = l[-700:].contiguous()
    w2, ids2 = gpu_lib.moe_ffn_router_fwd(tail, 6)
    d2 = gpu_lib.moe_ffn_router_bwd(dw[-700:].contiguous(), tail, ids2, renormalize=False)
    assert torch.equal(ids[-700:], ids2) and torch.equal(w[-700:], w2)
    assert torch.equal(d[-700:], d2)


@pytest.mark.parametrize("T,E,K", [((1 << 28) + 37, 2, 1), ((1 << 26) + 21, 17, 17)], ids=str)
def test_batches_of_more_rows_than_a_launch_takes(gpu_lib, T, E, K):
    """Every row as in a small batch: the rows repeat a table of 2^16 + 1, so no part looks like another."""
    say(f"[router] T={T} E={E} K={K}")
    n = (1 << 16) + 1
    table = torch.randn(n, E, device="cuda").bfloat16()
    l = table.repeat(T // n + 1, 1)[:T]
    dw = torch.randn(n, K, device="cuda").repeat(T // n + 1, 1)[:T]
    w0, i0 = gpu_lib.moe_ffn_router_fwd(table, K)
    d0 = gpu_lib.moe_ffn_router_bwd(dw[:n], table, i0, renormalize=False)
    w, ids = gpu_lib.moe_ffn_router_fwd(l, K)
    d = gpu_lib.moe_ffn_router_bwd(dw, l, ids, renormalize=False)
    for got, ref in ((w, w0), (ids, i0), (d, d0)):
        whole = T // n * n
        assert (got[:whole].view(T // n, -1) == ref.view(1, -1)).all()
        assert torch.equal(got[whole:], ref[:T - whole])
