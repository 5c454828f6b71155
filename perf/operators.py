"""The operators beside the expert FFN and the work they are measured on.

Three families: the router (logits to the expert ids and gates that the layer takes, and its gradient),
the MXFP4 quantisation of expert weights, and the expert FFN on MXFP4 weights.  ``run`` computes them in
their plain form from elementary torch operations, or, where ``own`` is true, with the library's calls.

MXFP4 and MXFP6 here: blocks of 32 consecutive values along the contraction axis share a power of two,
2^(floor(log2(largest magnitude)) - 2); each element is the value divided by it, as an e2m1 (MXFP4) or
e2m3 (MXFP6) number: rounded to nearest, ties to even, saturated at 6 and 7.5.
"""

import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases ------------------------------------------------------------------------------------

def _router(T, E, K, dtype, score, renormalize, bias=False, groups=1, topk_groups=1, group_top=1,
            scale=1.0, masked=0.0, grad=False):
    return dict(op="router", T=T, E=E, K=K, dtype=dtype, score=score, renormalize=renormalize,
                bias=bias, groups=groups, topk_groups=topk_groups, group_top=group_top, scale=scale,
                masked=masked, grad=grad)


def _quantize(E, Kd, N, panels, dtype):
    return dict(op="quantize", E=E, Kd=Kd, N=N, panels=panels, dtype=dtype)


def _ffn(T, H, I, E, K, act, routing="uniform"):
    return dict(op="ffn", T=T, H=H, I=I, E=E, K=K, act=act, routing=routing)


def listed():
    return [
        # one token of a serving loop: 256 experts in 8 groups, balance bias, sigmoid scores
        dict(_router(1, 256, 8, "f32", "sigmoid", True, True, 8, 4, 2, 2.5), name="router token"),
        # the prefill workload's routing (64 experts, top 6), logits as a bf16 product leaves them
        dict(_router(4096, 64, 6, "bf16", "softmax", True), name="router prefill"),
        # a long prompt batch over the grouped router
        dict(_router(32768, 256, 8, "f32", "sigmoid", True, True, 8, 4, 2, 2.5), name="router long"),
        # the forward+backward workload's routing (16 experts, top 4), with its gradient
        dict(_router(4096, 16, 4, "f32", "softmax", True, grad=True), name="router step"),
        # a padded training batch of odd sizes: gates are the plain probabilities, so that every
        # logit has a gradient; padded rows and switched-off experts are -inf
        dict(_router(19973, 160, 6, "bf16", "softmax", False, masked=0.05, grad=True),
             name="router step padded"),
        # weights as a checkpoint is loaded: the tiny fp32 layer, and the prefill layer's up_proj
        dict(_quantize(8, 256, 1024, 2, "f32"), name="quantize small"),
        dict(_quantize(64, 2048, 2816, 2, "bf16"), name="quantize up_proj"),
        # one token through the decode workload's experts
        dict(_ffn(1, 7168, 2048, 32, 8, "mxfp4"), name="ffn token"),
        # the decode workload, with the finer activations
        dict(_ffn(128, 7168, 2048, 32, 8, "mxfp6"), name="ffn decode"),
        # sizes that are no multiple of any tile
        dict(_ffn(601, 264, 200, 6, 2, "mxfp6"), name="ffn ragged"),
        # the prefill workload
        dict(_ffn(4096, 2048, 1408, 64, 6, "mxfp4"), name="ffn prefill"),
        # the skewed workload: popular experts with thousands of rows, others empty
        dict(_ffn(8192, 7168, 2048, 32, 8, "mxfp4", "zipf"), name="ffn skewed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "router", "quantize", "ffn", "ffn", "ffn"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "router":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(4, _log(rng, 8, 384) // groups)
        topk_groups = rng.randint(max(1, groups // 2), groups)
        K = rng.randint(1, min(16, topk_groups * (E // groups)))
        return _router(_log(rng, 1, 32768), E, K, dtype, rng.choice(["softmax", "sigmoid"]),
                       rng.random() < 0.6, rng.random() < 0.5, groups, topk_groups,
                       rng.choice([1, 2]), rng.choice([1.0, 2.5]), rng.choice([0.0, 0.0, 0.1]),
                       rng.random() < 0.5)
    if op == "quantize":
        return _quantize(rng.randint(1, 32), 8 * _log(rng, 4, 512), 16 * _log(rng, 4, 256),
                         rng.choice([1, 2]), dtype)
    E = _log(rng, 2, 64)
    return _ffn(_log(rng, 1, 4096), 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 256), E,
                rng.randint(1, min(8, E)), rng.choice(["mxfp4", "mxfp6"]),
                rng.choice(["uniform", "zipf"]))


def work(case):
    if case["op"] == "router":
        n, item = case["T"] * case["E"], 4 if case["dtype"] == "f32" else 2
        nbytes = n * item + case["T"] * case["K"] * 8 + (4 * case["E"] if case["bias"] else 0)
        flops = 4 * n
        if case["grad"]:
            nbytes += n * item + case["T"] * case["K"] * 4
            flops += 4 * n
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "quantize":
        n, item = case["E"] * case["Kd"] * case["N"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * (2 * item + 17 / 32), "flops": 4 * n}
    T, H, I, E, K = (case[k] for k in "THIEK")
    hit = E * (1 - (1 - K / E) ** T)  # experts that a uniform routing reaches
    return {"bytes": int(hit * 3 * H * I * 17 / 32 + 2 * T * H * 2 + T * K * 8),
            "flops": 6 * T * K * H * I}


# ---- inputs -----------------------------------------------------------------------------------

def _round_e2m1(a):
    """Magnitudes to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to even)."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0)


def _round_e2m3(a):
    """Magnitudes to the nearest in steps of 1/8 up to 2, 1/4 up to 4, 1/2 up to 7.5."""
    step = torch.where(a < 2, 0.125, torch.where(a < 4, 0.25, 0.5))
    return (torch.round(a / step) * step).clamp(max=7.5)


def _mx(v, fmt="mxfp4"):
    """The values that blocks of 32 along the last axis stand for once quantised (fp32)."""
    n = v.shape[-1]
    v = torch.nn.functional.pad(v, (0, -n % 32)).unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(top)[1] - 1 - 2
    e = torch.where(top > 0, e, 0).clamp(min=-125)
    unit, inverse = (((s * e + 127) << 23).view(torch.float32) for s in (1, -1))
    a = v.abs() * inverse
    q = (_round_e2m1(a) if fmt == "mxfp4" else _round_e2m3(a)) * unit
    return torch.copysign(q, v).flatten(-2)[..., :n]


def _mx_columns(w):
    """The same with the blocks down the columns of a weight [Kd, N] or [E, Kd, N]."""
    return _mx(w.float().transpose(-1, -2)).transpose(-1, -2).to(w.dtype)


def _weights(gen, E, Kd, N, dtype):
    w = torch.empty(E, Kd, N, dtype=dtype, device="cuda")
    for e in range(E):
        w[e] = torch.randn(Kd, N, generator=gen, device="cuda").mul_(Kd ** -0.5)
    return w


def _routing(gen, T, E, K, routing):
    """Distinct experts for each token, uniformly or by a Zipf popularity, and softmax gates."""
    draw = -torch.log(torch.empty(T, E, device="cuda").exponential_(generator=gen))
    if routing == "zipf":
        rank = torch.randperm(E, generator=gen, device="cuda")
        draw = draw - 1.2 * torch.log1p(rank.float())
        draw[:, rank >= max(K, E - 3)] = -math.inf  # up to three experts stay empty
    top, ids = torch.sort(draw, dim=1, descending=True, stable=True)
    return ids[:, :K].to(torch.int32).contiguous(), torch.softmax(top[:, :K], 1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "router":
        T, E, K = case["T"], case["E"], case["K"]
        logits = 1.5 * torch.randn(T, E, generator=gen, device="cuda")
        if case["masked"]:
            # rows behind the batch's last token, and experts that a token may not take
            pad = torch.rand(T, 1, generator=gen, device="cuda") < case["masked"]
            off = torch.rand(T, E, generator=gen, device="cuda") < case["masked"]
            logits.masked_fill_(pad | off, -math.inf)
        s["logits"] = logits.to(_DTYPES[case["dtype"]])
        s["bias"] = 0.1 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
        if case["grad"]:
            s["d_weights"] = torch.randn(T, K, generator=gen, device="cuda")
    elif case["op"] == "quantize":
        s["w"] = _weights(gen, case["E"], case["Kd"], case["N"], _DTYPES[case["dtype"]])
    else:
        T, H, I, E, K = (case[k] for k in "THIEK")
        s["x"] = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
        s["ids"], s["gates"] = _routing(gen, T, E, K, case["routing"])
        # a checkpoint's quantised weights: bf16 holds every value that MXFP4 stands for
        for name, shape in (("up", (E, H, 2 * I)), ("down", (E, I, H))):
            w = _weights(gen, *shape, torch.bfloat16)
            for e in range(E):
                w[e] = _mx_columns(w[e])
            s[name] = w
        if own:
            # the library's handle of the weights, laid out once, and the workspace that a serving
            # loop keeps between its steps
            import mixture_experts_ffn_amd as moe
            s["up"] = moe.moe_ffn_mxfp4_quantize(s["up"], panels=2)
            s["down"] = moe.moe_ffn_mxfp4_quantize(s["down"])
            problem = moe.Problem(T, H, I, E, K, moe.BF16, moe.I32)
            s["ws"] = torch.empty(moe.mxfp4_workspace_size(problem, act=case["act"]),
                                  dtype=torch.uint8, device="cuda")
        else:
            # rows of the fullest expert: the height of the plain form's padded products
            s["rows"] = int(torch.bincount(s["ids"].flatten().long(), minlength=E).max())
    return s


# ---- plain forms ------------------------------------------------------------------------------

def _scores(logits, score):
    """Expert scores in 64 bits (selection by sums compares values that lie close together)."""
    v = logits.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    top = v.amax(1, keepdim=True)
    p = torch.exp(v - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _router_plain(s):
    c, logits, bias = s["case"], s["logits"], s["bias"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    score = _scores(logits, c["score"])
    open_ = logits > -math.inf
    # a score grows with its logit, so without a bias the logits order the experts
    key = score + bias if bias is not None else logits.double()
    key = torch.where(open_, key, -math.inf)
    if c["topk_groups"] < G:
        rank = key if bias is not None or c["group_top"] == 1 else torch.where(open_, score, -math.inf)
        best = torch.sort(rank.view(T, G, -1), dim=2, descending=True).values
        group = best[..., :c["group_top"]].sum(-1)
        kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, kept, True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    value, ids = torch.sort(key, dim=1, descending=True, stable=True)
    live = value[:, :K] > -math.inf
    ids = torch.where(live, ids[:, :K], -1)
    at = ids.clamp(min=0)
    chosen = torch.where(live, score.gather(1, at), 0.0)
    total = chosen.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    gates = c["scale"] * (chosen / total if c["renormalize"] else chosen)
    out = {"weights": gates.float(), "ids": ids.int()}
    if c["grad"]:
        g = s["d_weights"].double() * c["scale"] * live
        if c["renormalize"]:
            g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
        d = torch.zeros_like(score).scatter_add_(1, at, g)  # gradient of each expert's score
        if c["score"] == "sigmoid":
            d = d * score * (1 - score)
        else:
            d = score * (d - (d * score).sum(1, keepdim=True))
        out["d_logits"] = d.to(logits.dtype)
    return out


def _ffn_plain(s):
    c, ids = s["case"], s["ids"].long()
    T, H, I, E, K = (c[k] for k in "THIEK")
    x = _mx(s["x"].float(), c["act"])
    flat = ids.flatten()
    if T * K <= E:  # a few slots: each with its own expert's weights
        rows = x.repeat_interleave(K, 0).unsqueeze(1)
        up, down = s["up"][flat].float(), s["down"][flat].float()
    else:  # each expert's rows, padded to the fullest expert's
        order = torch.sort(flat, stable=True).indices
        start = torch.cumsum(torch.bincount(flat, minlength=E), 0)
        first = torch.cat([start.new_zeros(1), start[:-1]])
        place = torch.empty_like(flat)
        place[order] = torch.arange(T * K, device=flat.device) - first[flat[order]]
        rows = torch.zeros(E, s["rows"], H, device=x.device)
        rows[flat, place] = x.repeat_interleave(K, 0)
        up, down = s["up"].float(), s["down"].float()
    h = torch.bmm(rows, up)
    gate, lin = h[..., :I], h[..., I:]
    act = _mx(gate / (1 + torch.exp(-gate)) * lin, c["act"])
    o = torch.bmm(act, down)
    o = o.squeeze(1) if T * K <= E else o[flat, place]
    return (s["gates"].unsqueeze(2) * o.view(T, K, H)).sum(1).to(torch.bfloat16)


# ---- the library's calls ----------------------------------------------------------------------

def _router_own(s):
    import mixture_experts_ffn_amd as moe
    c = s["case"]
    form = dict(score=c["score"], renormalize=c["renormalize"], scale=c["scale"])
    weights, ids = moe.moe_ffn_router_fwd(s["logits"], c["K"], bias=s["bias"], groups=c["groups"],
                                          topk_groups=c["topk_groups"], group_top=c["group_top"],
                                          **form)
    out = {"weights": weights, "ids": ids}
    if c["grad"]:
        out["d_logits"] = moe.moe_ffn_router_bwd(s["d_weights"], s["logits"], ids, **form)
    return out


def _quantize_own(s):
    import mixture_experts_ffn_amd as moe
    packed = moe.moe_ffn_mxfp4_quantize(s["w"], panels=s["case"]["panels"])
    return moe.moe_ffn_mxfp4_dequantize(packed)


def _ffn_own(s):
    import mixture_experts_ffn_amd as moe
    return moe.moe_ffn_mxfp4_fwd(s["x"], s["ids"], s["gates"], s["up"], s["down"],
                                 act=s["case"]["act"], ws=s["ws"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"router": _router_own, "quantize": _quantize_own, "ffn": _ffn_own}[op](state)
    if op == "quantize":
        return _mx_columns(state["w"])
    return _router_plain(state) if op == "router" else _ffn_plain(state)


# ---- from the definitions, in 64 bits ---------------------------------------------------------

def _grid(fmt):
    if fmt == "mxfp4":
        return [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    return [m / 8 for m in range(16)] + [2 + m / 4 for m in range(8)] + [4 + m / 2 for m in range(8)]


def _mx64(v, fmt):
    """Nearest grid value in every block of 32 along the last axis, by search, in 64 bits."""
    n = v.shape[-1]
    v = torch.nn.functional.pad(v, (0, -n % 32)).unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    exponent = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    # log2 next to a power of two may round up to it
    exponent = torch.where(torch.exp2(exponent) > top, exponent - 1, exponent)
    unit = torch.exp2(torch.where(top > 0, exponent, 0.0) - 2)
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=v.device)
    a = v.abs() / unit
    middle = (grid[1:] + grid[:-1]) / 2
    low = torch.searchsorted(middle, a)  # a value on a middle goes to the lower neighbour ...
    tie = a == middle[low.clamp(max=len(middle) - 1)]
    low = torch.where(tie & (low % 2 == 1), low + 1, low)  # ... unless that has an odd code
    return (torch.sign(v) * grid[low.clamp(max=len(grid) - 1)] * unit).flatten(-2)[..., :n]


def _router_exact(s):
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    v = s["logits"].double().clone().requires_grad_(c["grad"])
    closed = torch.isinf(v.detach())
    empty = closed.all(1, keepdim=True)
    with torch.set_grad_enabled(c["grad"]):
        if c["score"] == "sigmoid":
            score = torch.sigmoid(v)
        else:
            score = torch.softmax(v.masked_fill(empty, 0.0), 1)
    sel = score.detach() + (s["bias"].double() if s["bias"] is not None else 0.0)
    sel = sel.masked_fill(closed, -math.inf)
    if c["topk_groups"] < G:
        part = sel.view(T, G, E // G)
        total, rest = torch.zeros(T, G, dtype=torch.float64, device=v.device), part.clone()
        for _ in range(c["group_top"]):
            best = rest.max(2)
            total = total + best.values
            rest.scatter_(2, best.indices.unsqueeze(2), -math.inf)
        off = torch.ones(T, G, dtype=torch.bool, device=v.device)
        for _ in range(c["topk_groups"]):
            hi = total.masked_fill(~off, -math.inf).amax(1, keepdim=True)
            first = ((total == hi) & off).to(torch.int8).argmax(1, keepdim=True)
            off.scatter_(1, first, False)
        sel = part.masked_fill(off.unsqueeze(2), -math.inf).view(T, E)
    picks = []
    for _ in range(K):
        hi = sel.amax(1, keepdim=True)
        first = (sel == hi).to(torch.int8).argmax(1, keepdim=True)
        picks.append(torch.where(hi > -math.inf, first, -1))
        sel = sel.scatter(1, first, -math.inf)
    ids = torch.cat(picks, 1)
    live = ids >= 0
    with torch.set_grad_enabled(c["grad"]):
        chosen = score.gather(1, ids.clamp(min=0)) * live
        gates = chosen
        if c["renormalize"]:
            gates = chosen / torch.where(live.any(1, keepdim=True), chosen.sum(1, keepdim=True), 1.0)
        gates = c["scale"] * gates
        out = {"weights": gates.detach(), "ids": None}
        if c["grad"]:
            d, = torch.autograd.grad((gates * s["d_weights"].double()).sum(), v)
            out["d_logits"] = torch.where(torch.isfinite(d), d, 0.0)
    return out


def _ffn_exact(s):
    c, ids = s["case"], s["ids"].long()
    T, H, I, E, K = (c[k] for k in "THIEK")
    x = _mx64(s["x"].double(), c["act"])
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for e in range(E):
        token, k = (ids == e).nonzero(as_tuple=True)
        if len(token):
            h = x[token] @ s["up"][e].double()
            act = _mx64(torch.nn.functional.silu(h[:, :I]) * h[:, I:], c["act"])
            y.index_add_(0, token, s["gates"][token, k].double().unsqueeze(1)
                         * (act @ s["down"][e].double()))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "router":
        return _router_exact(s)
    if case["op"] == "ffn":
        return _ffn_exact(s)
    return torch.stack([_mx64(w.double().t(), "mxfp4").t() for w in s["w"]])
