"""Gradients that are views into a larger buffer: contiguous, but not at a multiple of 16 bytes, as
the backward of a concatenation hands them out.  The same bits as from a gradient of its own."""

import pytest
import torch

from gpu_util import say, to_device
from synth import Workload, make_inputs

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def through_a_view(y, dy, leaves):
    """Gradients of sum(cat([a, y]) * c) for the leaves: y's gradient lies behind three values."""
    a = torch.ones(3, dtype=y.dtype, device=y.device, requires_grad=True)
    joined = torch.cat([a, y.flatten()])
    seen = []
    y.register_hook(lambda g: seen.append(g.data_ptr() % 16))
    grads = torch.autograd.grad(joined, leaves, torch.cat([torch.zeros_like(a), dy.flatten()]))
    assert seen and seen[0] != 0  # else the view was copied on the way, and nothing is tested
    return grads


@pytest.mark.parametrize("transposed", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [150, 3000])
def test_grouped_mm(gpu_lib, dtype, transposed, M):
    say(f"[grouped] gradient views {M} {dtype} transposed={transposed}")
    gen = torch.Generator("cuda").manual_seed(1)
    E, Kd, N = 4, 264, 200
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(DT[dtype])
    x, w, dy = r(M, Kd), r(*((E, N, Kd) if transposed else (E, Kd, N))), r(M, N)
    off = torch.tensor([0, M // 3, M // 3, M // 2, M - 5], device="cuda")
    x.requires_grad_(), w.requires_grad_()
    f = lambda: gpu_lib.moe_ffn_grouped_mm(x, w, off, transposed=transposed)
    want = torch.autograd.grad(f(), (x, w), dy)
    got = through_a_view(f(), dy, (x, w))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_layer(gpu_lib):
    say("[layer] gradient views")
    w = Workload("views", 40, T=130, H=256, I=128, E=4, K=2)
    d = to_device(make_inputs(w, with_dy=True))
    leaves = [d[k].requires_grad_() for k in ("x", "topk_weights", "up_proj", "down_proj")]
    f = lambda: gpu_lib.moe_ffn(d["x"], d["topk_ids"], d["topk_weights"], d["up_proj"], d["down_proj"])
    want = torch.autograd.grad(f(), leaves, d["dy"])
    got = through_a_view(f(), d["dy"], leaves)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_router(gpu_lib):
    say("[router] gradient views")
    gen = torch.Generator("cuda").manual_seed(2)
    logits = torch.randn(100, 24, generator=gen, device="cuda", requires_grad=True)
    dw = torch.randn(100, 3, generator=gen, device="cuda")
    f = lambda: gpu_lib.moe_ffn_router(logits, 3)[0]
    want, = torch.autograd.grad(f(), logits, dw)
    got, = through_a_view(f(), dw, (logits,))
    assert torch.equal(want, got)
