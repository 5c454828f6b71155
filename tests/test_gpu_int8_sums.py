"""The int8 layer's gate-weighted sum takes an expert's output rows as the fp32 numbers that the
down projection gives: the one rounding to bf16 is that of y.

An output may be off by half a step of bf16 (2^-8 of the value) and by what the reference derives for
the sums in fp32 and for act codes beside a tie; a rounding of the rows on the way would be another
2^-8 of their magnitudes, far above that where the slots cancel."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import products as ref

pytestmark = pytest.mark.gpu


def as_f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(m, x, ids, gates, up, down):
    y = as_f64(m.moe_ffn_int8_fwd(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(gates).cuda(),
                                  m.moe_ffn_int8_quantize(up.cuda(), panels=2),
                                  m.moe_ffn_int8_quantize(down.cuda())))
    want, tol = ref.int8_ffn(as_f64(x), ids, gates, as_f64(up), as_f64(down))
    err = np.abs(y - want)
    assert (err <= tol).all(), (float((err / tol).max()), float((err > tol).mean()))
    return want, tol


def tensors(rng, T, H, I, E):
    t = lambda a: torch.from_numpy(a.astype(np.float32)).bfloat16()
    return (t(rng.standard_normal((T, H))), t(rng.standard_normal((E, H, 2 * I)) / np.sqrt(H)),
            t(rng.standard_normal((E, I, H)) / np.sqrt(I)))


# tiles of 32, 64 and 128 rows, rows of the output that end inside a column tile
SHAPES = [(1, 256, 128, 4), (40, 264, 200, 3), (900, 72, 1032, 2), (1100, 2056, 264, 1), (4100, 2056, 40, 2)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_one_slot_is_rounded_once(gpu_lib, shape):
    T, H, I, E = shape
    say(f"[int8] one slot {shape}")
    rng = np.random.default_rng(list(shape))
    x, up, down = tensors(rng, T, H, I, E)
    ids = rng.integers(0, E, (T, 1)).astype(np.int32)
    gates = (0.3 + 0.6 * rng.random((T, 1))).astype(np.float32)
    check(gpu_lib, x, ids, gates, up, down)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_slots_that_cancel(gpu_lib, shape):
    """Two experts of one up projection, whose down projections differ by a step of bf16 in each
    column's largest value, and so by up to 1/128 in the columns' scales, with gates 1 and -1."""
    T, H, I, _ = shape
    say(f"[int8] slots that cancel {shape}")
    rng = np.random.default_rng([7, *shape])
    x, up, down = tensors(rng, T, H, I, 1)
    up = up.repeat(2, 1, 1)
    down = torch.cat([down, down])
    top = down[0].float().abs().amax(0)
    first = down[0].float().abs().argmax(0)
    step = 2.0 ** (torch.floor(torch.log2(top)) - 7)
    cols = torch.arange(H)
    down[1, first, cols] = (down[0, first, cols].float() + step * down[0, first, cols].float().sign()).bfloat16()
    ids = np.tile(np.array([[0, 1]], np.int32), (T, 1))
    gates = np.tile(np.array([[1.0, -1.0]], np.float32), (T, 1))
    want, tol = check(gpu_lib, x, ids, gates, up, down)
    # rows rounded to bf16 before the sum would be off by about 2^-9 of each: more than this bound
    one, _ = ref.int8_ffn(as_f64(x), ids[:, :1], gates[:, :1], as_f64(up), as_f64(down))
    assert np.median(tol) < 2.0 ** -10 * np.median(np.abs(one))


def test_rows_past_32_bit_offsets(gpu_lib):
    """Rows of 5.2 GB in all: the last tokens as by themselves, bit for bit (the integer sums are exact
    and the rest goes in one order, whatever the tiles)."""
    T, H, I, E, K = 80000, 2048, 32, 8, 8
    say(f"[int8] layer {T}x{H}x{I}/{E} top {K}")
    gen = torch.Generator("cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x = r(T, H).bfloat16()
    up = gpu_lib.moe_ffn_int8_quantize((r(E, H, 2 * I) / H ** 0.5).bfloat16(), panels=2)
    down = gpu_lib.moe_ffn_int8_quantize((r(E, I, H) / I ** 0.5).bfloat16())
    ids = torch.rand(T, E, generator=gen, device="cuda").argsort(1).int()
    gates = torch.rand(T, K, generator=gen, device="cuda")
    y = gpu_lib.moe_ffn_int8_fwd(x, ids, gates, up, down)
    for part in (slice(0, 50), slice(T // 2, T // 2 + 700), slice(T - 300, T)):
        alone = gpu_lib.moe_ffn_int8_fwd(x[part].contiguous(), ids[part].contiguous(), gates[part].contiguous(), up, down)
        assert torch.equal(y[part], alone) and alone.any()
