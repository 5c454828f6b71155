"""int8 products whose row and column scales lie at the two ends of fp32: the product of the sum
and both scales is an ordinary number, whatever one of them times the sum would be.

The sum is exact and the product with the scales is held to three fp32 roundings (2^-24 each) and, below
fp32's smallest normal number, half of its smallest step."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import products as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134}  # half of the smallest step


def product(m, M, Kd, N, E, row, col, out, seed=0):
    """Codes of any size, scales of 2^row and 2^col times 1 to 2."""
    rng = np.random.default_rng([seed, M, Kd, N, E])
    codes = np.zeros((M, -(-Kd // 64) * 64), np.int8)
    codes[:, :Kd] = rng.integers(-127, 128, (M, Kd))
    codes[0, :Kd] = 127
    wc = rng.integers(-127, 128, (E, Kd, N)).astype(np.int8)
    wc[:, :, 0] = 127
    sx = ((1 + rng.random(M)) * 2.0 ** row).astype(np.float32)
    sw = ((1 + rng.random((E, N))) * 2.0 ** col).astype(np.float32)
    off = np.concatenate([[0], np.sort(rng.integers(0, M + 1, E - 1)), [M]]).astype(np.int32)
    w = m.moe_ffn_int8_pack(torch.from_numpy(wc).cuda(), torch.from_numpy(sw).cuda())
    x = m.Int8Rows(torch.from_numpy(codes).cuda(), torch.from_numpy(sx).cuda(), Kd, torch.float32)
    y = m.moe_ffn_int8_mm(x, w, torch.from_numpy(off).cuda(), out_dtype=DT[out])
    want = ref.int8_mm(codes[:, :Kd], sx.astype(np.float64), wc, sw.astype(np.float64), off)
    tol = 3 * (2.0 ** -24 * np.abs(want) + LEAST["f32"])
    tol = tol + HALF[out] * (np.abs(want) + tol) + LEAST[out]
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float(np.nanmax(err / tol)), int(np.isnan(err).sum()))


# streaming tiles and tiles of 64 and of 128 rows
SIZES = [(1, 1024, 136, 1), (90, 1032, 520, 5), (700, 1032, 2600, 1), (2300, 136, 4104, 3), (60, 72, 40, 65)]
# (row, col): the sum times the row's scale past the largest number, below the smallest normal one and to
# nothing, and the same with the column's; a product that is subnormal itself
SCALES = [(120, -130), (-140, 100), (-148, 126), (-130, 120), (126, -148), (100, -140), (-70, -75), (-140, -5), (0, 0)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("scales", SCALES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_scales_of_opposite_ends(gpu_lib, size, scales, out):
    say(f"[int8] scales {size} {scales} {out}")
    product(gpu_lib, *size, *scales, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_products_past_the_largest_number_are_infinite(gpu_lib, out):
    say(f"[int8] overflow {out}")
    w = gpu_lib.moe_ffn_int8_pack(torch.full((64, 8), 100, dtype=torch.int8, device="cuda"),
                                  torch.tensor([2.0 ** e for e in (100, 120, 0, -20, 0, 0, 0, 0)], device="cuda"))
    codes = torch.ones(3, 64, dtype=torch.int8, device="cuda")
    codes[1], codes[2] = -1, 0
    rows = gpu_lib.Int8Rows(codes, torch.full((3,), 2.0 ** 100, device="cuda"), 64, torch.float32)
    y = gpu_lib.moe_ffn_int8_mm(rows, w, out_dtype=DT[out])
    assert bool((y[0, :2] == float("inf")).all()) and bool((y[1, :2] == -float("inf")).all())
    assert bool(torch.isfinite(y[:2, 2:]).all()) and not y[2].any()


# tiles of 32, 64 and 128 rows
@pytest.mark.parametrize("shape", [(20, 264, 200, 3, 2), (900, 72, 1032, 2, 2), (1100, 2056, 264, 1, 1)], ids=str)
@pytest.mark.parametrize("e", [120, -118])
def test_layer_of_large_tokens_and_small_weights(gpu_lib, shape, e):
    """x times 2^e and the up projection times 2^-e: the same y as without, where no value or scale
    becomes subnormal (values below 2^-5 are left out for that)."""
    T, H, I, E, K = shape
    say(f"[int8] layer {shape} 2^{e}")
    rng = np.random.default_rng(list(shape))
    t = lambda a: torch.from_numpy(np.where(np.abs(a) < 2.0 ** -5, 0.0, a).astype(np.float32)).bfloat16()
    x, up = t(rng.standard_normal((T, H))), t(64 * rng.standard_normal((E, H, 2 * I)) / np.sqrt(H))
    down = gpu_lib.moe_ffn_int8_quantize(t(rng.standard_normal((E, I, H))).cuda())
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)).cuda()
    gates = torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda()
    y = [gpu_lib.moe_ffn_int8_fwd((x.float() * 2.0 ** s).bfloat16().cuda(), ids, gates,
                                  gpu_lib.moe_ffn_int8_quantize((up.float() * 2.0 ** -s).bfloat16().cuda(), panels=2),
                                  down) for s in (0, e)]
    assert bool(torch.isfinite(y[0]).all()) and torch.equal(y[0], y[1])
