"""Products on either side of the rule that says how their weights are loaded (three quarters of a
tile's rows a group at the mean, or one tile in all): the same formula, whichever is taken."""

import pytest

from gpu_util import say
import test_gpu_grouped as grouped
import test_gpu_int8 as int8

pytestmark = pytest.mark.gpu

# rows, groups: one group of one tile and of two; tiles of 16, 32 (streamed) and 64 rows at the rule's border
ROWS = [(16, 1), (17, 1), (32, 1), (33, 1), (72, 3), (73, 3), (96, 4), (97, 4), (48, 3), (49, 3), (192, 4), (193, 4)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("Kd,N", [(520, 264), (200, 6008)])
@pytest.mark.parametrize("M,E", ROWS)
def test_int8(gpu_lib, M, E, Kd, N, out):
    say(f"[int8] policy {M}x{Kd}x{N}/{E} {out}")
    x, w = int8.make(M, Kd, N, E, "bf16", seed=4)
    int8.check(gpu_lib, x, w, int8.offsets(M, E, seed=4), out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Kd,N", [(520, 264), (264, 1032)])
@pytest.mark.parametrize("M,E", ROWS)
def test_grouped(gpu_lib, M, E, Kd, N, dtype):
    say(f"[grouped] policy {M}x{Kd}x{N}/{E} {dtype}")
    grouped.check(gpu_lib, grouped.make(M, Kd, N, E, dtype, False, grouped.spread(M, E, seed=4)), dtype, False)


@pytest.mark.parametrize("T,E,K", [(24, 4, 4), (25, 4, 4), (32, 1, 1), (33, 1, 1), (48, 4, 4), (49, 4, 4)])
def test_layer(gpu_lib, T, E, K):
    say(f"[int8] policy, layer {T} tokens, {E} experts, {K} slots")
    int8.check_layer(gpu_lib, int8.layer(T, 264, 200, E, K, seed=4))
    int8.check_layer(gpu_lib, int8.layer(T, 264, 4104, E, K, seed=4))
