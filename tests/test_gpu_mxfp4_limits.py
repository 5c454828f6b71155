"""The MXFP4 forward at sizes next to its limits."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import operators as ops
from test_gpu_mxfp4 import check, make

pytestmark = pytest.mark.gpu


def as_f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("T", [3, 30, 60])
def test_codes_of_an_expert_past_2_gib(gpu_lib, T, act):
    """One expert of 17 * 2^20 columns a panel, all zero but 32 pieces of 64 columns, half of them
    past 2 GiB of codes: zeros add nothing and round nothing, so y is that of the pieces alone, with
    the same number of matrix instructions.  3, 30 and 60 rows take tiles of 32, 64 and 128."""
    m = gpu_lib
    H, I, P = 8, 17 << 20, 32
    say(f"[mxfp4] ffn {(T, H, I, 1, 1)} {act}")
    rng = np.random.default_rng(T)
    past = (1 << 31) // (2 * 1024) * 32 - I  # first column whose second panel lies past 2 GiB
    first = np.concatenate([[0, I - 64], rng.choice(past // 64, P // 2 - 1, replace=False)[1:] * 64,
                            past + rng.choice((I - past) // 64 - 1, P // 2, replace=False) * 64])
    first = np.unique(first)
    cols = torch.from_numpy((first[:, None] + np.arange(64)).reshape(-1)).cuda()
    n = len(cols)
    small_up = torch.from_numpy(rng.standard_normal((1, H, 2 * n)).astype(np.float32)).bfloat16()
    small_down = torch.from_numpy((rng.standard_normal((1, n, H)) / 40).astype(np.float32)).bfloat16()
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    ids, gates = np.zeros((T, 1), np.int32), np.ones((T, 1), np.float32)

    up = torch.zeros(1, H, 2 * I, dtype=torch.bfloat16, device="cuda")
    up[:, :, cols] = small_up[:, :, :n].cuda()
    up[:, :, I + cols] = small_up[:, :, n:].cuda()
    down = torch.zeros(1, I, H, dtype=torch.bfloat16, device="cuda")
    down[:, cols] = small_down.cuda()
    pu, pd = m.moe_ffn_mxfp4_quantize(up, panels=2), m.moe_ffn_mxfp4_quantize(down)
    assert pu.data.numel() > (1 << 31)
    del up, down
    y = m.moe_ffn_mxfp4_fwd(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(gates).cuda(),
                            pu, pd, act=act)
    torch.cuda.synchronize()
    ref, tol = ops.mxfp4_ffn(as_f64(x), ids, gates, as_f64(small_up), as_f64(small_down), act)
    assert (np.abs(as_f64(y) - ref) <= tol).all()
    assert np.abs(ref).max() > 0.5


@pytest.mark.parametrize("T,H,E", [(530000, 8192, 2), (17000, 262144, 1000)], ids=str)
def test_quantised_tokens_past_2_gib(gpu_lib, T, H, E):
    """The last tokens equal the same tokens in a call of their own; tiles of 128 and of 32 rows."""
    m = gpu_lib
    I = 8
    say(f"[mxfp4] ffn {(T, H, I, E, 1)}")
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    gates = torch.rand(T, 1, generator=g, device="cuda") + 0.5
    up = torch.empty(E, H, 2 * I, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    up /= H ** 0.5
    down = torch.empty(E, I, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    pu, pd = m.moe_ffn_mxfp4_quantize(up, panels=2), m.moe_ffn_mxfp4_quantize(down)
    y = m.moe_ffn_mxfp4_fwd(x, ids, gates, pu, pd)
    for at in (0, T - 300):
        sl = slice(at, at + 300)
        small = m.moe_ffn_mxfp4_fwd(x[sl].contiguous(), ids[sl].contiguous(),
                                    gates[sl].contiguous(), pu, pd).float()
        # sums may be taken in another order there, so an act value next to a border may differ:
        # by a quarter of itself at most, and few do
        d = (y[sl].float() - small).norm() / small.norm()
        assert d.item() < 0.05, d.item()


@pytest.mark.parametrize("act", ["mxfp4", "mxfp6"])
@pytest.mark.parametrize("shape", [
    (250, 1000, 520, 6, 1), (470, 520, 1000, 1, 1), (490, 520, 1000, 1, 1),  # 448, 512 and 544
    (333, 1000, 264, 9, 3), (1410, 1000, 72, 3, 1), (1500, 72, 1000, 3, 1),  # 1312, 1536 and 1600
    (2000, 520, 264, 5, 2), (2100, 1064, 520, 7, 2), (1900, 1064, 520, 7, 2)], ids=str)
def test_sizes_next_to_the_limits_of_the_tile_heights(gpu_lib, shape, act):
    """Numbers of 32-row tiles on both sides of the limits (512 and 1536, by format)."""
    say(f"[mxfp4] ffn {shape} {act}")
    check(gpu_lib, make(*shape, seed=12), act)
