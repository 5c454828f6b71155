"""What the autograd wrappers make of a gradient before the library sees it (no GPU needed)."""

import pytest
import torch

import mixture_experts_ffn_amd as m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", range(9))
def test_a_view_becomes_aligned(dtype, first):
    buffer = torch.arange(200).to(dtype)
    dy = buffer[first:first + 96].view(12, 8)
    got = m._own_gradient(dy)
    assert got.is_contiguous() and got.data_ptr() % 16 == 0 and torch.equal(got, dy)
    if dy.data_ptr() % 16 == 0:
        assert got.data_ptr() == dy.data_ptr()  # no copy that is not needed


def test_strided_broadcast_and_empty():
    wide = torch.randn(6, 24)
    for dy in (wide[:, 3:11], wide.t(), torch.ones(1).expand(6, 8), torch.randn(0, 8), wide[:0]):
        got = m._own_gradient(dy)
        assert got.is_contiguous() and got.data_ptr() % 16 == 0 and torch.equal(got, dy)


def test_what_a_concatenation_hands_out():
    """The views that this is for exist: contiguous, and off by the values in front."""
    y = torch.randn(4, 8, requires_grad=True)
    seen = []
    z = y * 1
    z.register_hook(seen.append)
    torch.cat([torch.ones(3, requires_grad=True), z.flatten()]).backward(torch.randn(35))
    assert seen[0].is_contiguous() and seen[0].data_ptr() % 16 == 12
