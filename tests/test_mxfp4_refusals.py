"""Calls of the MXFP4 forward that it cannot answer."""

import pytest
import torch

import mixture_experts_ffn_amd as m
from gpu_util import say


def call(device, x_grad, gate_grad, packed):
    x = torch.ones(4, 32, dtype=torch.bfloat16, device=device, requires_grad=x_grad)
    gates = torch.ones(4, 1, device=device, requires_grad=gate_grad)
    ids = torch.zeros(4, 1, dtype=torch.int32, device=device)
    return m.moe_ffn_mxfp4_fwd(x, ids, gates, *packed)


@pytest.mark.parametrize("x_grad,gate_grad", [(True, False), (False, True)])
def test_inputs_that_require_a_gradient(x_grad, gate_grad):
    """Refused before anything else is looked at; without gradients the CPU tensors are what is wrong."""
    w = m.MXFP4Weight(torch.zeros(16, dtype=torch.uint8), 1, 32, 32, 1, torch.bfloat16)
    with pytest.raises(m.MoEFFNError, match="no gradient") as ei:
        call("cpu", x_grad, gate_grad, (w, w))
    assert ei.value.status == 3
    with torch.no_grad(), pytest.raises(m.MoEFFNError) as ei:
        call("cpu", x_grad, gate_grad, (w, w))
    assert ei.value.status == 1


@pytest.mark.gpu
def test_inputs_that_require_a_gradient_on_the_gpu(gpu_lib):
    say("[mxfp4] inputs with gradients")
    packed = (m.moe_ffn_mxfp4_quantize(torch.ones(1, 32, 64, device="cuda"), panels=2),
              m.moe_ffn_mxfp4_quantize(torch.ones(1, 32, 32, device="cuda")))
    for grads in ((True, False), (False, True)):
        with pytest.raises(m.MoEFFNError):
            call("cuda", *grads, packed)
        for mode in (torch.no_grad, torch.inference_mode):
            with mode():
                y = call("cuda", *grads, packed)
            assert not y.requires_grad and (y > 0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.uint8, torch.float64, torch.float8_e4m3fn, None])
def test_packed_weights_of_another_dtype(dtype):
    """The dtype says what dequantisation writes: one that the library does not know is refused
    before any pointer is passed on (here: before the CPU tensor is)."""
    w = m.MXFP4Weight(torch.zeros(1 << 12, dtype=torch.uint8), 1, 32, 32, 1, dtype)
    for call_it in (lambda: m.moe_ffn_mxfp4_dequantize(w), lambda: w.nbytes):
        with pytest.raises(m.MoEFFNError) as ei:
            call_it()
        assert ei.value.status == 3
    for known in (torch.float32, torch.bfloat16):
        assert m.MXFP4Weight(None, 1, 128, 32, 1, known).nbytes == 128 * 32 // 2 + 256


def test_the_size_of_packed_weights_follows_their_sizes():
    """The forward compares it with what the buffer holds."""
    w = m.MXFP4Weight(None, 1, 128, 32, 1, torch.bfloat16)
    assert w.nbytes == 128 * 32 // 2 + 256
    w.E, w.N = 3, 64
    assert w.nbytes == 3 * 2 * (128 * 32 // 2 + 256)
    w.Kd = 12
    with pytest.raises(m.MoEFFNError):
        w.nbytes
