"""Tensors that a kernel could not read are refused before anything is launched."""
import pytest
import torch

from quantized_moe_amd import blockscale, lib


def test_gate_refuses_a_bias_in_host_memory():
    """The kernel reads the bias through the address in the description: nothing after gate() sees the tensor."""
    with pytest.raises(ValueError, match="GPU memory"):
        lib.gate(8, 2, bias=torch.zeros(8))


class _NoStream:
    cuda_stream = None


def test_router_logits_refuses_host_memory():
    w, x, z = torch.zeros(8, 256), torch.zeros(3, 256), torch.zeros(3, 8)
    with pytest.raises(ValueError, match="GPU memory"):
        lib.router_logits(w, x, z, stream=_NoStream)


def test_layer_refuses_host_memory():
    def pair(n, k):
        q, s = blockscale.quantize_weight(torch.ones(8, n, k))
        return q, s

    layer = blockscale.BlockScaleLayer(torch.zeros(8, 256), lib.gate(8, 2), pair(128, 256), pair(128, 256), pair(256, 128),
                                       max_tokens=4)
    with pytest.raises(ValueError, match="GPU memory"):
        layer.forward(torch.zeros(3, 256), torch.zeros(3, 256), stream=_NoStream)
