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


@pytest.mark.gpu
def test_streams_of_another_device_are_refused():
    """A launch on another device's stream would read this device's memory from there."""
    dev = "cuda:0"

    class Elsewhere:  # (its handle is this device's default stream: the calls would run)
        cuda_stream = 0
        device_index = 1

    def f(*n):
        return torch.zeros(*n, device=dev)

    def u8(*n):
        return torch.zeros(*n, dtype=torch.uint8, device=dev)

    def i32(*n):
        return torch.zeros(*n, dtype=torch.int32, device=dev)

    g = lib.gate(8, 2, bias=f(8))
    w, x, z, idx, wt, y, y2 = f(8, 256), f(4, 256), f(4, 8), i32(4, 2), f(4, 2), f(4, 128), f(4, 256)
    xq, xs, hq, hs, offsets, perm, pos = u8(4, 256), f(4, 2), u8(8, 128), f(8, 1), i32(9), i32(8), i32(8)
    wg, sg, wd, sd = u8(8, 128, 256), f(8, 1, 2), u8(8, 256, 128), f(8, 2, 1)
    work = u8(lib.blockscale_down_workspace_bytes(4, 2, 256))
    calls = [
        lambda s: lib.router_logits(w, x, z, stream=s),
        lambda s: lib.gate_topk(g, z, idx, wt, stream=s),
        lambda s: lib.blockscale_quantize(x, xq, xs, stream=s),
        lambda s: lib.blockscale_matmul(xq, xs, wg[0], sg[0], y, stream=s),
        lambda s: lib.blockscale_gateup(xq, xs, 2, offsets, perm, wg, sg, wg, sg, hq, hs, stream=s),
        lambda s: lib.blockscale_down(hq, hs, wt, offsets, pos, wd, sd, y2, work, stream=s),
    ]
    side = torch.cuda.Stream()
    for call in calls:
        torch.cuda.synchronize()
        with pytest.raises(ValueError, match="current device, cuda:0"):
            call(Elsewhere)
        call(side)
        torch.cuda.synchronize()
        call(None)
    torch.cuda.synchronize()


def test_largest_weight_is_taken():
    """65536 x 16384, every weight below 2^31 bytes: no limit besides those of N and K."""
    assert lib.blockscale_matmul_workspace_bytes(4, 65536, 16384) == 0
    for n, k in ((65537, 16384), (65536, 16400)):
        with pytest.raises(lib.MoeError, match="N 65537|K 16400"):
            lib.blockscale_matmul_workspace_bytes(4, n, k)


def test_workspaces_that_are_needed_and_not():
    """Few outputs of a long K take partial sums, the routed products of three tokens on their rows; else nothing."""
    P = 1 << 40  # a pointer that is never dereferenced: every call below is refused
    L = lib.lib()
    for M, N, K in ((64, 64, 16384), (300, 128, 16384), (33, 1, 4096)):
        need = lib.blockscale_matmul_workspace_bytes(M, N, K)
        assert need > 0 and need % (4 * M * N) == 0
        args = (P, K, P, M, P, P, N, K, P, 0, N)
        assert L.moe_blockscale_matmul(*args, P, need - 1, None) == lib.MOE_ERR_WORKSPACE
        assert L.moe_blockscale_matmul(*args, None, need, None) == lib.MOE_ERR_INVALID_ARG
    for M, N, K in ((1, 64, 16384), (32, 64, 16384), (64, 64, 3968), (4096, 4096, 16384)):
        assert lib.blockscale_matmul_workspace_bytes(M, N, K) == 0
    for T in (1, 2):
        assert lib.blockscale_down_workspace_bytes(T, 6, 4096) == 0
    need = lib.blockscale_down_workspace_bytes(3, 2, 256)
    assert need == 3 * 2 * 256 * 4
    args = (P, P, 3, 2, P, P, P, 8, P, P, 256, 256, None, P)
    assert L.moe_blockscale_down(*args, P, need - 1, None) == lib.MOE_ERR_WORKSPACE
    assert L.moe_blockscale_down(*args, None, need, None) == lib.MOE_ERR_INVALID_ARG
