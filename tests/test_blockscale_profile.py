"""Every launch of the gate and block-scaled operators is timed under a name of its own."""
import pytest
import torch

from quantized_moe_amd import lib
from test_blockscale import DEV, nb

gpu = pytest.mark.gpu


def names_of(call):
    lib.profile_reset()
    lib.profile_enable(True)
    try:
        call()
        torch.cuda.synchronize()
        got = lib.profile_collect()
    finally:
        lib.profile_enable(False)
        lib.profile_reset()
    return got


@gpu
@pytest.mark.parametrize("M,N,K,want", [(1, 64, 256, ["bs_matmul"]), (300, 640, 1040, ["bs_matmul"]),
                                        (70, 500, 8208, ["bs_matmul", "bs_matmul_sum"])])
def test_matmul_launches(M, N, K, want):
    need = lib.blockscale_matmul_workspace_bytes(M, N, K)
    assert (need > 0) == (len(want) == 2)
    xq, wq = torch.zeros(M, K, dtype=torch.uint8, device=DEV), torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    xs, ws, y = torch.ones(M, nb(K), device=DEV), torch.ones(nb(N), nb(K), device=DEV), torch.empty(M, N, device=DEV)
    work = torch.empty(need, dtype=torch.uint8, device=DEV)
    call = lambda: lib.blockscale_matmul(xq, xs, wq, ws, y, work)  # noqa: E731
    call()
    got = names_of(call)
    assert sorted(got) == want
    assert all(n == 1 and ms > 0 for n, ms in got.values())
