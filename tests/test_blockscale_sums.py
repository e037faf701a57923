"""Block-scaled products of rows in which large products cancel.

Each run of 8 inputs holds one pair of +-448 * 448 that cancels, beside products
of small whole numbers.  Every partial sum, in whatever order, is a whole number
below 2^23, so sums held in 32 bits make no error at all: fp32 outputs are the
exact numbers, bf16 outputs those rounded once.  Nothing is left to a tolerance.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib
from test_blockscale import DEV, F8, buckets, nb, up

gpu = pytest.mark.gpu


def cancelling(rng, shape, both):
    """(codes, the small part): codes of whole numbers in [-3, 3] with a pair of 448s in each run of 8
    columns, of opposite signs in one operand (`both` false) and of one sign per row in the other."""
    small = rng.integers(-3, 4, shape).astype(np.float32)
    runs = np.arange(0, shape[-1], 8)
    at = runs + runs // 8 % 7
    sign = np.where(rng.random(shape[:-1] + (1,)) < 0.5, -1.0, 1.0).astype(np.float32) if both else np.float32(1)
    small[..., at] = small[..., at + 1] = 0.0
    whole = small.copy()
    whole[..., at] = 448.0 * sign
    whole[..., at + 1] = 448.0 * sign if both else -448.0
    return torch.from_numpy(whole).to(F8), torch.from_numpy(small)


@gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 70, 1024), (9, 300, 4112), (30, 300, 1040), (32, 6200, 1024), (33, 520, 1552),
                                   (64, 129, 16384), (100, 300, 8192), (300, 1024, 4096), (530, 4100, 1296),
                                   (1000, 1100, 2064), (1100, 4100, 1040), (2090, 4100, 1040), (4097, 2050, 2064),
                                   (3500, 3900, 1024)])
def test_matmul_keeps_what_is_left_of_cancelling_products(M, N, K, out):
    rng = np.random.default_rng(M + N + K)
    (xq, x), (wq, w) = cancelling(rng, (M, K), True), cancelling(rng, (N, K), False)
    y = torch.empty(M, N, dtype=out, device=DEV)
    work = torch.empty(max(16, lib.blockscale_matmul_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    lib.blockscale_matmul(up(xq), torch.ones(M, nb(K), device=DEV), up(wq), torch.ones(nb(N), nb(K), device=DEV), y, work)
    want = x @ w.t()  # (whole numbers below 2^24: exact in fp32)
    assert torch.equal(y.cpu(), want.to(out))


@gpu
@pytest.mark.parametrize("T,k,E", [(1, 3, 4), (2, 2, 3), (8, 4, 40), (60, 3, 20), (500, 4, 60), (700, 2, 5)])
def test_down_keeps_what_is_left_of_cancelling_products(T, k, E):
    d, f = 272, 1040
    rng = np.random.default_rng(T + k + E)
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32))
    offsets, perm, pos = buckets(idx, E)
    (hq, h), (wq, w) = cancelling(rng, (T * k, f), True), cancelling(rng, (E, d, f), False)
    y = torch.empty(T, d, device=DEV)
    work = torch.empty(max(16, lib.blockscale_down_workspace_bytes(T, k, d)), dtype=torch.uint8, device=DEV)
    lib.blockscale_down(up(hq), torch.ones(T * k, nb(f), device=DEV), torch.ones(T, k, device=DEV), up(offsets), up(pos),
                        up(wq), torch.ones(E, nb(d), nb(f), device=DEV), y, work)
    ye = torch.cat([h[int(offsets[e]): int(offsets[e + 1])] @ w[e].t() for e in range(E)])
    assert torch.equal(y.cpu(), ye[pos.long()].view(T, k, d).sum(1))
