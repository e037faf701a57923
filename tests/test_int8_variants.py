"""The int8 operators where the other tests do not take them: every tile over many turns of
its stages, tiles that the XCDs take in turns, weights read past the caches in every
tile, long rows and many routes of one token.  References and tolerances as in
test_int8.py; the large ones take their exact sums from products in 64 bits on the GPU.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib
from test_blockscale import buckets
from test_int8 import bf16, gpu_of, make_codes, make_experts, make_scales, product, run_matmul, silu64
from test_int8_memory import INVALID, P, changed, refused

gpu = pytest.mark.gpu
DEV = "cuda:0"


def test_outputs_of_the_product_are_aligned():
    """Rows of y may begin at any element, y itself does not."""
    f = lib.lib().moe_int8_matmul
    args = (P, 256, P, 3, P, P, 64, 256, P, 0, 64, None, 0, None)
    for dtype, offsets in ((0, (4, 8, 12)), (1, (2, 4, 8, 14))):
        for o in offsets:
            refused(f(*changed(args, _8=P + o, _9=dtype)), INVALID, "y is not 16-byte aligned")


def exact_product(xq, xs, wq, ws):
    """test_int8.product on the GPU: whole numbers below 2^53 in 64 bits, then the three fp32 roundings."""
    s = xq.double() @ wq.double().t().contiguous()
    return (s.float() * xs[:, None]) * ws[None, :]


# the tiles of 64 x 32, 64 x 64, 64 x 128, 128 x 128 (one and two blocks a CU) and 256 x 256, with 8 to 37 K blocks and a
# remainder of 16 inputs
@gpu
@pytest.mark.parametrize("M,N,K", [(130, 2050, 1040), (700, 1300, 2320), (512, 3900, 2320), (450, 6100, 1040), (1500, 4090, 1040),
                                   (2500, 4100, 2320)])
def test_products_over_many_blocks(M, N, K):
    rng = np.random.default_rng(M + K)
    xq, xs, wq, ws = make_codes(rng, M, K), make_scales(rng, 1.0, M), make_codes(rng, N, K), make_scales(rng, 0.05, N)
    want = exact_product(*(gpu_of(a) for a in (xq, xs, wq, ws))).cpu()
    assert np.array_equal(want[:3].numpy(), product(xq[:3], xs[:3], wq, ws))
    y, _ = run_matmul(xq, xs, wq, ws, torch.float32)
    assert torch.equal(y.cpu(), want)
    y, _ = run_matmul(xq, xs, wq, ws, torch.bfloat16)
    assert torch.equal(y.cpu(), bf16(want.numpy()))


# rows of an expert on average, tile, what is looked at
GATEUP = [
    (1030, 4, 4, 592, 2064, False),    # 1030, 256 x 128: ten K blocks in three stages
    (8300, 8, 4, 208, 272, False),     # 4150, 256 x 128, the XCDs in turns
    (8300, 8, 4, 592, 272, True),      #       and with one expert in every route list
    (3400, 20, 2, 2160, 2064, True),   # 340, 256 x 128: the experts of fewer than 256 rows past the caches (178 MB)
    (5500, 100, 3, 272, 144, False),   # 165, 128 x 64, in turns
    (1248, 52, 3, 1600, 1040, False),  # 72, 128 x 64 past the caches (173 MB)
    (4100, 200, 2, 144, 80, False),    # 41, 64 x 64, in turns
    (24, 64, 4, 1312, 1040, False),    # 1.5, 64 x 64 past the caches (175 MB)
    (30, 1024, 16, 48, 48, False),     # as many experts and routes as there may be
    (1, 1024, 16, 144, 48, False),
]


@gpu
@pytest.mark.parametrize("T,E,k,d,f,crowd", GATEUP)
def test_gateup_in_every_tile(T, E, k, d, f, crowd):
    rng = np.random.default_rng(T + E + d)
    offsets, perm, _ = buckets(make_experts(rng, T, E, k, d, f, crowd), E)
    R, used = T * k, int(offsets[-1])
    xq, xs = gpu_of(make_codes(rng, T, d)), gpu_of(make_scales(rng, 1.0, T))
    wg, wu = (gpu_of(make_codes(rng, E, f, d)) for _ in range(2))
    sg, su = (gpu_of(make_scales(rng, 0.05, E, f)) for _ in range(2))
    perm = perm.to(DEV)
    for dtype in (torch.float32, torch.bfloat16):
        h = torch.full((R, f), 5.0, dtype=dtype, device=DEV)
        lib.int8_gateup(xq, xs, k, offsets.to(DEV), perm, wg, sg, wu, su, h)
        torch.cuda.synchronize()
        assert (h[used:] == 5.0).all()
        for e in range(E):
            a, b = int(offsets[e]), int(offsets[e + 1])
            if a == b:
                continue
            t = (perm[a:b] // k).long()
            g, u = (exact_product(xq[t], xs[t], w[e], s[e]).double().cpu().numpy() for w, s in ((wg, sg), (wu, su)))
            want = silu64(g) * u
            tol = np.abs(want) * (2 * np.abs(g) + 8) * 2.0 ** -24 + np.abs(g * u) * 2.0 ** -125
            if dtype == torch.bfloat16:
                tol = tol * 1.01 + np.abs(want) * 2.0 ** -8
            assert (np.abs(h[a:b].double().cpu().numpy() - want) <= tol).all(), e


DOWN = [
    (4200, 2, 2, 4112, 656, False),    # 4200, 256 x 256: six K blocks in two stages
    (8300, 8, 4, 592, 272, False),     # 4150, 256 x 256, the XCDs in turns
    (2600, 20, 2, 4112, 2064, True),   # 260, 256 x 256: the experts of fewer than 256 rows past the caches (170 MB)
    (5500, 100, 3, 272, 144, False),   # 165, 128 x 128, in turns
    (2250, 52, 3, 2064, 1600, True),   # 130, 128 x 128: the experts of fewer than 128 rows past the caches (172 MB)
    (4100, 200, 2, 144, 80, False),    # 41, 64 x 128 on two waves, in turns
    (520, 52, 3, 2064, 1600, False),   # 30, 64 x 128 on two waves, past the caches
    (2050, 600, 4, 144, 80, False),    # 14, 64 x 128 on eight waves, in turns
    (24, 64, 4, 2064, 1312, False),    # 1.5, 64 x 128 on eight waves, past the caches (173 MB)
    (30, 1024, 16, 48, 48, False),
] + [(T, E, k, 48, f, False)           # one and two tokens: runs of 128 inputs over 16 waves, six routes at a time
     for T in (1, 2) for E, k, f in ((20, 6, 2048), (20, 7, 2064), (16, 16, 2048), (20, 16, 4112), (24, 5, 16384), (1024, 16, 272),
                                     (16, 16, 128), (18, 13, 1040))]


@gpu
@pytest.mark.parametrize("T,E,k,d,f,crowd", DOWN)
def test_down_in_every_tile(T, E, k, d, f, crowd):
    rng = np.random.default_rng(T + E + f)
    idx = make_experts(rng, T, E, k, d, f, crowd)
    if T == 1 and k > 2:
        idx[0, [1, k - 1]] = -1                # routes without an expert
    offsets, _, pos = buckets(idx, E)
    R = T * k
    hq, hs = gpu_of(make_codes(rng, R, f)), gpu_of(make_scales(rng, 1.0, R))
    wd, sd = gpu_of(make_codes(rng, E, d, f)), gpu_of(make_scales(rng, 0.05, E, d))
    wt = gpu_of(rng.random((T, k)).astype(np.float32))
    ye = torch.zeros(R + 1, d, dtype=torch.float64, device=DEV)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            ye[a:b] = exact_product(hq[a:b], hs[a:b], wd[e], sd[e]).double()
    terms = ye[pos.to(DEV).long()].view(T, k, d) * wt.double()[:, :, None]
    add = gpu_of(rng.standard_normal((T, d)).astype(np.float32))
    need = lib.int8_down_workspace_bytes(T, k, d)
    work = torch.full((need,), 0x7f, dtype=torch.uint8, device=DEV) if need else None
    for a in (None, add):
        y = torch.full((T, d), 5.0, device=DEV)
        lib.int8_down(hq, hs, wt, offsets.to(DEV), pos.to(DEV), wd, sd, y, work, add=a)
        more = 0.0 if a is None else a.double()
        want, mags = terms.sum(1) + more, terms.abs().sum(1) + (0.0 if a is None else a.double().abs())
        assert ((y.double() - want).abs() <= (k + 1) * 2.0 ** -24 * mags).all()
