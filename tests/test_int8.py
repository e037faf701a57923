"""int8 operators against exact arithmetic on the CPU.

A product is a whole number's fp32 rounding times two scales, each product
rounded to fp32: the reference takes the sums in 64 bits, where they are exact
(at most 2^28), and then the same three roundings, so fp32 and bf16 outputs of the
dense product, and the codes and scales of the quantisation, have to be equal.
Tolerances, fixed before the first run:

* silu(g) = g / (1 + e^-g): the exponent's argument is rounded (|g| 2^-24 of e)
  after a constant that is (|g| 2^-24), exponential and reciprocal are off by a
  unit in the last place (2^-23 each), three roundings more and one for the
  product with u: (2 |g| + 8) 2^-24 of the value, and below the normal numbers
  |g u| 2^-125; bf16 outputs 2^-8 of the value more;
* a token's sum of k products is k multiply-adds: (k + 1) 2^-24 of the sum of
  magnitudes.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib
from test_blockscale import buckets

gpu = pytest.mark.gpu
DEV = "cuda:0"
F32 = np.float32


def make_codes(rng, *shape):
    """int8 codes of normal values, with zeros and the extremes (-128 too) among them."""
    q = np.clip(np.rint(rng.standard_normal(shape) * 35), -127, 127).astype(np.int8)
    flat = q.reshape(-1)
    for code in (0, -128, 127, -1):
        flat[rng.integers(0, flat.size, max(1, flat.size // 64))] = code
    return q


def make_scales(rng, rms, *shape):
    return (rms / 35 * np.exp(0.5 * rng.standard_normal(shape))).astype(F32)


def product(xq, xs, wq, ws):
    """The definition: fp32 of the exact sum, times the row's and the output's scale in fp32."""
    s = xq.astype(np.float64) @ wq.astype(np.float64).T
    return (s.astype(F32) * xs[:, None]) * ws[None, :]


def bf16(a):
    return torch.from_numpy(a).to(torch.bfloat16)


def gpu_of(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---------------------------------------------------------------- quantize ----
def quantize(x):
    s = (np.maximum(np.abs(x).max(1), F32(2.0 ** -100)) / F32(127)).astype(F32)
    return np.rint(x / s[:, None]).astype(np.int8), s


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 144), (6, 256), (7, 272), (64, 1040), (9, 2048), (33, 4096), (17, 4112), (5, 8208),
                                 (3, 16384)])
def test_quantize_is_exact(M, K, dtype):
    rng = np.random.default_rng(M * K)
    x = torch.from_numpy((rng.standard_normal((M, K)) * np.exp(2 * rng.standard_normal((M, 1)))).astype(F32)).to(dtype)
    if M > 2:
        x[1] = 0.0                       # a row of zeros
        x[2] = x[2] * 2.0 ** -115        # below the smallest scale's range
    ld, ldq = K + 32, K + 16
    xg = torch.full((M, ld), 7.0, dtype=dtype, device=DEV)[:, :K]
    xg.copy_(x)
    q = torch.full((M, ldq), 0x55, dtype=torch.int8, device=DEV)
    s = torch.full((M,), -1.0, device=DEV)
    lib.int8_quantize(xg, q[:, :K], s)
    want_q, want_s = quantize(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q[:, :K].cpu().numpy(), want_q)
    assert (q[:, K:] == 0x55).all()


@gpu
def test_quantize_ties_and_far_exponents():
    """Quotients half way between two codes, and rows at every power of two."""
    K = 512
    half = torch.arange(-127, 127, dtype=torch.float32) + 0.5
    rows = []
    for e in range(-126, 121, 3):
        row = torch.zeros(K)
        row[:254] = half * 2.0 ** e
        row[254:508] = torch.from_numpy(np.nextafter(half.numpy() * F32(2.0 ** e), F32(0)))
        row[511] = 127 * 2.0 ** e        # the scale is 2^e (from 2^-100 / 127 on)
        rows.append(row)
    x = torch.stack(rows)
    q, s = torch.empty(x.shape, dtype=torch.int8, device=DEV), torch.empty(len(rows), device=DEV)
    lib.int8_quantize(x.to(DEV), q, s)
    want_q, want_s = quantize(x.numpy())
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("K", [16, 1024, 8192])
def test_quantize_rows_that_are_not_numbers(K, bad, dtype):
    x = torch.ones(5, K, dtype=dtype)
    x[1, 0], x[3, K - 1] = bad, bad
    q, s = torch.empty(5, K, dtype=torch.int8, device=DEV), torch.empty(5, device=DEV)
    lib.int8_quantize(x.to(DEV), q, s)
    assert torch.isnan(s.cpu()).tolist() == [False, True, False, True, False]
    assert (q[[1, 3]] == 0).all() and (q[[0, 2, 4]] == 127).all()


# ------------------------------------------------------------------ matmul ----
def run_matmul(xq, xs, wq, ws, dtype, ldx=None, ldy=None, offset=0):
    M, K = xq.shape
    N = wq.shape[0]
    x = torch.full((M, ldx or K), 99, dtype=torch.int8, device=DEV)[:, :K]
    x.copy_(torch.from_numpy(xq))
    ybuf = torch.full((M * (ldy or N) + 64 + offset,), 3.0, dtype=dtype, device=DEV)
    y = ybuf[offset: offset + M * (ldy or N)].view(M, ldy or N)[:, :N]
    need = lib.int8_matmul_workspace_bytes(M, N, K)
    work = torch.full((need,), 0x7f, dtype=torch.uint8, device=DEV) if need else None
    lib.int8_matmul(x, gpu_of(xs), gpu_of(wq), gpu_of(ws), y, work)
    torch.cuda.synchronize()
    return y, ybuf


SHAPES = [(1, 1, 16), (1, 17, 144), (3, 70, 272), (16, 64, 1040), (17, 33, 528), (32, 100, 4112), (33, 65, 48), (64, 64, 128),
          (65, 130, 400), (100, 300, 8192), (250, 1000, 4112), (257, 259, 144), (300, 640, 1040), (1000, 1100, 2064),
          (700, 2500, 656), (1025, 1030, 80), (2048, 2050, 272), (4100, 3100, 208), (1, 4096, 4096), (24, 6200, 1040),
          (33, 250, 16384), (5, 70, 8208), (128, 4100, 272), (130, 2050, 144), (256, 4000, 144), (250, 5000, 80), (512, 3900, 208),
          (450, 6100, 144), (1000, 3900, 144), (1024, 4096, 4096), (1500, 4090, 272), (2500, 4100, 144), (4090, 4090, 144)]


@gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_is_exact(M, N, K):
    rng = np.random.default_rng(M + N + K)
    xq, xs, wq, ws = make_codes(rng, M, K), make_scales(rng, 1.0, M), make_codes(rng, N, K), make_scales(rng, 0.05, N)
    want = product(xq, xs, wq, ws)
    y, _ = run_matmul(xq, xs, wq, ws, torch.float32)
    assert np.array_equal(y.cpu().numpy(), want)
    y, _ = run_matmul(xq, xs, wq, ws, torch.bfloat16)
    assert torch.equal(y.cpu(), bf16(want))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(2, 30, 272), (20, 66, 144), (70, 129, 400), (300, 640, 1040), (450, 6100, 144), (1000, 3900, 144), (2050, 2050, 144), (4090, 4090, 144)])
def test_matmul_strides_and_what_lies_beside(M, N, K, dtype):
    """Rows of x and y further apart, y at an address of its element only: nothing beside the outputs is written."""
    rng = np.random.default_rng(M)
    xq, xs, wq, ws = make_codes(rng, M, K), make_scales(rng, 1.0, M), make_codes(rng, N, K), make_scales(rng, 0.05, N)
    want = torch.from_numpy(product(xq, xs, wq, ws)).to(dtype)
    for ldy in (N + 4, N + 3, -(-N // 8) * 8 + 8, -(-N // 8) * 8 + 4, -(-N // 8) * 8 + 2):  # every alignment of a row
        y, ybuf = run_matmul(xq, xs, wq, ws, dtype, ldx=K + 48, ldy=ldy)
        assert torch.equal(y.cpu(), want)
        y.fill_(3.0)
        assert (ybuf == 3.0).all()


@gpu
@pytest.mark.parametrize("M,N", [(1, 64), (32, 64), (64, 128), (300, 300), (1100, 1100), (2100, 2100)])
def test_matmul_largest_sums(M, N):
    """Every product 2^14: sums of 2^28, whole numbers past 2^24 that fp32 rounds."""
    K = 16384
    xq, wq = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
    xq[:, ::2], wq[:, 5] = 127, 3
    xq[0] = -128
    one_m, one_n = np.ones(M, F32), np.ones(N, F32)
    y, _ = run_matmul(xq, one_m, wq, one_n, torch.float32)
    row = (xq[:2].astype(np.int64) @ wq[:1].astype(np.int64).T)[:, 0].astype(F32)
    y = y.cpu().numpy()
    assert (y[0] == row[0]).all()
    if M > 1:
        assert (y[1:] == row[1]).all()


@gpu
@pytest.mark.parametrize("M,N,K", [(4, 40, 256), (40, 40, 256), (300, 300, 4096), (2048, 2048, 256)])
def test_matmul_scales_that_are_not_numbers(M, N, K):
    rng = np.random.default_rng(5)
    xq, xs, wq, ws = make_codes(rng, M, K), make_scales(rng, 1.0, M), make_codes(rng, N, K), make_scales(rng, 0.05, N)
    xs[M - 1], ws[3] = np.nan, np.inf
    wq[3] = 0                                  # 0 * inf
    y, _ = run_matmul(xq, xs, wq, ws, torch.float32)
    y = y.cpu().numpy()
    assert np.isnan(y[M - 1]).all() and np.isnan(y[:, 3]).all()
    y[M - 1], y[:, 3] = 0, 0
    assert np.isfinite(y).all()


# ----------------------------------------------------------------- experts ----
def make_experts(rng, T, E, k, d, f, crowd=False, holes=True):
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if not crowd else \
        np.stack([np.r_[0, 1 + rng.permutation(E - 1)[: k - 1]] for _ in range(T)]).astype(np.int32)
    if holes and T > 1:
        idx[rng.random((T, k)) < 0.1] = -1     # routes without an expert
        idx[T // 2] = -1                       # a token without any
    return torch.from_numpy(idx)


def silu64(g):
    return g / (1.0 + np.exp(-np.clip(g, -700, 700)))


EXPERTS = [(1, 8, 2, 64, 48), (1, 16, 6, 256, 272), (2, 4, 4, 144, 128), (3, 40, 5, 272, 144), (8, 64, 6, 512, 400), (60, 4, 2, 144, 272),
           (200, 8, 3, 256, 128), (130, 2, 2, 400, 528), (300, 3, 1, 128, 256), (700, 24, 4, 64, 80),
           (1030, 4, 4, 64, 2064), (1000, 3, 2, 2064, 64), (4200, 2, 2, 4112, 16), (2100, 8, 4, 80, 4000), (1200, 30, 4, 1040, 1040)]


@gpu
@pytest.mark.parametrize("crowd", [False, True])
@pytest.mark.parametrize("T,E,k,d,f", EXPERTS)
def test_gateup(T, E, k, d, f, crowd):
    rng = np.random.default_rng(T * E + d)
    idx = make_experts(rng, T, E, k, d, f, crowd)
    offsets, perm, _ = buckets(idx, E)
    R, used = T * k, int(offsets[-1])
    xq, xs = make_codes(rng, T, d), make_scales(rng, 1.0, T)
    wg, sg, wu, su = make_codes(rng, E, f, d), make_scales(rng, 0.05, E, f), make_codes(rng, E, f, d), make_scales(rng, 0.05, E, f)
    for dtype in (torch.float32, torch.bfloat16):
        h = torch.full((R, f), 5.0, dtype=dtype, device=DEV)
        lib.int8_gateup(gpu_of(xq), gpu_of(xs), k, offsets.to(DEV), perm.to(DEV), gpu_of(wg), gpu_of(sg), gpu_of(wu), gpu_of(su), h)
        torch.cuda.synchronize()
        got = h.float().cpu().numpy()
        assert (got[used:] == 5.0).all()
        for e in range(E):
            rows = slice(int(offsets[e]), int(offsets[e + 1]))
            t = perm[rows].numpy() // k
            g, u = product(xq[t], xs[t], wg[e], sg[e]).astype(np.float64), product(xq[t], xs[t], wu[e], su[e]).astype(np.float64)
            want = silu64(g) * u
            tol = np.abs(want) * (2 * np.abs(g) + 8) * 2.0 ** -24 + np.abs(g * u) * 2.0 ** -125
            if dtype == torch.bfloat16:
                tol = tol * 1.01 + np.abs(want) * 2.0 ** -8
            assert (np.abs(got[rows] - want) <= tol).all()


@gpu
@pytest.mark.parametrize("crowd", [False, True])
@pytest.mark.parametrize("T,E,k,d,f", EXPERTS)
def test_down(T, E, k, d, f, crowd):
    rng = np.random.default_rng(T * E + f)
    idx = make_experts(rng, T, E, k, d, f, crowd)
    offsets, perm, pos = buckets(idx, E)
    R = T * k
    hq, hs = make_codes(rng, R, f), make_scales(rng, 1.0, R)
    wd, sd = make_codes(rng, E, d, f), make_scales(rng, 0.05, E, d)
    wt = rng.random((T, k)).astype(F32)
    ye = np.zeros((R + 1, d), np.float64)
    for e in range(E):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        ye[rows] = product(hq[rows], hs[rows], wd[e], sd[e])
    terms = ye[pos.numpy()].reshape(T, k, d) * wt[:, :, None].astype(np.float64)
    add = rng.standard_normal((T, d)).astype(F32)
    need = lib.int8_down_workspace_bytes(T, k, d)
    work = torch.full((need,), 0x7f, dtype=torch.uint8, device=DEV) if need else None
    args = (gpu_of(hq), gpu_of(hs), gpu_of(wt), offsets.to(DEV), pos.to(DEV), gpu_of(wd), gpu_of(sd))
    for a in (None, add):
        y = torch.full((T, d), 5.0, device=DEV)
        lib.int8_down(*args, y, work, add=None if a is None else gpu_of(a))
        a64 = 0.0 if a is None else a.astype(np.float64)
        want, mags = terms.sum(1) + a64, np.abs(terms).sum(1) + np.abs(a64)
        assert (np.abs(y.cpu().numpy() - want) <= (k + 1) * 2.0 ** -24 * mags).all()
    y = gpu_of(add)
    lib.int8_down(*args, y, work, add=y)       # in place
    assert (np.abs(y.cpu().numpy() - want) <= (k + 1) * 2.0 ** -24 * mags).all()


@gpu
def test_rows_do_not_depend_on_the_batch():
    """A row's bits are the same alone and in any batch, for every way of computing it."""
    rng = np.random.default_rng(3)
    K, N = 1040, 1100
    xq, xs, wq, ws = make_codes(rng, 1500, K), make_scales(rng, 1.0, 1500), make_codes(rng, N, K), make_scales(rng, 0.05, N)
    full, _ = run_matmul(xq, xs, wq, ws, torch.float32)
    for M in (1, 16, 30, 40, 200, 700):
        y, _ = run_matmul(xq[:M], xs[:M], wq, ws, torch.float32)
        assert torch.equal(y, full[:M])
