"""Block-scaled E4M3 operators against 64-bit arithmetic on the CPU.

Tolerances, fixed before the first run:

* a product's fp32 sum of K terms in any order errs by at most K 2^-24 of the
  sum of magnitudes; the operators sum 128 at a time and then one
  multiply-add per block, so (128 + KB + 4) 2^-23 bounds it with room for
  truncation inside the matrix unit (SUM below);
* silu adds its own few ulp and the exponent's argument error |g| 2^-22;
* E4M3 codes are off by half a step: 2^-4 of the value, or 2^-10 of the scale
  among the subnormals; bf16 outputs by 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib

gpu = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


def nb(n):
    return -(-n // 128)


def SUM(K):
    return (128 + nb(K) + 4) * 2.0 ** -23


# ------------------------------------------------------------ CPU reference ----
def make_rows(rng, M, K, rms=1.0):
    """Codes (uint8 E4M3) and per-row scales, with zeros, subnormals and the extremes among them."""
    v = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32) * 110).clamp(-448, 448).to(F8)
    flat = v.view(torch.uint8).view(-1)
    for code in (0x00, 0x80, 0x01, 0x7e, 0xfe):
        flat[rng.integers(0, flat.numel(), max(1, flat.numel() // 64))] = code
    s = torch.from_numpy((rms / 110 * np.exp(0.5 * rng.standard_normal((M, nb(K))))).astype(np.float32))
    return v, s


def make_weight(rng, N, K, E=None, rms=0.05):
    if E is None:
        v, _ = make_rows(rng, N, K)
        return v, torch.from_numpy((rms / 110 * np.exp(0.5 * rng.standard_normal((nb(N), nb(K))))).astype(np.float32))
    parts = [make_weight(rng, N, K, rms=rms) for _ in range(E)]
    return (torch.stack([p[0].view(torch.uint8) for p in parts]).view(F8), torch.stack([p[1] for p in parts]))


def values_rows(q, s):
    return q.to(torch.float64) * s.double().repeat_interleave(128, 1)[:, : q.shape[1]]


def values_weight(q, s):
    N, K = q.shape
    return q.to(torch.float64) * s.double().repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[:N]


def product(x, w):
    """(x w^T, the sums of magnitudes) in 64 bits."""
    return x @ w.t(), x.abs() @ w.abs().t()


def up(t):
    """To the GPU (float8 tensors move as bytes)."""
    return t.view(torch.uint8).to(DEV).view(F8) if t.dtype == F8 else t.to(DEV)


def down(t):
    return t.view(torch.uint8).cpu().view(F8) if t.dtype == F8 else t.cpu()


def buckets(idx, E):
    """offsets, perm, pos of the routes (entries outside [0, E) have no place)."""
    flat = idx.view(-1).tolist()
    order = sorted((r for r in range(len(flat)) if 0 <= flat[r] < E), key=lambda r: flat[r])
    offsets = [0] * (E + 1)
    for r in order:
        offsets[flat[r] + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    pos = [len(flat)] * len(flat)
    for p, r in enumerate(order):
        pos[r] = p
    perm = order + [0] * (len(flat) - len(order))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(perm, dtype=torch.int32),
            torch.tensor(pos, dtype=torch.int32))


# ---------------------------------------------------------------- quantize ----
@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (7, 400), (64, 1040), (33, 4096), (5, 16384), (300, 256)])
def test_quantize_is_exact(M, K, dtype):
    rng = np.random.default_rng(M * K)
    x = rng.standard_normal((M, K)).astype(np.float32) * np.exp(2 * rng.standard_normal((M, 1))).astype(np.float32)
    x = torch.from_numpy(x).to(dtype)
    x[0, :16] = 0.0                     # a run of zeros; with K = 16 a whole group
    if M > 2:
        x[1] = 0.0                      # rows of zeros
        x[2] *= 2.0 ** -120             # below the smallest scale's range
    ld, ldq = K + 32, K + 16
    xg = torch.full((M, ld), 7.0, dtype=dtype, device=DEV)[:, :K]
    xg.copy_(x)
    qbuf = torch.full((M, ldq), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.empty(M, nb(K), device=DEV)
    lib.blockscale_quantize(xg, qbuf[:, :K], s)
    torch.cuda.synchronize()
    xf = torch.nn.functional.pad(x.float(), (0, -K % 128)).view(M, -1, 128)
    amax = xf.abs().amax(2).numpy()
    s_ref = np.maximum(amax, np.float32(2.0 ** -100)) / np.float32(448)
    assert np.array_equal(s.cpu().numpy(), s_ref)
    q_ref = torch.from_numpy(xf.numpy() / s_ref[:, :, None]).view(M, -1)[:, :K].to(F8)
    assert torch.equal(qbuf[:, :K].cpu(), q_ref.view(torch.uint8))
    assert (qbuf[:, K:] == 0x55).all()


@gpu
@pytest.mark.parametrize("exponent", [-126, -100, -81, -79, -40, 0, 60, 120])
def test_quantize_divides_exactly(exponent):
    """Groups of every size of scale; many quotients, among them values half way between two codes."""
    rng = np.random.default_rng(exponent + 200)
    M, K = 512, 1024
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[: M // 2] = np.round(x[: M // 2] * 16) / 16 * 1.9375   # few significant bits: ties
    x = (x * np.float32(2.0) ** exponent).astype(np.float32)
    q, s = torch.empty(M, K, dtype=F8, device=DEV), torch.empty(M, nb(K), device=DEV)
    lib.blockscale_quantize(torch.from_numpy(x).to(DEV), q, s)
    b = x.reshape(M, -1, 128)
    s_ref = np.maximum(np.abs(b).max(2), np.float32(2.0 ** -100)) / np.float32(448)
    assert np.array_equal(s.cpu().numpy(), s_ref)
    q_ref = torch.from_numpy((b / s_ref[:, :, None]).reshape(M, K)).to(F8)
    assert torch.equal(down(q).view(torch.uint8), q_ref.view(torch.uint8))


@gpu
def test_quantize_non_finite_groups():
    x = torch.ones(4, 384)
    x[0, 5], x[1, 200], x[2, 300] = float("inf"), float("nan"), float("-inf")
    q, s = torch.empty(4, 384, dtype=F8, device=DEV), torch.empty(4, 3, device=DEV)
    lib.blockscale_quantize(x.to(DEV), q, s)
    s, q = s.cpu(), down(q).float()
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(torch.isnan(s), bad)
    assert (q.view(4, 3, 128)[bad] == 0).all() and (q.view(4, 3, 128)[~bad] == 448).all()


# ------------------------------------------------------------------ matmul ----
MATMUL = [(1, 16, 16), (1, 1, 128), (2, 300, 400), (1, 2048, 2064), (4, 129, 4096), (15, 257, 1040), (16, 128, 256),
          (17, 64, 144), (33, 1100, 528), (65, 127, 2064), (100, 640, 384), (130, 513, 1040), (257, 300, 272),
          (300, 1024, 4096), (520, 776, 656)]


@gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", MATMUL)
def test_matmul(M, N, K, out):
    rng = np.random.default_rng(M + 7 * N + 13 * K)
    (xq, xs), (wq, ws) = make_rows(rng, M, K), make_weight(rng, N, K)
    xbuf = torch.full((M, K + 48), 0x7f, dtype=torch.uint8, device=DEV)  # NaN codes in the gaps
    xbuf[:, :K] = xq.view(torch.uint8).to(DEV)
    ybuf = torch.full((M, N + 3), -5.0, dtype=out, device=DEV)
    work = torch.empty(max(16, lib.blockscale_matmul_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    lib.blockscale_matmul(xbuf[:, :K], up(xs), up(wq), up(ws), ybuf[:, :N], work)
    torch.cuda.synchronize()
    y = ybuf.cpu().double()
    ref, mag = product(values_rows(xq, xs), values_weight(wq, ws))
    tol = SUM(K) * mag + (2.0 ** -8 * ref.abs() if out == torch.bfloat16 else 0)
    assert ((y[:, :N] - ref).abs() <= tol).all(), float(((y[:, :N] - ref).abs() / tol.clamp(min=1e-300)).max())
    assert (y[:, N:] == -5.0).all()


@gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(2090, 4100, 1040), (4097, 2050, 2064), (700, 640, 4112), (4000, 4200, 1040),
                                   (700, 5000, 144), (1030, 2300, 1168), (530, 4100, 1296), (33, 520, 1552), (1800, 1900, 16),
                                   (3900, 3800, 272), (100, 300, 8192), (40, 129, 4112), (250, 1999, 4096), (33, 1, 16384)])
def test_matmul_many_tiles(M, N, K, out):
    """Several tiles of the largest kind in both directions, the last ones short."""
    rng = np.random.default_rng(M + N)
    (xq, xs), (wq, ws) = make_rows(rng, M, K), make_weight(rng, N, K)
    y = torch.empty(M, N, dtype=out, device=DEV)
    work = torch.empty(max(16, lib.blockscale_matmul_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    lib.blockscale_matmul(up(xq), up(xs), up(wq), up(ws), y, work)
    rows = torch.from_numpy(np.unique(np.concatenate([np.arange(20), M - 1 - np.arange(60), rng.integers(0, M, 200)])))
    ref, mag = product(values_rows(xq, xs)[rows], values_weight(wq, ws))
    tol = SUM(K) * mag + (2.0 ** -8 * ref.abs() if out == torch.bfloat16 else 0)
    err = (y.cpu().double()[rows] - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert torch.isfinite(y).all()


@gpu
def test_matmul_of_a_shared_k_repeats_bitwise():
    rng = np.random.default_rng(6)
    M, N, K = 70, 500, 8208
    (xq, xs), (wq, ws) = make_rows(rng, M, K), make_weight(rng, N, K)
    args = [up(t) for t in (xq, xs, wq, ws)]
    n = lib.blockscale_matmul_workspace_bytes(M, N, K)
    assert n > 0
    outs = []
    for fill in (0x00, 0x7f, 0xff):  # whatever the workspace held before
        y = torch.empty(M, N, device=DEV)
        lib.blockscale_matmul(*args, y, torch.full((n,), fill, dtype=torch.uint8, device=DEV))
        outs.append(y)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@gpu
def test_matmul_nan_codes_and_scales_stay_in_their_rows():
    rng = np.random.default_rng(5)
    M, N, K = 40, 200, 400
    (xq, xs), (wq, ws) = make_rows(rng, M, K), make_weight(rng, N, K)
    xq.view(torch.uint8)[3, 130] = 0x7f
    xs[7, 1] = float("nan")
    wq.view(torch.uint8)[150, 399] = 0xff
    y = torch.empty(M, N, device=DEV)
    work = torch.empty(max(16, lib.blockscale_matmul_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    lib.blockscale_matmul(up(xq), up(xs), up(wq), up(ws), y, work)
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3], bad[7], bad[:, 150] = True, True, True
    assert torch.equal(torch.isnan(y.cpu()), bad)


@gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(12, 300, 1040), (30, 300, 1040), (300, 600, 1040), (70, 500, 8208), (900, 1100, 2064),
                                   (1100, 4100, 1040), (3500, 3900, 1040)])
def test_matmul_nan_in_every_variant(M, N, K, out):
    rng = np.random.default_rng(M)
    (xq, xs), (wq, ws) = make_rows(rng, M, K), make_weight(rng, N, K)
    xq.view(torch.uint8)[3, 1030] = 0x7f
    xq.view(torch.uint8)[M - 1, 0] = 0xff
    wq.view(torch.uint8)[150, K - 1] = 0xff
    xs[7, 1] = float("nan")
    y = torch.empty(M, N, dtype=out, device=DEV)
    work = torch.empty(max(16, lib.blockscale_matmul_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    lib.blockscale_matmul(up(xq), up(xs), up(wq), up(ws), y, work)
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3], bad[7], bad[M - 1], bad[:, 150] = True, True, True, True
    assert torch.equal(torch.isnan(y.cpu()), bad)


# ----------------------------------------------------------------- experts ----
EXPERTS = [
    # T, k, E, d, f, share of routes without an expert
    (1, 1, 1, 16, 16, 0.0), (1, 6, 12, 1040, 528, 0.0), (2, 3, 5, 400, 144, 0.3), (8, 6, 40, 256, 384, 0.0),
    (5, 2, 1000, 256, 128, 0.0), (37, 4, 7, 528, 272, 0.1), (130, 2, 3, 272, 640, 0.0), (300, 6, 16, 512, 256, 0.02),
    (64, 1, 1, 384, 400, 0.0), (3, 2, 4, 128, 16, 1.0),
]


def expert_case(T, k, E, d, f, missing):
    rng = np.random.default_rng(T + 3 * k + 5 * E + 7 * d + 11 * f)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    if E > 2 and T > 20:  # crowd one expert
        idx[: T // 2, 0] = np.where((idx[: T // 2, 1:] == 1).any(1), idx[: T // 2, 0], 1)
    idx[rng.random((T, k)) < missing] = -1
    idx = torch.from_numpy(idx)
    wt = torch.from_numpy(rng.random((T, k), np.float32))
    return rng, idx, wt, buckets(idx, E)


@gpu
@pytest.mark.parametrize("T,k,E,d,f,missing", EXPERTS)
def test_gateup(T, k, E, d, f, missing):
    rng, idx, wt, (offsets, perm, pos) = expert_case(T, k, E, d, f, missing)
    xq, xs = make_rows(rng, T, d)
    wg, sg = make_weight(rng, f, d, E)
    wu, su = make_weight(rng, f, d, E)
    hq = torch.full((T * k, f), 0x33, dtype=torch.uint8, device=DEV)
    hs = torch.full((T * k, nb(f)), -3.0, device=DEV)
    lib.blockscale_gateup(up(xq), up(xs), k, up(offsets), up(perm), up(wg), up(sg), up(wu), up(su), hq, hs)
    torch.cuda.synchronize()
    hq, hs = hq.cpu(), hs.cpu()
    n = int(offsets[E])
    assert (hq[n:] == 0x33).all() and (hs[n:] == -3.0).all()
    x = values_rows(xq, xs)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        xe = x[(perm[a:b] // k).long()]
        g, gm = product(xe, values_weight(wg[e], sg[e]))
        u, um = product(xe, values_weight(wu[e], su[e]))
        dg, du = SUM(d) * gm, SUM(d) * um
        sg64 = torch.sigmoid(g)
        h = g * sg64 * u
        # |silu'| <= 1.1; silu's own error
        dh = 1.1 * dg * (u.abs() + du) + (g * sg64).abs() * (du + u.abs() * (2.0 ** -20 + g.abs() * 2.0 ** -22))
        pad = lambda v: torch.nn.functional.pad(v, (0, -f % 128)).view(b - a, -1, 128)  # noqa: E731
        s_ref, ds = pad(h).abs().amax(2) / 448, pad(dh).amax(2) / 448
        s_ref = s_ref.clamp(min=2.0 ** -100 / 448)
        s = hs[a:b].double()
        assert ((s - s_ref).abs() <= ds + 2.0 ** -22 * s_ref).all()
        v = hq[a:b].view(F8).double() * s.repeat_interleave(128, 1)[:, :f]
        tol = 2.0 ** -4 * (h.abs() + dh) + 2.0 ** -10 * s.repeat_interleave(128, 1)[:, :f] + dh
        assert ((v - h).abs() <= tol).all(), float(((v - h).abs() / tol).max())
        assert (pad(hq[a:b].view(F8).double()).abs().amax(2) == 448).all()


@gpu
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("T,k,E,d,f,missing", EXPERTS)
def test_down(T, k, E, d, f, missing, add):
    rng, idx, wt, (offsets, perm, pos) = expert_case(T, k, E, d, f, missing)
    hq, hs = make_rows(rng, T * k, f)
    n = int(offsets[E])
    hq.view(torch.uint8)[n:] = 0x7f  # rows of no route are not read into anything
    wd, sd = make_weight(rng, d, f, E)
    base = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)) if add else None
    y = torch.full((T, d), float("nan"), device=DEV)
    work = torch.full((max(16, lib.blockscale_down_workspace_bytes(T, k, d)),), 0xff, dtype=torch.uint8, device=DEV)
    lib.blockscale_down(up(hq), up(hs), up(wt), up(offsets), up(pos), up(wd), up(sd), y, work,
                        add=None if base is None else up(base))
    torch.cuda.synchronize()
    ref = torch.zeros(T, d, dtype=torch.float64) if base is None else base.double()
    mag = ref.abs()
    tol = torch.zeros_like(ref)
    h = values_rows(hq, hs)
    for r in range(n):
        e = int(torch.searchsorted(offsets[1:], r, right=True))
        t, j = int(perm[r]) // k, int(perm[r]) % k
        ye, m = product(h[r: r + 1], values_weight(wd[e], sd[e]))
        w = float(wt[t, j])
        ref[t] += w * ye[0]
        mag[t] += w * ye[0].abs()
        tol[t] += w * SUM(f) * m[0]
    tol += (k + 2) * 2.0 ** -23 * mag
    err = (y.cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


@gpu
def test_down_adds_in_place():
    rng, idx, wt, (offsets, perm, pos) = expert_case(9, 2, 4, 256, 128, 0.2)
    hq, hs = make_rows(rng, 18, 128)
    wd, sd = make_weight(rng, 256, 128, 4)
    base = torch.from_numpy(rng.standard_normal((9, 256)).astype(np.float32)).to(DEV)
    work = torch.empty(lib.blockscale_down_workspace_bytes(9, 2, 256), dtype=torch.uint8, device=DEV)
    args = [up(t) for t in (hq, hs, wt, offsets, pos, wd, sd)]
    y = torch.empty(9, 256, device=DEV)
    lib.blockscale_down(*args, y, work, add=base)
    lib.blockscale_down(*args, base, work, add=base)
    assert torch.equal(y, base)


@gpu
def test_weights_past_32_bit_offsets():
    """The last of 520 experts starts past 2^32 bytes."""
    E, d, f, T, k = 520, 4096, 2064, 3, 2
    rng = np.random.default_rng(11)
    wg = torch.zeros(E, f, d, dtype=torch.uint8, device=DEV)
    sg = torch.zeros(E, nb(f), nb(d), device=DEV)
    assert (E - 1) * f * d > 1 << 32
    last, sl = make_weight(rng, f, d)
    wg[E - 1], sg[E - 1] = last.view(torch.uint8).to(DEV), sl.to(DEV)
    xq, xs = make_rows(rng, T, d)
    idx = torch.tensor([[0, E - 1], [E - 1, 2], [5, E - 1]], dtype=torch.int32)
    offsets, perm, pos = buckets(idx, E)
    hq = torch.zeros(T * k, f, dtype=torch.uint8, device=DEV)
    hs = torch.zeros(T * k, nb(f), device=DEV)
    lib.blockscale_gateup(up(xq), up(xs), k, up(offsets), up(perm), wg, sg, wg, sg, hq, hs)
    a = int(offsets[E - 1])
    g, gm = product(values_rows(xq, xs)[(perm[a:] // k).long()], values_weight(last, sl))
    h = g * torch.sigmoid(g) * g
    s = hs[a:].cpu().double().repeat_interleave(128, 1)[:, :f]
    v = hq[a:].cpu().view(F8).double() * s
    dh = 2.2 * SUM(d) * gm * g.abs() + h.abs() * 2.0 ** -18
    assert ((v - h).abs() <= 2.0 ** -4 * (h.abs() + dh) + 2.0 ** -10 * s + dh).all()
    assert (hq[:a] == 0).all()
    # the same tensor as down weights: f outputs of d inputs
    y = torch.empty(T, f, device=DEV)
    wt = torch.ones(T, k)
    hq2, hs2 = make_rows(rng, T * k, d)
    work = torch.empty(lib.blockscale_down_workspace_bytes(T, k, f), dtype=torch.uint8, device=DEV)
    lib.blockscale_down(up(hq2), up(hs2), up(wt), up(offsets), up(pos), wg, sg, y, work)
    ref, mag = product(values_rows(hq2, hs2)[a:], values_weight(last, sl))
    order = (perm[a:] // k).long()
    assert ((y.cpu().double()[order] - ref).abs() <= 1.01 * SUM(d) * mag).all()


# ------------------------------------------------- streams, graphs, repeats ----
def chain(T, k, E, d, f):
    """quantize -> gateup -> down on fixed inputs: a callable and its outputs."""
    rng, idx, wt, (offsets, perm, pos) = expert_case(T, k, E, d, f, 0.0)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(DEV)
    wg, sg = (up(t) for t in make_weight(rng, f, d, E))
    wu, su = (up(t) for t in make_weight(rng, f, d, E))
    wd, sd = (up(t) for t in make_weight(rng, d, f, E))
    wt, offsets, perm, pos = up(wt), up(offsets), up(perm), up(pos)
    xq, xs = torch.empty(T, d, dtype=F8, device=DEV), torch.empty(T, nb(d), device=DEV)
    hq, hs = torch.empty(T * k, f, dtype=F8, device=DEV), torch.empty(T * k, nb(f), device=DEV)
    y, y2 = torch.empty(T, d, device=DEV), torch.empty(T, f, dtype=torch.bfloat16, device=DEV)
    work = torch.empty(lib.blockscale_down_workspace_bytes(T, k, d), dtype=torch.uint8, device=DEV)
    work2 = torch.empty(max(16, lib.blockscale_matmul_workspace_bytes(T, f, d)), dtype=torch.uint8, device=DEV)

    def run(stream=None):
        lib.blockscale_quantize(x, xq, xs, stream=stream)
        lib.blockscale_gateup(xq, xs, k, offsets, perm, wg, sg, wu, su, hq, hs, stream=stream)
        lib.blockscale_down(hq, hs, wt, offsets, pos, wd, sd, y, work, add=x, stream=stream)
        lib.blockscale_matmul(xq, xs, wg[0], sg[0], y2, work2, stream=stream)

    return run, [y, y2]


@gpu
@pytest.mark.parametrize("T", [1, 7, 200])
def test_streams_repeats_and_graphs_give_the_same_bits(T):
    run, outs = chain(T, 4, 9, 1040, 528)
    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]

    def same():
        torch.cuda.synchronize()
        ok = all(torch.equal(a, b) for a, b in zip(outs, want))
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        return ok

    assert same()
    side = torch.cuda.Stream()
    run(side)
    assert same()
    with torch.cuda.stream(side):
        run()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(4):
        graph.replay()
        assert same()
        run()
        assert same()


# ------------------------------------------------------------ no-ops, checks ----
def test_empty_calls_are_no_ops():
    L = lib.lib()
    assert L.moe_blockscale_quantize(None, 0, 256, 0, 256, None, 256, None, None) == lib.MOE_OK
    assert L.moe_blockscale_matmul(None, 256, None, 0, None, None, 64, 256, None, 0, 64, None, 0, None) == lib.MOE_OK
    assert L.moe_blockscale_gateup(None, None, 0, 2, None, None, 4, None, None, None, None, 256, 256, None, None,
                                   None) == lib.MOE_OK
    assert L.moe_blockscale_down(None, None, 0, 2, None, None, None, 4, None, None, 256, 256, None, None, None, 0,
                                 None) == lib.MOE_OK
    assert lib.blockscale_down_workspace_bytes(0, 2, 256) >= 0


P = 1 << 40  # a pointer that is never dereferenced: every call below is refused


def quantize_args(**kw):
    a = dict(x=P, x_dtype=0, ldx=256, M=4, K=256, q=P, ldq=256, s=P, stream=None)
    a.update(kw)
    return list(a.values())


def matmul_args(**kw):
    a = dict(xq=P, ldx=256, xs=P, M=4, wq=P, ws=P, N=64, K=256, y=P, y_dtype=0, ldy=64, workspace=P, n=1 << 40,
             stream=None)
    a.update(kw)
    return list(a.values())


def gateup_args(**kw):
    a = dict(xq=P, xs=P, T=4, k=2, offsets=P, perm=P, E=8, w_gate=P, s_gate=P, w_up=P, s_up=P, f=256, d=256, hq=P, hs=P,
             stream=None)
    a.update(kw)
    return list(a.values())


def down_args(**kw):
    a = dict(hq=P, hs=P, T=4, k=2, wt=P, offsets=P, pos=P, E=8, w_down=P, s_down=P, d=256, f=256, add=None, y=P,
             workspace=P, n=1 << 40, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(x_dtype=2), "UNSUPPORTED"), (dict(M=-1), "INVALID_ARG"), (dict(M=(1 << 20) + 1), "INVALID_ARG"),
    (dict(K=0), "INVALID_ARG"), (dict(K=24), "INVALID_ARG"), (dict(K=16400, ldx=16400, ldq=16400), "INVALID_ARG"),
    (dict(ldx=252), "INVALID_ARG"), (dict(ldx=257), "INVALID_ARG"), (dict(x_dtype=1, ldx=260), "INVALID_ARG"),
    (dict(ldq=240), "INVALID_ARG"), (dict(ldq=264), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"),
    (dict(x=P + 4), "INVALID_ARG"), (dict(q=P + 8), "INVALID_ARG"), (dict(s=None), "INVALID_ARG"),
])
def test_quantize_refusals(kw, code):
    assert lib.lib().moe_blockscale_quantize(*quantize_args(**kw)) == getattr(lib, "MOE_ERR_" + code)
    assert "moe_blockscale_quantize" in lib.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(y_dtype=7), "UNSUPPORTED"), (dict(M=-2), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"),
    (dict(N=65537), "INVALID_ARG"), (dict(K=40), "INVALID_ARG"), (dict(K=16384, N=65536, ldx=16384, ldy=65536), "OK?"),
    (dict(ldx=240), "INVALID_ARG"), (dict(ldx=260), "INVALID_ARG"), (dict(ldx=(1 << 22) + 16), "INVALID_ARG"), (dict(ldy=63), "INVALID_ARG"),
    (dict(xq=None), "INVALID_ARG"), (dict(xs=P + 4), "INVALID_ARG"), (dict(wq=P + 1), "INVALID_ARG"),
    (dict(ws=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"),
])
def test_matmul_refusals(kw, code):
    if code == "OK?":  # N * K = 2^30 is allowed: only its workspace query is asked here
        assert lib.blockscale_matmul_workspace_bytes(4, 65536, 16384) >= 0
        return
    assert lib.lib().moe_blockscale_matmul(*matmul_args(**kw)) == getattr(lib, "MOE_ERR_" + code)
    assert "moe_blockscale_matmul" in lib.last_error()


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=65537), dict(k=0), dict(k=17, E=64), dict(k=9), dict(E=0), dict(E=1025), dict(f=8), dict(f=250),
    dict(d=0), dict(d=16400), dict(xq=None), dict(xq=P + 8), dict(xs=None), dict(offsets=None), dict(perm=P + 4),
    dict(w_gate=None), dict(s_gate=P + 2), dict(w_up=P + 8), dict(s_up=None), dict(hq=None), dict(hs=P + 4),
])
def test_gateup_refusals(kw):
    assert lib.lib().moe_blockscale_gateup(*gateup_args(**kw)) == lib.MOE_ERR_INVALID_ARG
    assert "moe_blockscale_gateup" in lib.last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"), (dict(k=9), "INVALID_ARG"), (dict(E=1025), "INVALID_ARG"),
    (dict(d=100), "INVALID_ARG"), (dict(f=16400), "INVALID_ARG"), (dict(hq=None), "INVALID_ARG"),
    (dict(hs=P + 4), "INVALID_ARG"), (dict(wt=None), "INVALID_ARG"), (dict(offsets=None), "INVALID_ARG"),
    (dict(pos=None), "INVALID_ARG"), (dict(w_down=P + 8), "INVALID_ARG"), (dict(s_down=None), "INVALID_ARG"),
    (dict(y=None), "INVALID_ARG"), (dict(add=P + 4), "INVALID_ARG"),
])
def test_down_refusals(kw, code):
    assert lib.lib().moe_blockscale_down(*down_args(**kw)) == getattr(lib, "MOE_ERR_" + code)
    assert "moe_blockscale_down" in lib.last_error()


def test_small_workspaces_are_refused():
    need = lib.blockscale_down_workspace_bytes(40, 2, 256)
    if need:
        assert lib.lib().moe_blockscale_down(*down_args(T=40, n=need - 1)) == lib.MOE_ERR_WORKSPACE
        assert lib.lib().moe_blockscale_down(*down_args(T=40, workspace=None, n=need)) == lib.MOE_ERR_INVALID_ARG
    for M, N, K in ((1, 64, 16384), (64, 64, 16384), (300, 128, 16384)):
        need = lib.blockscale_matmul_workspace_bytes(M, N, K)
        if need:
            a = matmul_args(M=M, N=N, K=K, ldx=K, ldy=N, n=need - 1)
            assert lib.lib().moe_blockscale_matmul(*a) == lib.MOE_ERR_WORKSPACE


def test_binding_checks_shapes_and_dtypes():
    x, q, s = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="s has shape"):
        lib.blockscale_quantize(x, q, torch.zeros(4, 1), stream=_NoStream)
    with pytest.raises(TypeError, match="x must be"):
        lib.blockscale_quantize(x.half(), q, s, stream=_NoStream)
    with pytest.raises(ValueError, match="contiguous rows"):
        lib.blockscale_quantize(torch.zeros(256, 4).t(), q, s, stream=_NoStream)
    with pytest.raises(ValueError, match="q has shape"):
        lib.blockscale_quantize(x, q[:2], s, stream=_NoStream)
    w, ws, y = torch.zeros(64, 256, dtype=torch.uint8), torch.zeros(1, 2), torch.zeros(4, 64)
    with pytest.raises(ValueError, match="ws has shape"):
        lib.blockscale_matmul(q, s, w, torch.zeros(2, 2), y, stream=_NoStream)
    with pytest.raises(ValueError, match="wq has shape"):
        lib.blockscale_matmul(q, s, w[:, :128].contiguous(), ws, y, stream=_NoStream)
    with pytest.raises(ValueError, match="wq must be contiguous"):
        lib.blockscale_matmul(q, s, torch.zeros(64, 512, dtype=torch.uint8)[:, :256], ws, y, stream=_NoStream)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    wg, sg = torch.zeros(8, 128, 256, dtype=torch.uint8), torch.zeros(8, 1, 2)
    hq, hs = torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(8, 1)
    with pytest.raises(ValueError, match="perm has shape"):
        lib.blockscale_gateup(q, s, 2, i32(9), i32(7), wg, sg, wg, sg, hq, hs, stream=_NoStream)
    with pytest.raises(ValueError, match="offsets has shape"):
        lib.blockscale_gateup(q, s, 2, i32(8), i32(8), wg, sg, wg, sg, hq, hs, stream=_NoStream)
    with pytest.raises(ValueError, match="hq has shape"):
        lib.blockscale_gateup(q, s, 2, i32(9), i32(8), wg, sg, wg, sg, hq[:4], hs, stream=_NoStream)
    with pytest.raises(TypeError, match="pos must be"):
        lib.blockscale_down(hq, hs, torch.zeros(4, 2), i32(9), torch.zeros(8), torch.zeros(8, 256, 128, dtype=torch.uint8),
                            torch.zeros(8, 2, 1), torch.zeros(4, 256), None, stream=_NoStream)


class _NoStream:
    cuda_stream = None


def test_binding_refuses_host_memory():
    x, q, s = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    w, ws, y = torch.zeros(64, 256, dtype=torch.uint8), torch.zeros(1, 2), torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU memory"):
        lib.blockscale_quantize(x, q, s, stream=_NoStream)
    with pytest.raises(ValueError, match="GPU memory"):
        lib.blockscale_matmul(q, s, w, ws, y, stream=_NoStream)


@gpu
def test_binding_names_what_is_wrong_on_the_gpu_too():
    f = lambda *n: torch.zeros(*n, device=DEV)  # noqa: E731
    u8 = lambda *n: torch.zeros(*n, dtype=torch.uint8, device=DEV)  # noqa: E731
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    x, q, s, w, ws, y = f(4, 256), u8(4, 256), f(4, 2), u8(64, 256), f(1, 2), f(4, 64)
    with pytest.raises(TypeError, match="x must be"):
        lib.blockscale_quantize(x.half(), q, s)
    with pytest.raises(ValueError, match="s has shape"):
        lib.blockscale_quantize(x, q, s[:3])
    with pytest.raises(lib.MoeError, match="ldx"):
        lib.blockscale_quantize(f(4, 258)[:, :256], q, s)  # rows not 16 bytes apart: the library's own check
    with pytest.raises(ValueError, match="contiguous rows"):
        lib.blockscale_matmul(u8(256, 4).t(), s, w, ws, y)
    with pytest.raises(TypeError, match="xs must be"):
        lib.blockscale_matmul(q, s.double(), w, ws, y)
    with pytest.raises(ValueError, match="wq must be contiguous"):
        lib.blockscale_matmul(q, s, u8(64, 512)[:, :256], ws, y)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        lib.blockscale_matmul(q, s, w, ws, y, u8(64, 64)[:, ::2])
    with pytest.raises(ValueError, match="GPU memory"):
        lib.blockscale_matmul(q, s.cpu(), w, ws, y)
    wg, sg, hq, hs = u8(8, 128, 256), f(8, 1, 2), u8(8, 128), f(8, 1)
    with pytest.raises(ValueError, match="offsets has shape"):
        lib.blockscale_gateup(q, s, 2, i32(8), i32(8), wg, sg, wg, sg, hq, hs)
    with pytest.raises(TypeError, match="pos must be"):
        lib.blockscale_down(hq, hs, f(4, 2), i32(9), f(8), u8(8, 256, 128), f(8, 2, 1), f(4, 256), None)
    with pytest.raises(ValueError, match="add has shape"):
        lib.blockscale_down(hq, hs, f(4, 2), i32(9), i32(8), u8(8, 256, 128), f(8, 2, 1), f(4, 256), u8(65536), add=f(4, 255))
    with pytest.raises(TypeError, match="arguments"):
        lib._load_calls().matmul(q, s)
    with pytest.raises(AttributeError):
        lib.blockscale_quantize(x, q, s, stream=7)


@gpu
@pytest.mark.parametrize("T,k,f", [(2, 16, 1424), (1, 16, 16), (2, 5, 128), (1, 16, 272), (2, 7, 1040), (1, 9, 2064),
                                   (2, 16, 4112)])
def test_two_tokens_that_share_an_expert_and_lose_routes(T, k, f):
    """The one-launch down product: one and two tokens, routes of which some have no place, few blocks and many."""
    rng = np.random.default_rng(21)
    E, d = 20, 80
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[0, 3] = idx[T - 1, 0] = idx[T - 1, k - 1] = -1
    offsets, perm, pos = (t.to(DEV) for t in buckets(torch.from_numpy(idx), E)[-3:])
    hq, hs = make_rows(rng, T * k, f)
    wq, ws = make_weight(rng, d, f, E)
    wt = torch.from_numpy(rng.random((T, k)).astype(np.float32))
    y = torch.full((T, d), float("nan"), device=DEV)
    assert lib.blockscale_down_workspace_bytes(T, k, d) == 0
    lib.blockscale_down(up(hq), up(hs), up(wt), offsets, pos, up(wq), up(ws), y, None)
    ref, mag = torch.zeros(T, d, dtype=torch.float64), torch.zeros(T, d, dtype=torch.float64)
    p = pos.cpu().tolist()
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if e < 0:
                continue
            r = p[t * k + j]
            a, b = product(values_rows(hq[r: r + 1], hs[r: r + 1]), values_weight(wq[e], ws[e]))
            ref[t] += wt[t, j].double() * a[0]
            mag[t] += wt[t, j].double() * b[0]
    tol = (SUM(f) + (k + 2) * 2.0 ** -24) * mag
    assert ((y.cpu().double() - ref).abs() <= tol).all()
