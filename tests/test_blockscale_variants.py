"""Values of the block-scaled products in each variant that a rule on sizes chooses.

The tolerances are those of test_blockscale.py: SUM(K) of the sums of magnitudes
for a product, 2^-8 of the value for bf16, half a step for E4M3 codes.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib
from test_blockscale import DEV, F8, SUM, buckets, make_rows, make_weight, nb, product, up, values_rows, values_weight

gpu = pytest.mark.gpu


# ------------------------------------------------------------------ matmul ----
@gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(32, 6150, 2064), (17, 6200, 144), (9, 70, 8208), (30, 70, 4112), (1100, 4100, 1040),
                                   (1000, 1100, 2064), (700, 1500, 1040)])
def test_matmul_values(M, N, K, out):
    rng = np.random.default_rng(M + 3 * N + 5 * K)
    (xq, xs), (wq, ws) = make_rows(rng, M, K), make_weight(rng, N, K)
    y = torch.empty(M, N, dtype=out, device=DEV)
    work = torch.empty(max(16, lib.blockscale_matmul_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    lib.blockscale_matmul(up(xq), up(xs), up(wq), up(ws), y, work)
    ref, mag = product(values_rows(xq, xs), values_weight(wq, ws))
    tol = SUM(K) * mag + (2.0 ** -8 * ref.abs() if out == torch.bfloat16 else 0)
    err = (y.cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())


@gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(12, 300, 1040), (30, 300, 1040), (32, 6150, 1040), (300, 600, 1040), (70, 500, 8208),
                                   (1000, 1100, 2064), (530, 4100, 1296), (1100, 4100, 1040), (2090, 4100, 1040),
                                   (3500, 3900, 1040)])
def test_matmul_values_beside_numbers_that_are_not(M, N, K, out):
    rng = np.random.default_rng(M + N)
    (xq, xs), (wq, ws) = make_rows(rng, M, K), make_weight(rng, N, K)
    clean = values_rows(xq, xs), values_weight(wq, ws)
    xq.view(torch.uint8)[3, 1030] = 0x7f
    xq.view(torch.uint8)[M - 1, 0] = 0xff
    wq.view(torch.uint8)[150, K - 1] = 0xff
    xs[7, 1] = float("nan")
    y = torch.empty(M, N, dtype=out, device=DEV)
    work = torch.empty(max(16, lib.blockscale_matmul_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    lib.blockscale_matmul(up(xq), up(xs), up(wq), up(ws), y, work)
    y = y.cpu().double()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3], bad[7], bad[M - 1], bad[:, 150] = True, True, True, True
    assert torch.equal(torch.isnan(y), bad)
    rows = torch.from_numpy(np.unique(np.concatenate([np.arange(min(M, 20)), M - 1 - np.arange(min(M, 60)),
                                                      rng.integers(0, M, 200)])))
    ref, mag = product(clean[0][rows], clean[1])
    tol = SUM(K) * mag + (2.0 ** -8 * ref.abs() if out == torch.bfloat16 else 0)
    assert ((y[rows] - ref).abs() <= tol)[~bad[rows]].all()


# ----------------------------------------------------------------- experts ----
# What chooses: the rows per expert (tiles of 16, 32, 48 or 128 rows) and, for
# tiles of BM rows, whether there are 128 BM rows (each XCD then takes groups of
# tiles in turn).  For each such tile a case below and one above, with outputs of
# several tiles and short ends everywhere.
SIZES = [
    # T, k, E, d, f                 tile of gate/up, of down
    (2048, 1, 1024, 272, 272),    # 16 in turn, 16 in turn
    (1100, 2, 600, 272, 400),     # 16 in turn, 32
    (60, 3, 20, 528, 272),        # 32, 32
    (1400, 3, 400, 528, 144),     # 32 in turn, 32 in turn
    (500, 2, 60, 272, 272),       # 48, 48
    (1600, 4, 60, 528, 272),      # 48 in turn, 48 in turn
    (700, 2, 5, 528, 400),        # 128, 128
    (300, 1, 1, 272, 272),        # 128, 128: one expert
    (4200, 4, 40, 528, 272),      # 128 in turn, 128 in turn
]
KINDS = ["uniform", "crowded", "few", "lost"]


def routes(rng, T, k, E, kind):
    """Routes to all experts alike; half of the tokens to one of them; to k + 1 of them; a third without an expert."""
    among = rng.permutation(E)[: min(E, k + 1)] if kind == "few" else np.arange(E)
    idx = np.argsort(rng.random((T, len(among))), axis=1)[:, :k]
    idx = among[idx].astype(np.int32)
    if kind == "crowded" and E > 1:
        one = E // 3
        idx[: T // 2, 0] = np.where((idx[: T // 2, 1:] == one).any(1), idx[: T // 2, 0], one)
    if kind == "lost":
        idx[rng.random((T, k)) < 0.3] = -1
    return buckets(torch.from_numpy(idx), E)


def experts_of(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,k,E,d,f", SIZES)
def test_gateup_values(T, k, E, d, f, kind):
    rng = np.random.default_rng(T + 3 * k + 5 * E + len(kind))
    offsets, perm, pos = routes(rng, T, k, E, kind)
    xq, xs = make_rows(rng, T, d)
    wg, sg = make_weight(rng, f, d, E)
    wu, su = make_weight(rng, f, d, E)
    hq = torch.full((T * k, f), 0x33, dtype=torch.uint8, device=DEV)
    hs = torch.full((T * k, nb(f)), -3.0, device=DEV)
    lib.blockscale_gateup(up(xq), up(xs), k, up(offsets), up(perm), up(wg), up(sg), up(wu), up(su), hq, hs)
    hq, hs = hq.cpu(), hs.cpu()
    n = int(offsets[E])
    assert (hq[n:] == 0x33).all() and (hs[n:] == -3.0).all()
    x = values_rows(xq, xs)
    for e, a, b in experts_of(offsets):
        xe = x[(perm[a:b] // k).long()]
        g, gm = product(xe, values_weight(wg[e], sg[e]))
        u, um = product(xe, values_weight(wu[e], su[e]))
        dg, du = SUM(d) * gm, SUM(d) * um
        s64 = torch.sigmoid(g)
        h = g * s64 * u
        # |silu'| <= 1.1; silu's own error
        dh = 1.1 * dg * (u.abs() + du) + (g * s64).abs() * (du + u.abs() * (2.0 ** -20 + g.abs() * 2.0 ** -22))
        pad = lambda v: torch.nn.functional.pad(v, (0, -f % 128)).view(b - a, -1, 128)  # noqa: E731
        s_ref, ds = pad(h).abs().amax(2) / 448, pad(dh).amax(2) / 448
        s = hs[a:b].double()
        assert ((s - s_ref).abs() <= ds + 2.0 ** -22 * s_ref).all(), e
        wide = s.repeat_interleave(128, 1)[:, :f]
        tol = 2.0 ** -4 * (h.abs() + dh) + 2.0 ** -10 * wide + dh
        assert ((hq[a:b].view(F8).double() * wide - h).abs() <= tol).all(), e


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,k,E,d,f", SIZES)
def test_down_values(T, k, E, d, f, kind):
    rng = np.random.default_rng(2 * T + 3 * k + 5 * E + len(kind))
    offsets, perm, pos = routes(rng, T, k, E, kind)
    hq, hs = make_rows(rng, T * k, f)
    n = int(offsets[E])
    hq.view(torch.uint8)[n:] = 0x7f  # rows of no route are not read into anything
    wd, sd = make_weight(rng, d, f, E)
    wt = torch.from_numpy(rng.random((T, k), np.float32))
    y = torch.full((T, d), float("nan"), device=DEV)
    work = torch.full((max(16, lib.blockscale_down_workspace_bytes(T, k, d)),), 0xff, dtype=torch.uint8, device=DEV)
    lib.blockscale_down(up(hq), up(hs), up(wt), up(offsets), up(pos), up(wd), up(sd), y, work)
    h = values_rows(hq, hs)
    ye, ym = torch.zeros(T * k + 1, d, dtype=torch.float64), torch.zeros(T * k + 1, d, dtype=torch.float64)
    for e, a, b in experts_of(offsets):
        ye[a:b], ym[a:b] = product(h[a:b], values_weight(wd[e], sd[e]))
    w = wt.double()[:, :, None]
    at = pos.long().view(T, k)  # (T k: the row of zeros)
    ref = (w * ye[at]).sum(1)
    tol = SUM(f) * (w * ym[at]).sum(1) + (k + 2) * 2.0 ** -23 * (w * ye[at].abs()).sum(1)
    err = (y.cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


@gpu
def test_a_token_has_the_same_bits_in_every_batch():
    """Gate/up in every tile, and down of three tokens and more: the first tokens of the largest batch by themselves."""
    k, E, d, f, most = 2, 6, 400, 272, 8200
    rng = np.random.default_rng(17)
    idx = torch.from_numpy(np.argsort(rng.random((most, E)), axis=1)[:, :k].astype(np.int32))
    (xq, xs), (wg, sg), (wu, su), (wd, sd) = make_rows(rng, most, d), *(make_weight(rng, *s, E) for s in ((f, d), (f, d), (d, f)))
    wt = torch.from_numpy(rng.random((most, k), np.float32))
    want = None
    for T in (most, 700, 300, 30, 10, 3, 2, 1):
        offsets, perm, pos = buckets(idx[:T], E)
        hq = torch.empty(T * k, f, dtype=torch.uint8, device=DEV)
        hs = torch.empty(T * k, nb(f), device=DEV)
        y = torch.empty(T, d, device=DEV)
        work = torch.empty(max(16, lib.blockscale_down_workspace_bytes(T, k, d)), dtype=torch.uint8, device=DEV)
        lib.blockscale_gateup(up(xq[:T]), up(xs[:T]), k, up(offsets), up(perm), up(wg), up(sg), up(wu), up(su), hq, hs)
        lib.blockscale_down(hq, hs, up(wt[:T]), up(offsets), up(pos), up(wd), up(sd), y, work)
        at = pos.long().to(DEV)
        have = hq[at], hs[at], y  # (by route, by route, by token)
        if want is None:
            want = have
        assert torch.equal(have[0], want[0][: T * k]) and torch.equal(have[1], want[1][: T * k])
        if T > 2:
            assert torch.equal(y, want[2][:T])
