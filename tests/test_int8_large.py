"""Offsets past 32 bits, and calls of nothing: the results are those of the same rows in a small call."""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib
from test_balance import forward, make
from test_int8 import make_codes, make_scales

gpu = pytest.mark.gpu
DEV = "cuda:0"


def up(a):
    return torch.from_numpy(a).to(DEV)


@gpu
def test_quantize_past_32_bits():
    M, K = 140000, 16384
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    last = torch.randn(5, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(torch.bfloat16)
    x[-5:] = last
    q, s = torch.full((M, K), 7, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    lib.int8_quantize(x, q, s)
    q5, s5 = torch.empty(5, K, dtype=torch.int8, device=DEV), torch.empty(5, device=DEV)
    lib.int8_quantize(last, q5, s5)
    assert torch.equal(q[-5:], q5) and torch.equal(s[-5:], s5)
    assert (s[:-5] == float(np.float32(2.0 ** -100) / np.float32(127))).all()
    assert not any(bool(part.any()) for part in q[:-5].split(20000))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product_past_32_bits(dtype):
    M, N, K = 140000, 16384, 16
    rng = np.random.default_rng(2)
    xq, xs = up(make_codes(rng, M, K)), up(make_scales(rng, 1.0, M))
    wq, ws = up(make_codes(rng, N, K)), up(make_scales(rng, 1.0, N))
    y = torch.empty(M, N, dtype=dtype, device=DEV)
    lib.int8_matmul(xq, xs, wq, ws, y)
    for a in (0, 65530, 131072, M - 300):
        part = torch.empty(300, N, dtype=dtype, device=DEV)
        lib.int8_matmul(xq[a: a + 300].contiguous(), xs[a: a + 300].clone(), wq, ws, part)
        assert torch.equal(y[a: a + 300], part)


@gpu
@pytest.mark.parametrize("T", [2, 40])
def test_experts_past_32_bits(T):
    E, d, f, k = 300, 4096, 2048, 3
    rng = np.random.default_rng(T)
    idx = torch.tensor([[299, 0, 298]] * T, dtype=torch.int32, device=DEV)
    R = T * k
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    counts, perm, pos = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (E, R, R))
    lib.bucket(idx, E, counts, offsets, perm, pos)
    few = torch.tensor([[2, 0, 1]] * T, dtype=torch.int32, device=DEV)   # the same, of three experts
    offsets3, counts3, perm3, pos3 = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (4, 3, R, R))
    lib.bucket(few, 3, counts3, offsets3, perm3, pos3)
    w, s = torch.zeros(E, f, d, dtype=torch.int8, device=DEV), torch.ones(E, f, device=DEV)
    w3, s3 = up(make_codes(rng, 3, f, d)), up(make_scales(rng, 0.02, 3, f))
    w[[0, 298, 299]], s[[0, 298, 299]] = w3, s3
    xq, xs, wt = up(make_codes(rng, T, d)), up(make_scales(rng, 1.0, T)), up(rng.random((T, k)).astype(np.float32))
    h, h3 = torch.empty(R, f, device=DEV), torch.empty(R, f, device=DEV)
    lib.int8_gateup(xq, xs, k, offsets, perm, w, s, w, s, h)
    lib.int8_gateup(xq, xs, k, offsets3, perm3, w3, s3, w3, s3, h3)
    assert torch.equal(h, h3)
    hq, hs = up(make_codes(rng, R, f)), up(make_scales(rng, 1.0, R))
    wd, sd, wd3, sd3 = w.view(E, d, f), torch.ones(E, d, device=DEV), w3.view(3, d, f), up(make_scales(rng, 0.02, 3, d))
    sd[[0, 298, 299]] = sd3
    work = torch.empty(lib.int8_down_workspace_bytes(T, k, d), dtype=torch.uint8, device=DEV)
    y, y3 = torch.empty(T, d, device=DEV), torch.empty(T, d, device=DEV)
    lib.int8_down(hq, hs, wt, offsets, pos, wd, sd, y, work)
    lib.int8_down(hq, hs, wt, offsets3, pos3, wd3, sd3, y3, work)
    assert torch.equal(y, y3)


@gpu
def test_balance_past_32_bits():
    T, E, k, stride = 65536, 24, 3, 40000
    rng = np.random.default_rng(3)
    z, idx, starts = make(rng, T, E, k, 4, dtype=torch.bfloat16)
    wide = torch.empty(T, stride, dtype=torch.bfloat16, device=DEV)
    zw = wide[:, 100: 100 + E]
    zw.copy_(z)
    a = forward(z.to(DEV), idx, starts, "softmax", 1.0, 4)
    b = forward(zw, idx, starts, "softmax", 1.0, 4)
    assert all(torch.equal(u, v) for u, v in zip(a[:3], b[:3]))
    dz, dw = torch.empty(T, E, dtype=torch.bfloat16, device=DEV), wide[:, 30000: 30000 + E]
    for v, out in ((z.to(DEV), dz), (zw, dw)):
        lib.balance_loss_backward(v, torch.from_numpy(idx).to(DEV), a[0], a[1], torch.ones(4, device=DEV), out, starts=a[3])
    assert torch.equal(dz, dw)


@gpu
def test_calls_of_no_rows():
    i8 = lambda *n: torch.zeros(*n, dtype=torch.int8, device=DEV)  # noqa: E731
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device=DEV)  # noqa: E731
    f = lambda *n: torch.zeros(*n, device=DEV)  # noqa: E731
    lib.int8_quantize(f(0, 64), i8(0, 64), f(0))
    lib.int8_matmul(i8(0, 64), f(0), i8(8, 64), f(8), f(0, 8))
    lib.int8_gateup(i8(0, 64), f(0), 2, i32(5), i32(0), i8(4, 16, 64), f(4, 16), i8(4, 16, 64), f(4, 16), f(0, 16))
    lib.int8_down(i8(0, 16), f(0), f(0, 2), i32(5), i32(0), i8(4, 64, 16), f(4, 64), f(0, 64), None)
    lib.balance_loss_backward(f(0, 8), i32(0, 2), i32(1, 8), i32(1), f(1), f(0, 8))
    counts, tokens, loss = i32(1, 8) + 5, i32(1) + 5, f(1) + 5
    lib.balance_loss(f(0, 8), i32(0, 2), counts, tokens, loss, None)
    assert not counts.any() and not tokens.any() and not loss.any()
    # every route without a place: the rows belong to the last expert (offsets[E] = T * k), nothing
    # reads them, and only the added term is left
    T, k, E = 40, 2, 4
    idx, offsets, perm, pos = i32(T, k) - 1, i32(E + 1), i32(T * k), i32(T * k)
    lib.bucket(idx, E, i32(E), offsets, perm, pos)
    h = f(T * k, 16) + 5
    lib.int8_gateup(i8(T, 64), f(T), k, offsets, perm, i8(E, 16, 64), f(E, 16), i8(E, 16, 64), f(E, 16), h)
    assert offsets.tolist() == [0, 0, 0, 0, T * k] and not h.any()  # (codes of 0)
    h = f(T * k, 16) + 5
    lib.int8_gateup(i8(T, 64), f(T), k, i32(E + 1), perm, i8(E, 16, 64), f(E, 16), i8(E, 16, 64), f(E, 16), h)
    assert (h == 5).all()  # offsets of 0: no rows at all
    for T in (1, 2, 40):
        add, y = torch.randn(T, 64, device=DEV), f(T, 64)
        offsets[E] = T * k
        work = torch.empty(lib.int8_down_workspace_bytes(T, k, 64), dtype=torch.uint8, device=DEV).fill_(0xff)
        lib.int8_down(i8(T * k, 16), f(T * k), f(T, k), offsets, torch.full((T * k,), T * k, dtype=torch.int32, device=DEV),
                      i8(E, 64, 16), f(E, 64), y, work, add=add)
        assert torch.equal(y, add)
