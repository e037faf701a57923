"""The gate's reciprocal: on the CPU for every fp32 significand, on the GPU for every logit.

Two Newton steps with fused residuals, r + r (1 - x r), from any start within a
unit of 1 / x (what the hardware's reciprocal instruction promises), end at the
fp32 number nearest to 1 / x, but for one significand: x = 2 - 2^-23 lies so near
the middle of two results that only the nearest start stays right.  Whether the
hardware gives that one is seen on the GPU.  x in [1, 2) stands for all of [1,
2^117] in the steps: a power of two scales each exactly.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib

f4 = np.float32


def fma_step(x, r):
    """fp32 fma(fma(-x, r, 1), r, r); x, r fp32 numbers held in 64 bits."""
    e = (1.0 - x * r).astype(f4).astype(np.float64)  # (x r has 48 bits, 1 - x r no more: exact before its rounding)
    p = e * r                                        # (exact)
    s = r + p
    low = (r - s) + p                                # the rounding of s, exactly (|p| < |r|)
    y = s.astype(f4)
    # s half way between two fp32 numbers, but the exact sum beside it
    other = np.nextafter(y, np.where(s > y, f4(np.inf), f4(-np.inf)).astype(f4))
    half = (s != y) & (np.abs(s - y) == np.abs(other.astype(np.float64) - s))
    up = np.maximum(y, other)
    down = np.minimum(y, other)
    y = np.where(half & (low > 0), up, np.where(half & (low < 0), down, y))
    return y.astype(np.float64)


def test_every_significand():
    hard = []
    for first in range(0, 1 << 23, 1 << 20):
        x = (np.arange(first, first + (1 << 20), dtype=np.uint32) + np.uint32(0x3f800000)).view(f4).astype(np.float64)
        want = (1.0 / x).astype(f4)  # (the quotient of fp32 numbers rounded to 64 and then to 32 bits is correctly rounded)
        for start in (want, np.nextafter(want, f4(0)), np.nextafter(want, f4(2))):
            r = fma_step(x, fma_step(x, start.astype(np.float64)))
            wrong = r.astype(f4) != want
            assert not (wrong & (start == want)).any()
            hard += x[wrong].tolist()
    assert set(hard) == {2 - 2.0 ** -23}


def test_the_fused_step_against_whole_numbers():
    """fma_step against exact rationals, at random and for starts a few units off."""
    from fractions import Fraction

    def nearest(v):
        y = f4(float(v))  # (a neighbour at least)
        near = [y, np.nextafter(y, f4(-4)), np.nextafter(y, f4(4))]
        best = min(abs(Fraction(float(c)) - v) for c in near)
        near = [c for c in near if abs(Fraction(float(c)) - v) == best]
        return next((c for c in near if c.view(np.uint32) % 2 == 0), near[0]) if len(near) > 1 else near[0]

    rng = np.random.default_rng(1)
    for _ in range(2000):
        x = (np.uint32(0x3f800000) + np.uint32(rng.integers(0, 1 << 23))).view(f4)
        r = f4(1.0 / float(x))
        r = (r.view(np.uint32) + np.uint32(rng.integers(0, 5)) - np.uint32(2)).view(f4)
        e = nearest(1 - Fraction(float(x)) * Fraction(float(r)))
        want = nearest(Fraction(float(e)) * Fraction(float(r)) + Fraction(float(r)))
        got = fma_step(np.array([x], np.float64), np.array([r], np.float64))[0]
        assert float(want) == got


@pytest.mark.gpu
def test_the_score_of_every_logit():
    """All fp32 logits up to 80 in magnitude: one expert's plain weight is 1 / (1 + exp32(-z)), bit for bit."""
    dev = "cuda:0"
    g = lib.gate(1, 1, renormalize=False)
    n, T = 1 << 24, 65536
    idx, wt = torch.empty(T, 1, dtype=torch.int32, device=dev), torch.empty(n, 1, device=dev)
    log2e, hi, lo, magic = (float.fromhex(h) for h in ("0x1.715476p0", "0x1.62e400p-1", "0x1.7f7d1cp-20", "0x1.8p23"))
    steps = [float.fromhex(h) for h in ("0x1.6c16c2p-10", "0x1.111112p-7", "0x1.555556p-5", "0x1.555556p-3", "0x1p-1", "0x1p0",
                                        "0x1p0")]
    last = int(np.array(80.0, f4).view(np.uint32))
    for sign in (0, -1 << 31):
        for first in range(0, last + 1, n):
            bits = torch.arange(first, first + n, dtype=torch.int32, device=dev).clamp_(max=last) | sign
            z = bits.view(torch.float32).view(n, 1)
            for t in range(0, n, T):
                lib.gate_topk(g, z[t: t + T], idx, wt[t: t + T])
            u = -z
            k = (u * log2e + magic) - magic
            r = (u - k * hi) - k * lo
            p = torch.full_like(r, steps[0])
            for c in steps[1:]:
                p = p * r + c
            e = p * ((k.to(torch.int32) + 127) << 23).view(torch.float32)
            want = (1.0 / (1.0 + e).double()).float()
            assert torch.equal(wt, want), (sign, first)
