"""The gate in each layout that the numbers of experts and groups choose.

Lanes per group: 64 (no groups chosen), 8 (5 to 8 groups), or another power of
two; experts per lane: up to 4, 6, 8, 16 or 32, with every lane full or not.
"""
import numpy as np
import pytest
import torch

from test_gate import check, f4

gpu = pytest.mark.gpu

# E, groups, kept groups
ONE = [(200, 1, 1), (256, 1, 1), (300, 1, 1), (384, 1, 1), (450, 1, 1), (512, 1, 1), (1000, 1, 1), (1024, 1, 1)]
EIGHT_LANES = [(160, 8, 3), (256, 8, 4), (352, 8, 4), (384, 8, 2), (480, 8, 5), (512, 8, 3), (800, 8, 4), (1024, 8, 7),
               (1020, 5, 2), (1022, 7, 4), (996, 6, 5)]
OTHER = [(240, 2, 1), (300, 2, 1), (500, 2, 1), (1000, 2, 1), (1023, 3, 2), (768, 4, 3), (990, 10, 6), (1008, 16, 9),
         (1023, 31, 20), (1023, 33, 20), (1024, 64, 40), (63, 21, 16)]


@gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,KG", ONE + EIGHT_LANES + OTHER)
def test_layouts(E, G, KG, score):
    rng = np.random.default_rng(E + G)
    k = min(16, KG * (E // G))
    plain = (2 * rng.standard_normal((5, E))).astype(f4)
    ties = (np.round(4 * rng.standard_normal((4, E))) / 4).astype(f4)
    masked = plain[:4].copy()
    masked[rng.random((4, E)) < 0.5] = -np.inf
    masked[3] = -np.inf
    close = (1 + rng.integers(0, 200, (3, E)) * f4(2.0 ** -22)).astype(f4)
    z = torch.from_numpy(np.concatenate([plain, ties, masked, close]))
    bias = (0.1 * rng.standard_normal(E)).astype(f4)
    for dtype in (torch.float32, torch.bfloat16):
        for kk, gs, b in ((k, "max", None), (k, "top2", None), (min(k, 6), "top2", bias), (1, "max", bias)):
            check(z.to(dtype), kk, score, G, KG, gs, True, 2.5, b)
