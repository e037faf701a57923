"""The balance loss with every number of experts a lane: a block for all tokens, and waves
that take one or several tokens each.  References and tolerances of test_balance.py."""
import pytest
import torch

import test_balance

gpu = pytest.mark.gpu

# (tokens, experts, routes, sequences)
SMALL = [(100, 100, 16, 3), (128, 200, 9, 2), (60, 512, 12, 4), (128, 1024, 16, 12), (33, 700, 10, 5), (7, 448, 16, 2)]
LARGE = [(300, 512, 16, 3), (129, 385, 9, 2), (1100, 450, 8, 70), (260, 641, 11, 20)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S", SMALL + LARGE)
def test_experts_of_a_lane(T, E, k, S, score, dtype):
    test_balance.test_loss_and_gradient(T, E, k, S, score, dtype)


@gpu
@pytest.mark.parametrize("score,dtype", [("softmax", torch.float32), ("sigmoid", torch.bfloat16)])
@pytest.mark.parametrize("T,E,k,S", [(9000, 100, 3, 5), (8500, 250, 5, 3), (9000, 384, 6, 3), (8500, 450, 8, 70), (17000, 700, 4, 6)])
def test_several_tokens_a_wave(T, E, k, S, score, dtype):
    test_balance.test_loss_and_gradient(T, E, k, S, score, dtype)
