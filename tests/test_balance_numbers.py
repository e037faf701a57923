"""The balance calls' numbers, from Python on."""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib
from test_balance import Q, STEP, forward, make, plain
from test_int8_memory import DEV, make_calls

gpu = pytest.mark.gpu


class Bare:  # (a stream by its handle alone: the default one)
    cuda_stream = 0


BAD = [("half", TypeError), (None, TypeError), (10 ** 400, OverflowError)]


@pytest.mark.parametrize("name", ["balance_loss", "balance_loss_backward"])
@pytest.mark.parametrize("dev", ["cpu", pytest.param(DEV, marks=gpu)])
def test_an_alpha_that_is_no_number(name, dev):
    """The error is Python's own, whatever the stream is made of and wherever the tensors are (-1 was taken for
    the number where the stream named no device)."""
    call, args = make_calls(dev)[name]
    for alpha, error in BAD:
        with pytest.raises(error):
            call(**args, alpha=alpha, stream=Bare)


@gpu
@pytest.mark.parametrize("name", ["balance_loss", "balance_loss_backward"])
def test_an_alpha_of_minus_one(name):
    """The value that a failed conversion would leave is a number like any other."""
    call, args = make_calls(DEV)[name]
    call(**args, alpha=-1)
    call(**args, alpha=-1.0)
    with pytest.raises(lib.MoeError, match="alpha is not finite"):
        call(**args, alpha=1e39)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,alpha,g", [(2000, 64, 1, 2e38, 1e-6), (1, 8, 1, 3e38, 1e-30), (2000, 64, 1, 1e10, 1e30), (2000, 64, 1, 1e10, -1e30),
                                           (2000, 64, 1, 1.0, 3e-35), (2000, 64, 1, -1e-30, 1e-5), (3000, 100, 4, 1e-38, 1e10),
                                           (4000, 1000, 8, 1e-44, 1e30)])
def test_far_alphas_and_gradients(T, E, k, alpha, g, score):
    """Factors g alpha E / (k n^2) in fp32's range whose parts are not: the gradient is the formula's.  Tolerances as in
    test_balance.py; a factor below the normal numbers is off by 2^-150, times c <= 2^13 here: below 2^-126."""
    rng = np.random.default_rng(T)
    z, idx, starts = make(rng, T, E, k, 1, mask=0.02)
    idx[:, 0] = np.where(rng.random(T) < 0.9, 5, idx[:, 0])   # (most routes on one expert: large differences)
    c, n, loss, _ = forward(z.to(DEV), idx, starts, score, alpha, 1)
    alpha, g = float(np.float32(alpha)), float(np.float32(g))
    want, dz, unit = plain(z.double().numpy(), idx, starts, score, alpha, np.array([g]))[2:]
    assert abs(float(loss) - want[0]) <= abs(want[0]) * (Q(E, 6.0) + STEP) + 2.0 ** -126
    got = torch.empty(T, E, device=DEV)
    lib.balance_loss_backward(z.to(DEV), torch.from_numpy(idx).to(DEV), c, n, torch.full((1,), g, device=DEV), got, score=score, alpha=alpha)
    assert (np.abs(got.double().cpu().numpy() - dz) <= unit * (2 * Q(E, 6.0) + 8 * STEP) + 2.0 ** -126).all()
