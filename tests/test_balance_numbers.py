"""The balance calls' numbers, from Python on."""
import pytest

from quantized_moe_amd import lib
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
