"""The differentiable balance loss in a program's hands: buffers that later calls write over.
Tolerances as in test_balance.py.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import balance, lib
from test_balance import Q, STEP, make, plain

gpu = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def calls_on_the_cpu(monkeypatch):
    """The library's two balance calls replaced: the routes that each of them was given."""
    got = {"forward": [], "backward": []}

    def forward(z, idx, counts, tokens, loss, work, score, alpha, starts):
        got["forward"].append(idx.clone())
        counts.zero_(), tokens.zero_(), loss.zero_()

    def backward(z, idx, counts, tokens, grad_loss, dz, score, alpha, starts):
        got["backward"].append(idx.clone())
        dz.zero_()

    monkeypatch.setattr(lib, "balance_loss", forward)
    monkeypatch.setattr(lib, "balance_loss_backward", backward)
    monkeypatch.setattr(lib, "balance_loss_workspace_bytes", lambda *a: 0)
    return got


def test_gradient_of_overwritten_routes_on_the_cpu(calls_on_the_cpu):
    """Routes that a kernel wrote over, which torch cannot know of: the backward call gets those of its forward call."""
    idx = torch.tensor([[0, 1], [-1, -1]], dtype=torch.int32)
    z = torch.zeros(2, 4, requires_grad=True)
    loss, _, _ = balance.balance_loss(z, idx)
    idx.numpy()[:] = [[-1, -1], [2, 3]]
    loss.sum().backward()
    assert calls_on_the_cpu["backward"][0].tolist() == [[0, 1], [-1, -1]]


def gradient(z, idx, starts, score, alpha, weights):
    """The definition's gradient and what a value of it may be off by."""
    dz, unit = plain(z.double().numpy(), idx, starts, score, alpha, weights)[3:]
    return dz, unit * (2 * Q(z.shape[1], 6.0) + 8 * STEP) + 2.0 ** -126


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [60, 700])
def test_two_micro_batches_over_one_buffer_of_routes(T, score):
    """Two batches through one gate's buffers, then one backward pass: padding lies elsewhere in each."""
    rng = np.random.default_rng(T)
    E, k = 24, 3
    gate = lib.gate(E, k, score=score)
    idx, wt = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    total, batches = 0.0, []
    for first in (0, T // 2):
        z = make(rng, T, E, k, 1, mask=0)[0]
        z[first: first + T // 4] = -float("inf")      # no route
        leaf = z.to(DEV).requires_grad_()
        lib.gate_topk(gate, leaf.detach(), idx, wt)
        total = total + balance.balance_loss(leaf, idx, score=score, alpha=0.3)[0].sum()
        batches.append((z, leaf, idx.cpu().numpy()))
    total.backward()
    for z, leaf, routes in batches:
        assert ((routes < 0).all(1)).sum() == T // 4
        want, tol = gradient(z, routes, [0, T], score, 0.3, np.ones(1))
        assert (np.abs(leaf.grad.double().cpu().numpy() - want) <= tol).all()


@gpu
@pytest.mark.parametrize("how", ["router_logits", "int8_matmul", "blockscale_matmul", "balance_loss"])
def test_values_that_were_written_over_are_refused(how):
    """Logits in a buffer of the library's calls, and the counts that were returned: another call's outputs in
    their place stop the backward pass."""
    T, E, d, k = 40, 16, 256, 3
    i8 = lambda *n: torch.ones(*n, dtype=torch.int8, device=DEV)  # noqa: E731
    f = lambda *n: torch.ones(*n, device=DEV)  # noqa: E731
    z, idx = torch.randn(T, E, device=DEV), torch.zeros(T, k, dtype=torch.int32, device=DEV)
    leaf = z.detach().requires_grad_()                 # (its gradient is the router's to use)
    loss, counts, tokens = balance.balance_loss(leaf, idx)
    if how == "router_logits":
        lib.router_logits(f(E, d), f(T, d), z)
    elif how == "int8_matmul":
        lib.int8_matmul(i8(T, d), f(T), i8(E, d), f(E), z)
    elif how == "blockscale_matmul":
        lib.blockscale_matmul(i8(T, d).view(torch.uint8), f(T, 2), i8(E, d).view(torch.uint8), f(1, 2), z)
    else:
        lib.balance_loss(torch.randn(T, E, device=DEV), idx, counts, tokens, torch.empty(1, device=DEV), None)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()


@gpu
def test_inputs_and_refused_calls_do_not_count_as_written():
    T, E = 5, 8
    z, idx = torch.randn(T, E, device=DEV), torch.zeros(T, 2, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    out = [torch.empty(1, E, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV), torch.empty(1, device=DEV)]
    versions = lambda: [t._version for t in (z, idx, starts, *out)]  # noqa: E731
    old = versions()
    with pytest.raises(lib.MoeError, match="alpha"):
        lib.balance_loss(z, idx, *out, None, alpha=float("inf"), starts=starts)
    assert versions() == old
    lib.balance_loss(z, idx, *out, None, starts=starts)
    assert versions() == [v + (i > 2) for i, v in enumerate(old)]
    with torch.inference_mode():
        more = [torch.empty_like(t) for t in out]
        lib.balance_loss(z, idx, *more, None, starts=starts)
        assert all(torch.equal(a, b) for a, b in zip(out, more))
        logits = torch.empty(T, E, device=DEV)
        lib.router_logits(torch.ones(E, 256, device=DEV), torch.ones(T, 256, device=DEV), logits)
    lib.balance_loss(z, idx, *more, None, starts=starts)   # tensors without a version, outside of that mode
    lib.router_logits(torch.ones(E, 256, device=DEV), torch.ones(T, 256, device=DEV), logits)
    assert (logits == 256).all()


def test_strides_on_the_cpu(calls_on_the_cpu, monkeypatch):
    """Rows that overlap, columns with gaps, routes and starts that are columns of something: the calls get rows one after another."""
    inner, seen = lib.balance_loss, []
    monkeypatch.setattr(lib, "balance_loss", lambda z, idx, *a, **kw: (seen.append((z, idx, kw["starts"])), inner(z, idx, *a, **kw)))
    starts = torch.tensor([[0, 2], [2, 3], [5, 5]], dtype=torch.int32)[:, 0]
    for z in (torch.zeros(1, 6).expand(5, 6), torch.zeros(1, 1).expand(5, 1), torch.zeros(30).as_strided((5, 6), (3, 1)),
              torch.zeros(6, 5).t(), torch.zeros(5, 12)[:, ::2], torch.zeros(5, 9)[:, :6]):
        balance.balance_loss(z.requires_grad_(), torch.zeros(5, 2, dtype=torch.int32)[:, ::2], starts=starts)
    assert len(seen) == 6
    for z, idx, st in seen:
        assert (z.stride(1) == 1 or z.shape[1] == 1) and z.stride(0) >= z.shape[1] and idx.is_contiguous() and st.tolist() == [0, 2, 5]
        assert st.is_contiguous()
    assert seen[-1][0].stride(0) == 9  # (rows further apart are taken as they are)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [50, 600])
def test_expanded_logits(T, score):
    """One row of logits for every token, as a bias of the router gives them: its gradient is the sum over the tokens."""
    rng = np.random.default_rng(T)
    E, k = 12, 2
    idx = make(rng, T, E, k, 1)[1]
    row = torch.from_numpy(rng.standard_normal((1, E)).astype(np.float32))
    leaf = row.to(DEV).requires_grad_()
    routes = torch.from_numpy(np.repeat(idx, 2, 1)).to(DEV)[:, ::2]
    starts = torch.tensor([0, 9, T // 3, 9, T, 9], dtype=torch.int32, device=DEV)[::2]
    loss, counts, tokens = balance.balance_loss(leaf.expand(T, E), routes, score=score, starts=starts)
    z = row.expand(T, E).contiguous()
    c, n, want, dz, unit = plain(z.double().numpy(), idx, [0, T // 3, T], score, 1.0, np.ones(2))
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(tokens.cpu().numpy(), n)
    assert (np.abs(loss.detach().cpu().numpy() - want) <= want * (Q(E, 6.0) + STEP)).all()
    loss.sum().backward()
    tol = unit * (2 * Q(E, 6.0) + 8 * STEP) + 2.0 ** -126
    # torch's sum over the rows: at most T fp32 additions of the terms' magnitudes
    assert (np.abs(leaf.grad.double().cpu().numpy() - dz.sum(0)) <= tol.sum(0) + T * STEP * np.abs(dz).sum(0)).all()


@gpu
@pytest.mark.parametrize("S", [1, 2000])
def test_a_batch_without_tokens(S):
    """No rows at all: losses of 0 and a gradient of no rows; without a gradient to take, the same."""
    E = 16
    starts = None if S == 1 else torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    idx = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    leaf = torch.empty(0, E, device=DEV, requires_grad=True)
    loss, counts, tokens = balance.balance_loss(leaf, idx, starts=starts)
    loss.sum().backward()
    assert loss.shape == (S,) and not loss.any() and not counts.any() and not tokens.any() and leaf.grad.shape == (0, E)
    with torch.no_grad():
        assert not balance.balance_loss(leaf, idx, starts=starts)[0].requires_grad
