"""The balance loss, its counts and its gradient against 64-bit arithmetic on the CPU.

Tolerances, fixed before the first run, in units of 2^-24 (a rounding to nearest is
off by at most one): with |z| <= Z among the experts that are in,

* a softmax term e^(z - m): the difference 2 Z, the constant and its product 4 Z,
  the exponential 2: 6 Z + 2; a sigmoid: 2 Z + 2 for the exponential, 4 more;
* a sum of E terms over 64 lanes: E / 64 + 6 additions; sum and weighted sum both
  carry a term's error, and their quotient one: Q = 2 (6 Z + 4) + 2 (E / 64 + 7) + 1;
* the loss is a sum of such quotients of one sign (64 bits) rounded once: Q + 2;
* a gradient is p (c - q) times a factor of 5 roundings: (term, sum) + 5 of p (c + q), and Q of p q;
  bf16 outputs 2^-8 of the value more.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import lib

gpu = pytest.mark.gpu
DEV = "cuda:0"
STEP = 2.0 ** -24
LOW = -(2.0 ** 127)


def plain(z, idx, starts, score, alpha, grad=None):
    """counts, tokens, loss, dz, p and the unit of p (c + q) factor, a sequence at a time in 64 bits."""
    T, E = z.shape
    k = idx.shape[1]
    S = len(starts) - 1
    counts, tokens, loss = np.zeros((S, E), np.int64), np.zeros(S, np.int64), np.zeros(S)
    dz, unit = np.zeros((T, E)), np.zeros((T, E))
    out = np.isnan(z) | (z <= LOW)
    z = np.minimum(np.where(out, 0.0, z), np.finfo(np.float32).max)
    for s in range(S):
        rows = [t for t in range(starts[s], starts[s + 1]) if ((idx[t] >= 0) & (idx[t] < E)).any()]
        n = tokens[s] = len(rows)
        if n == 0:
            continue
        for t in rows:
            for e in idx[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        a, slope = np.zeros((n, E)), np.ones((n, E))
        for i, t in enumerate(rows):
            live = ~out[t]
            if not live.any():
                continue
            if score == "softmax":
                a[i, live] = np.exp(z[t, live] - z[t, live].max())
            else:
                zc = np.clip(z[t, live], -80, 80)
                a[i, live], slope[i, live] = 1 / (1 + np.exp(-zc)), 1 / (1 + np.exp(zc))
        total = a.sum(1, keepdims=True)
        p = np.divide(a, total, out=np.zeros_like(a), where=total > 0)
        loss[s] = alpha * E * np.sum(counts[s] / (k * n) * p.sum(0) / n)
        if grad is not None:
            coef = grad[s] * alpha * E / (k * n * n)
            q = p @ counts[s]
            dz[rows] = coef * p * (counts[s] - q[:, None]) * slope
            unit[rows] = abs(coef) * p * (counts[s] + q[:, None]) * slope
    return counts, tokens, loss, dz, unit


def Q(E, Z):
    return (2 * (6 * Z + 4) + 2 * (E / 64 + 7) + 3) * STEP


def make(rng, T, E, k, S, mask=0.05, dtype=torch.float32, Z=6.0):
    z = torch.from_numpy(np.clip(rng.standard_normal((T, E)) * 2, -Z, Z).astype(np.float32))
    if mask:
        u = rng.random((T, E))
        z[torch.from_numpy(u < mask)] = -np.inf
        z[torch.from_numpy((u >= mask) & (u < 1.5 * mask))] = torch.finfo(dtype).min
        z[torch.from_numpy((u >= 1.5 * mask) & (u < 1.7 * mask))] = np.nan
        z[torch.from_numpy(rng.random(T) < mask)] = -np.inf
    z = z.to(dtype)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    if T:
        idx[rng.random((T, k)) < 0.1] = -1
        idx[rng.random(T) < 0.1] = -1
        idx[rng.random((T, k)) < 0.02] = E + 3          # no expert either
    cuts = np.sort(rng.integers(0, T + 1, S + 1)) if S > 1 else np.array([0, T])
    if S > 2:
        cuts[1] = cuts[0]                               # an empty sequence
    return z, idx, cuts.astype(np.int32)


def forward(z, idx, starts, score, alpha, S, explicit=True):
    E = z.shape[1]
    c, n = torch.full((S, E), -7, dtype=torch.int32, device=DEV), torch.full((S,), -7, dtype=torch.int32, device=DEV)
    loss = torch.full((S,), float("nan"), device=DEV)
    need = lib.balance_loss_workspace_bytes(z.shape[0], S, E)
    work = torch.full((need,), 0x7f, dtype=torch.uint8, device=DEV) if need else None
    st = torch.from_numpy(starts).to(DEV) if explicit else None
    lib.balance_loss(z, torch.from_numpy(idx).to(DEV), c, n, loss, work, score=score, alpha=alpha, starts=st)
    torch.cuda.synchronize()
    return c, n, loss, st


CASES = [(0, 8, 2, 1), (0, 16, 2, 2000), (128, 384, 6, 32), (128, 384, 6, 33), (129, 384, 6, 3), (3, 5, 5, 1700), (4097, 9, 3, 1500), (1, 1, 1, 1), (1, 384, 6, 1), (5, 3, 2, 2), (64, 384, 6, 1), (70, 64, 4, 3), (300, 65, 16, 7), (257, 1000, 8, 2),
         (1024, 384, 6, 5), (1500, 130, 3, 200), (2100, 200, 6, 1), (9000, 16, 2, 300), (20000, 40, 2, 1)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S", CASES)
def test_loss_and_gradient(T, E, k, S, score, dtype):
    rng = np.random.default_rng(T + E + S)
    z, idx, starts = make(rng, T, E, k, S, dtype=dtype)
    alpha = 0.7
    grad = rng.standard_normal(S).astype(np.float32)
    zbuf = torch.zeros(T, E + 5, dtype=dtype, device=DEV)[:, 3: 3 + E]
    zbuf.copy_(z)
    c, n, loss, st = forward(zbuf, idx, starts, score, alpha, S, explicit=S > 1)
    counts, tokens, want, dz, unit = plain(z.double().numpy(), idx, starts, score, alpha, grad)
    assert np.array_equal(c.cpu().numpy(), counts) and np.array_equal(n.cpu().numpy(), tokens)
    assert (np.abs(loss.cpu().numpy() - want) <= want * (Q(E, 6.0) + STEP)).all()
    got = torch.full((T, E + 2), 9.0, dtype=dtype, device=DEV)
    lib.balance_loss_backward(zbuf, torch.from_numpy(idx).to(DEV), c, n, torch.from_numpy(grad).to(DEV), got[:, :E], score=score,
                              alpha=alpha, starts=st)
    torch.cuda.synchronize()
    tol = unit * (2 * Q(E, 6.0) + 8 * STEP) + (np.abs(dz) * 2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0)
    assert (np.abs(got[:, :E].double().cpu().numpy() - dz) <= tol + 2.0 ** -126).all()
    assert (got[:, E:] == 9.0).all()


def test_formula_against_differences():
    """The gradient that the GPU's is compared with, by central differences of the loss in 64 bits."""
    rng = np.random.default_rng(1)
    for score in ("softmax", "sigmoid"):
        z, idx, starts = make(rng, 7, 6, 2, 2)
        z = z.double().numpy()
        grad = np.array([0.3, -1.2])
        dz = plain(z, idx, starts, score, 0.7, grad)[3]
        for t in range(7):
            for e in range(6):
                if not np.isfinite(z[t, e]) or z[t, e] <= LOW:
                    assert dz[t, e] == 0
                    continue
                ends = []
                for h in (1e-5, -1e-5):
                    v = z.copy()
                    v[t, e] += h
                    ends.append(plain(v, idx, starts, score, 0.7)[2] @ grad)
                # the difference is off by h^2 / 6 of the third derivative and by the values' last bits over 2 h
                assert abs((ends[0] - ends[1]) / 2e-5 - dz[t, e]) <= 1e-9


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(score):
    """Infinities count as the largest number; far logits give probabilities of 0 and 1, no NaN."""
    big = 3e38
    z = torch.tensor([[np.inf, np.inf, 0.0, -np.inf], [big, -1e38, 5.0, np.nan], [90.0, -90.0, 0.0, 0.0], [-100.0, -120.0, -90.0, -85.0],
                      [-1e38, -1e38, -1.5e38, -1e38]], dtype=torch.float32)
    idx = np.array([[0, 1], [0, 2], [0, 2], [3, 2], [0, 1]], np.int32)
    starts = np.array([0, 5], np.int32)
    c, n, loss, _ = forward(z.to(DEV), idx, starts, score, 1.0, 1)
    _, _, want, dz, unit = plain(z.double().numpy(), idx, starts, score, 1.0, np.ones(1))
    assert abs(float(loss) - want[0]) <= want[0] * Q(4, 100.0)
    got = torch.empty(5, 4, device=DEV)
    lib.balance_loss_backward(z.to(DEV), torch.from_numpy(idx).to(DEV), c, n, torch.ones(1, device=DEV), got, score=score)
    assert (np.abs(got.double().cpu().numpy() - dz) <= unit * 2 * Q(4, 100.0) + 2.0 ** -126).all()


@gpu
def test_large_gradients_of_far_logits():
    """Every sigmoid at its smallest, e^-80: the probabilities are those of equal logits, whatever the sequence's gradient."""
    z = torch.full((1, 3), -90.0, device=DEV)
    idx = np.array([[0, 1]], np.int32)
    c, n, _, _ = forward(z, idx, np.array([0, 1], np.int32), "sigmoid", 1.0, 1)
    for g in (1e-20, 1.0, 1e30):
        got = torch.empty(1, 3, device=DEV)
        lib.balance_loss_backward(z, torch.from_numpy(idx).to(DEV), c, n, torch.full((1,), g, device=DEV), got, score="sigmoid")
        _, _, _, dz, unit = plain(z.cpu().double().numpy(), idx, [0, 1], "sigmoid", 1.0, np.array([g]))
        assert np.abs(dz).max() > 0.1 * g
        assert (np.abs(got.double().cpu().numpy() - dz) <= unit * 2 * Q(3, 80.0)).all()


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,empty", [(8195, 3), (16449, 100), (65529, 1)])
def test_empty_sequences_at_the_end(T, empty, score):
    """Sequences that begin where the last token ends, with several tokens a wave and a last
    wave that has fewer: they have no partial sum (and no place in the workspace) of their own."""
    rng = np.random.default_rng(T)
    z, idx, _ = make(rng, T, 24, 3, 1)
    starts = np.array([0, 0, T // 3, T // 3, T - 1] + [T] * (empty + 1), np.int32)
    S = len(starts) - 1
    c, n, loss, _ = forward(z.to(DEV), idx, starts, score, 0.5, S)
    rc, rn, rl, _, _ = plain(z.double().numpy(), idx, starts, score, 0.5)
    assert (c.cpu().numpy() == rc).all() and (n.cpu().numpy() == rn).all()
    got = loss.double().cpu().numpy()
    assert (got[rn == 0] == 0).all()
    assert (np.abs(got - rl) <= rl * (Q(24, 6.0) + STEP)).all()


@gpu
def test_even_load_gives_alpha():
    """Every expert asked for alike: the loss is alpha and no logit is pushed."""
    T, E = 512, 64
    idx = np.stack([(np.arange(2) * 32 + t) % E for t in range(T)]).astype(np.int32)
    z = torch.zeros(T, E, device=DEV)
    for score in ("softmax", "sigmoid"):
        c, n, loss, st = forward(z, idx, np.array([0, T], np.int32), score, 0.25, 1)
        assert float(loss) == 0.25 and (c == 16).all() and int(n) == T
        dz = torch.empty_like(z)
        lib.balance_loss_backward(z, torch.from_numpy(idx).to(DEV), c, n, torch.ones(1, device=DEV), dz, score=score, alpha=0.25)
        assert (dz == 0).all()


# ------------------------------------------------------- the torch function ----
@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,S", [(40, 3), (700, 4)])
def test_autograd(T, S, score, dtype):
    """balance.balance_loss as a training step uses it: with other terms of z, weights per sequence, logits that are not contiguous."""
    from quantized_moe_amd import balance

    rng = np.random.default_rng(T)
    E, k = 24, 3
    z, idx, starts = make(rng, T, E, k, S, dtype=dtype)
    weights = rng.standard_normal(S).astype(np.float32)
    leaf = z.t().contiguous().to(DEV).requires_grad_()          # z itself is its transpose
    st, wt = torch.from_numpy(starts).to(DEV), torch.from_numpy(weights).to(DEV)
    loss, counts, tokens = balance.balance_loss(leaf.t(), torch.from_numpy(idx).to(DEV), score=score, alpha=0.3, starts=st)
    assert loss.requires_grad and not counts.requires_grad and not tokens.requires_grad
    (loss * wt).sum().backward()
    c, n, want, dz, unit = plain(z.double().numpy(), idx, starts, score, 0.3, weights)
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(tokens.cpu().numpy(), n)
    assert (np.abs(loss.detach().cpu().numpy() - want) <= want * (Q(E, 6.0) + STEP)).all()
    tol = unit * (2 * Q(E, 6.0) + 8 * STEP) + (np.abs(dz) * 2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0)
    assert (np.abs(leaf.grad.t().double().cpu().numpy() - dz) <= tol + 2.0 ** -126).all()
    # the mean over sequences: a broadcast gradient
    leaf.grad = None
    balance.balance_loss(leaf.t(), torch.from_numpy(idx).to(DEV), score=score, alpha=0.3, starts=st)[0].mean().backward()
    dz, unit = plain(z.double().numpy(), idx, starts, score, 0.3, np.full(S, 1 / S, np.float32))[3:]
    tol = unit * (2 * Q(E, 6.0) + 8 * STEP) + (np.abs(dz) * 2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0)
    assert (np.abs(leaf.grad.t().double().cpu().numpy() - dz) <= tol + 2.0 ** -126).all()


@gpu
def test_gradient_against_differences_on_the_gpu():
    """Central differences of the kernel's own loss, over a step of 1/16: they are off by h^2 / 6 of the third derivative, which
    is at most 6 of the loss's share of a token, and by the loss's rounding over 2 h."""
    rng = np.random.default_rng(4)
    T, E, k, h = 6, 8, 2, 2.0 ** -4
    for score in ("softmax", "sigmoid"):
        z, idx, starts = make(rng, T, E, k, 1, mask=0)
        c, n, loss, _ = forward(z.to(DEV), idx, starts, score, 1.0, 1)
        dz = torch.empty(T, E, device=DEV)
        lib.balance_loss_backward(z.to(DEV), torch.from_numpy(idx).to(DEV), c, n, torch.ones(1, device=DEV), dz, score=score)
        share = E * float(c.max()) / (k * float(n) ** 2)
        for t in range(T):
            for e in range(E):
                ends = []
                for d in (h, -h):
                    v = z.clone()
                    v[t, e] += d
                    ends.append(float(forward(v.to(DEV), idx, starts, score, 1.0, 1)[2]))
                assert abs((ends[0] - ends[1]) / (2 * h) - float(dz[t, e])) <= h * h * share + float(loss) * (Q(E, 6.0) + STEP) / h


@gpu
def test_step_in_a_graph():
    """Forward and backward captured, replayed on new logits with eager calls between."""
    rng = np.random.default_rng(9)
    T, E, k = 900, 72, 4
    z, idx, starts = make(rng, T, E, k, 5)
    zg, ig, st = z.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(starts).to(DEV)
    c, n, loss = torch.empty(5, E, dtype=torch.int32, device=DEV), torch.empty(5, dtype=torch.int32, device=DEV), torch.empty(5, device=DEV)
    work = torch.empty(lib.balance_loss_workspace_bytes(T, 5, E), dtype=torch.uint8, device=DEV)
    dz, g = torch.empty_like(zg), torch.ones(5, device=DEV)

    def step():
        lib.balance_loss(zg, ig, c, n, loss, work, starts=st)
        lib.balance_loss_backward(zg, ig, c, n, g, dz, starts=st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        zg.copy_(z.roll(i, 0))
        ig.copy_(torch.from_numpy(np.roll(idx, 7 * i, 0)))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (c, n, loss, dz)]
        for t in (c, n, loss, dz):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((c, n, loss, dz), want))


@gpu
def test_identical_calls_give_identical_bits():
    rng = np.random.default_rng(10)
    for T, S in ((100, 3), (5000, 1), (5000, 70)):
        z, idx, starts = make(rng, T, 96, 4, S)
        first = forward(z.to(DEV), idx, starts, "softmax", 1.0, S)
        for _ in range(5):
            again = forward(z.to(DEV), idx, starts, "softmax", 1.0, S)
            assert all(torch.equal(a, b) for a, b in zip(first[:3], again[:3]))
