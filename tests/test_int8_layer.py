"""The int8 layer as a whole: each step's result against the definition on what the
step before it left (the operators themselves are pinned in test_int8.py and
test_balance.py; here it is that they are joined rightly).  Tolerances as there.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import int8, lib
from test_balance import Q, STEP, plain
from test_int8 import product, quantize, silu64

gpu = pytest.mark.gpu
DEV = "cuda:0"


def make_layer(E, d, f, k, shared_f, max_tokens, seed, max_sequences=1, **gate_kw):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    w = [int8.quantize_weight(0.05 * rnd(*s)) for s in ((E, f, d), (E, f, d), (E, d, f))]
    shared = None
    if shared_f:
        shared = [int8.quantize_weight(0.05 * rnd(*s)) for s in ((shared_f, d), (shared_f, d), (d, shared_f))]
    gate = lib.gate(E, k, bias=0.05 * rnd(E), **gate_kw)
    return int8.Int8Layer(0.05 * rnd(E, d), gate, *w, shared=shared, max_tokens=max_tokens, max_sequences=max_sequences), rnd


def test_quantize_weight_on_the_cpu():
    rng = np.random.default_rng(1)
    for shape in ((128, 128), (200, 300), (3, 130, 144)):
        w = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
        w[..., 0, :] = 0.0
        q, s = int8.quantize_weight(w)
        assert q.shape == w.shape and q.dtype == torch.int8 and s.shape == shape[:-1]
        # half a code, and the roundings of the scale and the quotient
        assert ((q.double() * s.double()[..., None] - w.double()).abs() <= (0.5 + 127 * 2.0 ** -22) * s.double()[..., None]).all()
        assert (q[..., 0, :] == 0).all() and (q[..., 1:, :].abs().amax(-1) == 127).all()


def n(t):
    return t.cpu().numpy()


@gpu
@pytest.mark.parametrize("T", [1, 2, 9, 70, 150])
@pytest.mark.parametrize("shared_f", [0, 144])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer(T, shared_f, dtype):
    E, d, f, k = 12, 512, 272, 3
    layer, rnd = make_layer(E, d, f, k, shared_f, 150, T, score="sigmoid", n_groups=4, top_groups=2, group_score="top2",
                            scale=1.5)
    x = rnd(T, d).to(dtype)
    y = torch.full((T, d), float("nan"), device=DEV)
    layer.forward(x, y)
    torch.cuda.synchronize()
    idx, wt, pos = n(layer.idx[:T]), n(layer.wt[:T]), n(layer.pos[: T * k])
    z, i2, w2 = torch.empty(T, E, device=DEV), torch.empty_like(layer.idx[:T]), torch.empty_like(layer.wt[:T])
    lib.router_logits(layer.w_router, x, z)
    lib.gate_topk(layer.gate, z, i2, w2)
    assert np.array_equal(n(i2), idx) and np.array_equal(n(w2), wt)
    xq, xs, h, hq, hs = (n(t) for t in (layer.xq[:T], layer.xs[:T], layer.h[: T * k], layer.hq[: T * k], layer.hs[: T * k]))
    for (q, s), v in ((quantize(n(x.float())), (xq, xs)), (quantize(h), (hq, hs))):
        assert np.array_equal(q, v[0]) and np.array_equal(s, v[1])
    ref, mag = np.zeros((T, d)), np.zeros((T, d))
    w = [(n(q), n(s)) for q, s in (layer.w_gate, layer.w_up, layer.w_down)]
    for t in range(T):
        for j in range(k):
            e, r = idx[t, j], pos[t * k + j]
            g, u = (product(xq[t: t + 1], xs[t: t + 1], q[e], s[e])[0].astype(np.float64) for q, s in w[:2])
            want = silu64(g) * u
            assert (np.abs(h[r] - want) <= np.abs(want) * (2 * np.abs(g) + 8) * STEP + 2.0 ** -125).all()
            term = wt[t, j].astype(np.float64) * product(hq[r: r + 1], hs[r: r + 1], w[2][0][e], w[2][1][e])[0]
            ref[t] += term
            mag[t] += np.abs(term)
    if shared_f:
        sh, sq, ss = n(layer.sh[:T]), n(layer.sq[:T]), n(layer.ss[:T])
        g, u = (product(xq, xs, n(q), n(s)).astype(np.float64) for q, s in layer.shared[:2])
        want = silu64(g) * u
        assert (np.abs(sh - want) <= np.abs(want) * (2 * np.abs(g) + 8) * STEP + 2.0 ** -125).all()
        q, s = quantize(sh)
        assert np.array_equal(q, sq) and np.array_equal(s, ss)
        add = product(sq, ss, n(layer.shared[2][0]), n(layer.shared[2][1]))
        assert np.array_equal(n(layer.add[:T]), add)
        ref, mag = ref + add, mag + np.abs(add)
    assert (np.abs(n(y) - ref) <= (k + 1) * STEP * mag).all()


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [5, 150])
def test_balance_of_a_forward_call(T, score):
    """Padding, as tokens of which every expert is masked, is in no count."""
    E, d, k = 12, 256, 3
    layer, rnd = make_layer(E, d, 64, k, 0, 150, T, max_sequences=3, score=score)
    x, y = rnd(T, d), torch.empty(T, d, device=DEV)
    layer.forward(x, y)
    starts = torch.tensor([0, T // 3, T // 3, T - 1], dtype=torch.int32, device=DEV)
    for st in (None, starts):
        counts, tokens, loss = layer.balance(T, alpha=0.5, starts=st)
        cuts = [0, T] if st is None else st.tolist()
        z, idx = n(layer.z[:T]).astype(np.float64), n(layer.idx[:T])
        c, m, want, _, _ = plain(z, idx, cuts, score, 0.5)
        assert np.array_equal(n(counts), c) and np.array_equal(n(tokens), m)
        assert (np.abs(n(loss) - want) <= want * (Q(E, np.abs(z).max()) + STEP)).all()
        if st is None:
            assert np.array_equal(n(counts)[0], n(layer.counts))  # as the bucketing counts them


@gpu
def test_forward_in_a_graph_and_with_masked_experts():
    layer, rnd = make_layer(16, 256, 128, 4, 128, 40, 3, score="softmax", n_groups=1, top_groups=1)
    layer.gate.bias_tensor[3:] = -float("inf")  # three experts left for four routes
    x, y = rnd(40, 256), torch.empty(40, 256, device=DEV)
    layer.forward(x, y)
    balance = [t.clone() for t in layer.balance(40)]
    torch.cuda.synchronize()
    assert (layer.idx[:, 3] == -1).all() and (layer.idx[:, :3] >= 0).all() and (balance[0][0, :3] == 40).all()
    want = y.clone()
    assert torch.isfinite(want).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, y)
        got = layer.balance(40)
    for _ in range(3):
        y.zero_()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip(got, balance))
        layer.forward(x, y)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_layer_refusals():
    layer = object.__new__(int8.Int8Layer)
    layer.k, layer.max_tokens, layer.max_sequences = 2, 4, 1
    with pytest.raises(ValueError, match="made for 4"):
        layer.forward(torch.zeros(5, 256), None)
    with pytest.raises(ValueError, match="made for 4 in 1"):
        layer.balance(5)
    with pytest.raises(ValueError, match="made for 4 in 1"):
        layer.balance(4, starts=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="the router 8"):
        int8.Int8Layer(torch.zeros(8, 256), lib.gate(4, 2), (torch.zeros(8, 128, 256), None), None, None)


@gpu
def test_example_runs_and_gives_the_routers_gradient():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "int8_layer.py")
    spec = importlib.util.spec_from_file_location("int8_layer_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    grad = example.main(["--experts", "16", "--width", "256", "--hidden", "128", "--tokens", "1,40"])
    assert grad.shape == (16, 256) and torch.isfinite(grad).all() and float(grad.norm()) > 0
