"""The block-scaled layer as a whole: each step's result against 64-bit
arithmetic on what the step before it left (the operators themselves are pinned
in test_blockscale.py and test_gate.py; here it is that they are joined rightly).

Tolerances, fixed before the first run: the sums' bound of test_blockscale.py;
for the shared expert's and the routed products' total one more rounding per
term.
"""
import numpy as np
import pytest
import torch

from quantized_moe_amd import blockscale, lib

gpu = pytest.mark.gpu
DEV = "cuda:0"


def nb(n):
    return -(-n // 128)


def rows(q, s):
    return q.cpu().to(torch.float64) * s.cpu().double().repeat_interleave(128, 1)[:, : q.shape[1]]


def matrix(q, s):
    N, K = q.shape
    return q.cpu().to(torch.float64) * s.cpu().double().repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[:N]


def make_layer(E, d, f, k, shared_f, max_tokens, seed, **gate_kw):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    w = [blockscale.quantize_weight(0.05 * rnd(*s)) for s in ((E, f, d), (E, f, d), (E, d, f))]
    shared = None
    if shared_f:
        shared = [blockscale.quantize_weight(0.05 * rnd(*s)) for s in ((shared_f, d), (shared_f, d), (d, shared_f))]
    gate = lib.gate(E, k, bias=0.05 * rnd(E), **gate_kw)
    return blockscale.BlockScaleLayer(0.05 * rnd(E, d), gate, *w, shared=shared, max_tokens=max_tokens), rnd


def test_quantize_weight_on_the_cpu():
    rng = np.random.default_rng(1)
    for shape in ((128, 128), (200, 300), (3, 130, 144)):
        w = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
        q, s = blockscale.quantize_weight(w)
        assert q.shape == w.shape and s.shape == (*shape[:-2], nb(shape[-2]), nb(shape[-1]))
        v = q.float() * s.repeat_interleave(128, -1)[..., : shape[-1]].repeat_interleave(128, -2)[..., : shape[-2], :]
        step = 2.0 ** -4 * w.abs() + 2.0 ** -10 * float(s.max())
        assert ((v - w).abs() <= 1.001 * step).all()
        assert float(q.float().abs().max()) == 448.0


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
    idx, wt = layer.idx[:T].cpu(), layer.wt[:T].cpu()
    assert ((idx >= 0) & (idx < E)).all() and all(len(set(r)) == k for r in idx.tolist())
    assert torch.allclose(wt.sum(1), torch.full((T,), 1.5), rtol=1e-5)
    # the routes are the gate's, and the codes the quantiser's, of this x
    z, i2, w2 = torch.empty(T, E, device=DEV), torch.empty_like(layer.idx[:T]), torch.empty_like(layer.wt[:T])
    lib.router_logits(layer.w_router, x, z)
    lib.gate_topk(layer.gate, z, i2, w2)
    assert torch.equal(i2.cpu(), idx) and torch.equal(w2.cpu(), wt)
    xv = rows(layer.xq[:T], layer.xs[:T])
    assert ((xv - x.cpu().double()).abs() <= 2.0 ** -4 * x.cpu().double().abs()
            + 2.0 ** -10 * layer.xs[:T].cpu().double().repeat_interleave(128, 1)).all()
    # hidden rows by route, then y, from the layer's own codes
    pos, hv = layer.pos[: T * k].cpu(), rows(layer.hq[: T * k], layer.hs[: T * k])
    hs = layer.hs[: T * k].cpu().double().repeat_interleave(128, 1)[:, :f]
    ref, mag = torch.zeros(T, d, dtype=torch.float64), torch.zeros(T, d, dtype=torch.float64)
    tol = torch.zeros(T, d, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e, r = int(idx[t, j]), int(pos[t * k + j])
            gw, uw = matrix(layer.w_gate[0][e], layer.w_gate[1][e]), matrix(layer.w_up[0][e], layer.w_up[1][e])
            gate, up = gw @ xv[t], uw @ xv[t]
            h = gate * torch.sigmoid(gate) * up
            slack = 2.0 ** -14 * (gw.abs() @ xv[t].abs() * (1 + up.abs()) + uw.abs() @ xv[t].abs() * (1 + gate.abs()))
            assert ((hv[r] - h).abs() <= 2.0 ** -4 * h.abs() + 2.0 ** -10 * hs[r] + slack).all()
            dw = matrix(layer.w_down[0][e], layer.w_down[1][e])
            w = float(wt[t, j])
            ref[t] += w * (dw @ hv[r])
            m = w * (dw.abs() @ hv[r].abs())
            mag[t] += m
            tol[t] += (128 + nb(f) + 4) * 2.0 ** -23 * m
    if shared_f:
        sv = rows(layer.sq[:T], layer.ss[:T])
        dw = matrix(*layer.shared[2])
        ref += sv @ dw.t()
        m = sv.abs() @ dw.abs().t()
        mag += m
        tol += (128 + nb(shared_f) + 4) * 2.0 ** -23 * m
        gate, up = xv @ matrix(*layer.shared[0]).t(), xv @ matrix(*layer.shared[1]).t()
        h = gate * torch.sigmoid(gate) * up
        assert float((sv - h).norm() / h.norm()) < 2.0 ** -4
    tol += (k + 2) * 2.0 ** -23 * mag
    assert ((y.cpu().double() - ref).abs() <= tol).all()


@gpu
def test_forward_in_a_graph_and_with_masked_experts():
    layer, rnd = make_layer(16, 256, 128, 4, 128, 40, 3, score="softmax", n_groups=1, top_groups=1)
    layer.gate.bias_tensor[3:] = -float("inf")  # three experts left for four routes
    x, y = rnd(40, 256), torch.empty(40, 256, device=DEV)
    layer.forward(x, y)
    torch.cuda.synchronize()
    assert (layer.idx[:, 3] == -1).all() and (layer.wt[:, 3] == 0).all() and (layer.idx[:, :3] >= 0).all()
    want = y.clone()
    assert torch.isfinite(want).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, y)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        layer.forward(x, y)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_layer_refusals():
    layer = object.__new__(blockscale.BlockScaleLayer)
    layer.k, layer.max_tokens = 2, 4
    with pytest.raises(ValueError, match="made for 4"):
        layer.forward(torch.zeros(5, 256), None)
    with pytest.raises(ValueError, match="the router 8"):
        blockscale.BlockScaleLayer(torch.zeros(8, 256), lib.gate(4, 2), (torch.zeros(8, 128, 256), None), None, None)
