"""The gate (scores, groups, top-k of given logits) against a plain program.

Selections are compared exactly: the definition fixes every fp32 step that
orders the experts.  Weights are compared with 64-bit scores.  Their error,
fixed before the first run: the score sequences are within 4e-7 of the exact
functions, a softmax sum of E terms adds (E / 64 + 6) 2^-24 and its division
2^-24, the renormalising sum and division (k + 1) 2^-24: 4e-6 covers them.
"""
import math

import numpy as np
import pytest
import torch

from quantized_moe_amd import lib

gpu = pytest.mark.gpu
DEV = "cuda:0"
WT_REL = 4e-6
f4 = np.float32


# ------------------------------------------------------------ CPU reference ----
def exp32(t):
    n = (t * f4(float.fromhex("0x1.715476p0")) + f4(1.5 * 2 ** 23)) - f4(1.5 * 2 ** 23)
    r = (t - n * f4(float.fromhex("0x1.62e400p-1"))) - n * f4(float.fromhex("0x1.7f7d1cp-20"))
    p = f4(float.fromhex("0x1.6c16c2p-10"))
    for c in ("0x1.111112p-7", "0x1.555556p-5", "0x1.555556p-3", "0x1p-1", "0x1p0", "0x1p0"):
        p = p * r + f4(float.fromhex(c))
    return np.ldexp(p, int(n))


def gate_row(z, k, score, G, KG, group_score, renorm, scale, bias):
    """One token, expert by expert, as the definition reads."""
    E = len(z)
    live = [e for e in range(E) if z[e] > -(2.0 ** 127)]  # (false for NaN)
    z = np.minimum(z, np.finfo(f4).max).astype(f4)
    s, s64 = {}, {}
    if score == "sigmoid":
        for e in live:
            zc = f4(min(max(z[e], f4(-80)), f4(80)))
            s[e] = f4(1) / (f4(1) + exp32(-zc))
            s64[e] = 1.0 / (1.0 + math.exp(-float(zc)))
    elif live:
        m = max(z[e] for e in live)
        with np.errstate(over="ignore"):
            u = {e: max(f4(z[e] - m), f4(-80)) for e in live}
        part = np.zeros(64, f4)
        for e in live:
            part[e % 64] += exp32(u[e])
        step = 32
        while step:
            part[:step] = part[:step] + part[step: 2 * step]
            step //= 2
        total64 = sum(math.exp(float(u[e])) for e in live)
        for e in live:
            s[e] = exp32(u[e]) / part[0]
            s64[e] = math.exp(float(u[e])) / total64
    v = {}
    for e in live:
        if bias is not None:
            v[e] = f4(s[e] + bias[e])
        elif KG < G and group_score == "top2":
            v[e] = s[e]
        else:
            v[e] = z[e]
    v = {e: x for e, x in v.items() if x > -math.inf}
    if KG < G:
        values = {}
        for g in range(G):
            own = sorted((v[e] for e in v if e // (E // G) == g), reverse=True)
            if own:
                values[g] = f4(own[0] + own[1]) if group_score == "top2" and len(own) > 1 else own[0]
        kept = sorted(values, key=lambda g: (-values[g], g))[:KG]
        v = {e: x for e, x in v.items() if e // (E // G) in kept}
    chosen = sorted(v, key=lambda e: (-v[e], e))[:k]
    total = sum(s64[e] for e in chosen)
    w = [s64[e] / (total if renorm else 1.0) * scale for e in chosen]
    pad = k - len(chosen)
    return chosen + [-1] * pad, w + [0.0] * pad


def check(z, k, score, G, KG, group_score, renorm, scale, bias, z_dev=None):
    T, E = z.shape
    g = lib.gate(E, k, score=score, n_groups=G, top_groups=KG, group_score=group_score, renormalize=renorm, scale=scale,
                 bias=None if bias is None else torch.from_numpy(bias).to(DEV))
    zd = z.to(DEV) if z_dev is None else z_dev
    idx = torch.full((T, k), 12345, dtype=torch.int32, device=DEV)
    wt = torch.full((T, k), math.nan, device=DEV)
    lib.gate_topk(g, zd, idx, wt)
    torch.cuda.synchronize()
    idx, wt = idx.cpu().numpy(), wt.cpu().numpy()
    zf = z.float().numpy()
    for t in range(T):
        want_i, want_w = gate_row(zf[t], k, score, G, KG, group_score, renorm, scale, bias)
        assert idx[t].tolist() == want_i, (t, idx[t].tolist(), want_i)
        assert np.allclose(wt[t], want_w, rtol=WT_REL, atol=1e-37), (t, wt[t], want_w)


CASES = [
    # E, k, G, KG, group score
    (1, 1, 1, 1, "max"), (2, 2, 2, 2, "top2"), (5, 3, 5, 3, "top2"), (8, 2, 4, 2, "max"), (64, 6, 8, 3, "top2"),
    (65, 5, 1, 1, "max"), (100, 8, 10, 4, "top2"), (96, 4, 3, 1, "max"), (128, 8, 64, 8, "top2"), (256, 8, 8, 4, "top2"),
    (257, 16, 1, 1, "max"), (384, 6, 8, 4, "top2"), (384, 6, 1, 1, "max"), (512, 16, 4, 2, "max"), (1024, 10, 16, 5, "top2"),
    (1000, 7, 40, 11, "top2"), (60, 16, 6, 3, "top2"),
]


@gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,KG,group_score", CASES)
def test_gate(E, k, G, KG, group_score, score):
    rng = np.random.default_rng(E * 31 + k)
    for dtype in (torch.float32, torch.bfloat16):
        for with_bias in (False, True):
            z = torch.from_numpy((2 * rng.standard_normal((9, E))).astype(f4)).to(dtype)
            bias = (0.1 * rng.standard_normal(E)).astype(f4) if with_bias else None
            check(z, k, score, G, KG, group_score, with_bias == (dtype == torch.float32), 2.5 if with_bias else 1.0, bias)


@gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_masks_and_extremes(score, with_bias):
    rng = np.random.default_rng(3)
    E, k, G, KG = 48, 6, 6, 2
    lowest = {torch.float32: np.finfo(f4).min, torch.bfloat16: float(torch.finfo(torch.bfloat16).min)}
    for dtype in (torch.float32, torch.bfloat16):
        z = np.round(2 * rng.standard_normal((40, E))).astype(f4)       # many equal logits
        z[0] = 0.0                                                      # all equal
        z[1] = -math.inf                                                # nothing left
        z[2] = lowest[dtype]
        z[3] = math.nan
        z[4, 2:] = -math.inf                                            # fewer than k
        z[5, :] = -math.inf
        z[5, [7, 8, 30, 40, 41]] = [1, 1, 1, 1, 1]                      # groups of one and two
        z[6, 5], z[6, 9] = math.inf, math.inf
        z[7] = -100.0 - np.arange(E)                                    # every sigmoid at its floor
        z[8] = 90.0 + np.arange(E)
        z[9, ::2] = -0.0
        z[9, 1::2] = 0.0
        z[10, 3] = math.nan
        z[11, 4] = 3e38
        z[11, 5:9] = -1.5e38                                            # low, but not masked
        z[12, :] = lowest[dtype]
        z[12, 47] = -1e38
        bias = None
        if with_bias:
            bias = (np.round(4 * rng.standard_normal(E)) / 8).astype(f4)
            bias[[1, 20]] = -math.inf
            bias[2] = math.nan
            bias[30] = math.inf
        for gs in ("max", "top2"):
            for renorm in (False, True):
                for G_, KG_ in ((G, KG), (1, 1), (G, G)):
                    check(torch.from_numpy(z).to(dtype), k, score, G_, KG_, gs, renorm, 1.5, bias)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_logits(dtype):
    rng = np.random.default_rng(4)
    T, E = 37, 77
    buf = torch.full((T, E + 6), math.inf, dtype=dtype, device=DEV)
    z = torch.from_numpy(rng.standard_normal((T, E)).astype(f4)).to(dtype)
    for first in (0, 1, 3, 5):
        view = buf[:, first: first + E]
        view.copy_(z)
        check(z, 5, "softmax", 7, 3, "top2", True, 1.0, None, z_dev=view)
        buf.fill_(math.inf)


@gpu
@pytest.mark.parametrize("T", [1, 2, 3, 63, 64, 65, 1000, 65536])
def test_every_token_count(T):
    """All rows of a batch against the same rows one at a time (those are pinned above)."""
    rng = np.random.default_rng(T)
    E, k = 384, 6
    base = torch.from_numpy(rng.standard_normal((min(T, 500), E)).astype(f4)).to(DEV)
    z = base[torch.arange(T, device=DEV) % base.shape[0]].contiguous()
    bias = torch.from_numpy((0.05 * rng.standard_normal(E)).astype(f4)).to(DEV)
    g = lib.gate(E, k, score="sigmoid", n_groups=8, top_groups=4, group_score="top2", bias=bias)
    idx, wt = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    lib.gate_topk(g, z, idx, wt)
    one_i, one_w = torch.empty(1, k, dtype=torch.int32, device=DEV), torch.empty(1, k, device=DEV)
    for t in range(0, base.shape[0], max(1, base.shape[0] // 40)):
        lib.gate_topk(g, base[t: t + 1], one_i, one_w)
        same = torch.arange(t, T, base.shape[0], device=DEV)
        assert (idx[same] == one_i).all() and (wt[same] == one_w).all()


@gpu
def test_agrees_with_the_sigmoid_router():
    """One group, sigmoid, renormalised: the routes of route_topk (its weights are computed in double)."""
    rng = np.random.default_rng(8)
    E, d, T, k = 384, 512, 50, 6
    w = torch.from_numpy((0.05 * rng.standard_normal((E, d))).astype(f4)).to(DEV)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(f4)).to(DEV)
    bias = torch.from_numpy((0.05 * rng.standard_normal(E)).astype(f4)).to(DEV)
    for b in (None, bias):
        i1, w1 = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
        lib.route_topk(w, x, k, i1, w1, torch.empty(T * E * 4, dtype=torch.uint8, device=DEV), bias=b)
        z = torch.empty(T, E, device=DEV)
        lib.router_logits(w, x, z)
        i2, w2 = torch.empty_like(i1), torch.empty_like(w1)
        lib.gate_topk(lib.gate(E, k, bias=b), z, i2, w2)
        assert torch.equal(i1, i2)
        assert torch.allclose(w1, w2, rtol=WT_REL, atol=0)


@gpu
def test_sigmoid_scores_have_the_defined_bits():
    """Two million logits, one expert: the plain weight is the score, bit for bit."""
    rng = np.random.default_rng(10)
    g = lib.gate(1, 1, renormalize=False)
    for i in range(32):
        z = (rng.uniform(-85, 85, 65536) if i % 2 else 3 * rng.standard_normal(65536)).astype(f4)
        if i == 0:
            z[:8] = [0.0, -0.0, 80.0, -80.0, 81.0, -81.0, np.finfo(f4).max, -1e38]
        zd = torch.from_numpy(z).to(DEV).view(-1, 1)
        idx, wt = torch.empty(65536, 1, dtype=torch.int32, device=DEV), torch.empty(65536, 1, device=DEV)
        lib.gate_topk(g, zd, idx, wt)
        u = -np.clip(z, f4(-80), f4(80))
        n = (u * f4(float.fromhex("0x1.715476p0")) + f4(1.5 * 2 ** 23)) - f4(1.5 * 2 ** 23)
        r = (u - n * f4(float.fromhex("0x1.62e400p-1"))) - n * f4(float.fromhex("0x1.7f7d1cp-20"))
        p = np.full_like(r, f4(float.fromhex("0x1.6c16c2p-10")))
        for c in ("0x1.111112p-7", "0x1.555556p-5", "0x1.555556p-3", "0x1p-1", "0x1p0", "0x1p0"):
            p = p * r + f4(float.fromhex(c))
        want = f4(1) / (f4(1) + np.ldexp(p, n.astype(np.int32)))
        assert (idx == 0).all()
        assert np.array_equal(wt.cpu().numpy().ravel().view(np.uint32), want.view(np.uint32))


@gpu
def test_equal_values_in_one_lane_and_across():
    """Few distinct logits: every round has equals in a lane's slots, in other lanes and in other groups."""
    rng = np.random.default_rng(12)
    for E, G, KG in ((384, 8, 3), (384, 1, 1), (96, 3, 2), (1000, 40, 7), (256, 4, 2)):
        z = rng.integers(0, 4, (24, E)).astype(f4)
        z[:6] += (rng.random((6, E)) < 0.02).astype(f4) * rng.random((6, E)).astype(f4)  # a few that are unique
        for dtype in (torch.float32, torch.bfloat16):
            for bias in (None, (rng.integers(0, 3, E) / 4).astype(f4)):
                check(torch.from_numpy(z).to(dtype), 12, "sigmoid", G, KG, "top2", True, 1.0, bias)


@gpu
@pytest.mark.parametrize("E,k,G,KG", [(384, 6, 8, 4), (384, 6, 1, 1), (256, 8, 8, 4), (100, 4, 10, 6), (1024, 16, 1, 1),
                                      (1024, 8, 4, 2), (48, 3, 3, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_values_a_few_units_apart(E, k, G, KG, score):
    """Values that differ by a few of their last bits, in a token's best, its groups or both; biases of every size."""
    rng = np.random.default_rng(E + k + G)
    base = rng.integers(-2, 3, (20, E)).astype(f4)
    z = (base * (1 + rng.integers(-3, 4, (20, E)) * f4(2.0 ** -23))).astype(f4)
    z[10:] += (rng.random((10, E)) * 1e-5).astype(f4)
    tiny = (rng.integers(-4, 5, E) * 2.0 ** -24).astype(f4)
    for bias in (None, tiny, tiny + f4(1000.0), (rng.choice([-1e6, 1e6], E) + rng.random(E)).astype(f4),
                 rng.choice([3e38, -3e38, 2e30, 1.0, math.inf, -math.inf], E).astype(f4),
                 (rng.standard_normal(E) * 1e-3).astype(f4)):
        for gs in ("max", "top2"):
            check(torch.from_numpy(z), k, score, G, KG, gs, True, 1.0, bias)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_best_experts_crowd_in_one_place(dtype):
    """The best values at distances of 8, 16, 32 and 64 experts, the ones that share registers."""
    rng = np.random.default_rng(14)
    for E, k, G, KG in ((384, 6, 1, 1), (1024, 16, 1, 1), (384, 6, 8, 4), (1000, 8, 2, 1), (960, 5, 8, 5)):
        z = (0.01 * rng.standard_normal((24, E))).astype(f4)
        for t in range(24):
            step = (8, 16, 32, 64)[t % 4]
            at = np.arange(rng.integers(0, step), E, step)
            at = at[: rng.integers(3, 9)]
            z[t, at] += 2 + 0.25 * rng.permutation(len(at)).astype(f4)
        for bias in (None, (0.01 * rng.standard_normal(E)).astype(f4)):
            check(torch.from_numpy(z).to(dtype), k, "sigmoid", G, KG, "max", True, 1.0, bias)


@gpu
def test_streams_and_graph_replays():
    rng = np.random.default_rng(9)
    z = torch.from_numpy(rng.standard_normal((300, 100)).astype(f4)).to(DEV)
    g = lib.gate(100, 4, score="softmax", n_groups=10, top_groups=3, group_score="top2")
    idx, wt = torch.empty(300, 4, dtype=torch.int32, device=DEV), torch.empty(300, 4, device=DEV)
    lib.gate_topk(g, z, idx, wt)
    torch.cuda.synchronize()
    want_i, want_w = idx.clone(), wt.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.gate_topk(g, z, idx, wt)
    for _ in range(3):
        for call in (lambda: lib.gate_topk(g, z, idx, wt, stream=side), graph.replay):
            idx.zero_(), wt.zero_()
            torch.cuda.synchronize()
            call()
            torch.cuda.synchronize()
            assert torch.equal(idx, want_i) and torch.equal(wt, want_w)


# ---------------------------------------------------------------- refusals ----
P = 1 << 40  # never dereferenced: every call below is refused


def refused(gate_kw=None, **kw):
    g = lib.MoeGate(abi_version=lib.MOE_ABI_VERSION, n_experts=64, top_k=4, score=0, n_groups=8, top_groups=2,
                    group_score=0, renormalize=1, scale=1.0, bias=None)
    for name, v in (gate_kw or {}).items():
        setattr(g, name, v)
    a = dict(z=P, z_dtype=0, z_stride=64, T=4, idx=P, wt=P, stream=None)
    a.update(kw)
    import ctypes
    return lib.lib().moe_gate_topk(ctypes.byref(g), *a.values())


@pytest.mark.parametrize("gate_kw", [
    dict(n_experts=0), dict(n_experts=1025), dict(n_groups=0), dict(n_groups=7), dict(n_experts=130, n_groups=65),
    dict(top_groups=0), dict(top_groups=9), dict(top_k=0), dict(top_k=17), dict(top_groups=1, top_k=9),
    dict(renormalize=2), dict(scale=math.inf), dict(scale=math.nan), dict(bias=P + 2),
])
def test_gate_refusals(gate_kw):
    assert refused(gate_kw) == lib.MOE_ERR_INVALID_ARG
    assert "moe_gate_topk" in lib.last_error()


def test_gate_unsupported():
    for gate_kw in (dict(abi_version=2), dict(score=2), dict(group_score=-1)):
        assert refused(gate_kw) == lib.MOE_ERR_UNSUPPORTED
    assert refused(z_dtype=5) == lib.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(z=None), dict(z=P + 2), dict(z=P + 1, z_dtype=1), dict(z_stride=63), dict(T=-1),
                                dict(T=65537), dict(idx=None), dict(wt=P + 4)])
def test_gate_argument_refusals(kw):
    assert refused(**kw) == lib.MOE_ERR_INVALID_ARG


def test_no_tokens_is_a_no_op():
    assert refused(T=0, z=None, idx=None, wt=None) == lib.MOE_OK


def test_router_logits_refusals():
    L = lib.lib()
    assert L.moe_router_logits(P, 384, 4096, P, 0, 0, P, None) == lib.MOE_OK
    for args in ((None, 384, 4096, P, 0, 1, P), (P, 0, 4096, P, 0, 1, P), (P, 384, 4000, P, 0, 1, P),
                 (P, 384, 4096, None, 0, 1, P), (P, 384, 4096, P, 0, -1, P), (P, 384, 4096, P, 0, 1, P + 4)):
        assert L.moe_router_logits(*args, None) == lib.MOE_ERR_INVALID_ARG
    assert L.moe_router_logits(P, 384, 4096, P, 9, 1, P, None) == lib.MOE_ERR_UNSUPPORTED


def test_binding_checks_the_gate_call():
    g = lib.gate(64, 4)
    i, w = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4)
    with pytest.raises(ValueError, match="logits per row"):
        lib.gate_topk(g, torch.zeros(3, 63), i, w)
    with pytest.raises(TypeError, match="z must be"):
        lib.gate_topk(g, torch.zeros(3, 64, dtype=torch.float16), i, w)
    with pytest.raises(ValueError, match="idx has shape"):
        lib.gate_topk(g, torch.zeros(3, 64), i[:2], w)
    with pytest.raises(TypeError, match="wt must be"):
        lib.gate_topk(g, torch.zeros(3, 64), i, w.double())
    with pytest.raises(ValueError, match="bias has shape"):
        lib.gate(64, 4, bias=torch.zeros(63))
