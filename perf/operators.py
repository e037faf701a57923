"""What is measured of the gate and of the block-scaled 8-bit operators.

Five operators, called through quantized_moe_amd.lib:

  gate      lib.gate_topk            scores, groups and top-k of given router logits
  quantize  lib.blockscale_quantize  activations to E4M3 with a scale per 128 values of a row
  matmul    lib.blockscale_matmul    E4M3 x E4M3 with a scale per 128 (rows) and per 128 x 128 (weights)
  gateup    lib.blockscale_gateup    the routed experts' gate/up product, SwiGLU, requantised
  down      lib.blockscale_down      the routed experts' down product and the weighted sum per token

Sizes are those of this repository's layer (384 experts, 6 per token,
d = 4096, f = 2048) and of its limits (d, f up to 8192, 65536 tokens).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token's routes while it is decoded: nothing but latency
        dict(name="gate_token", op="gate", T=1, E=384, k=6, score="sigmoid", groups=8, top_groups=4, group_score="top2",
             bias=True, renorm=True, scale=2.5, dtype="f32", mask=0.0),
        # a prompt through a softmax gate, logits as a bf16 router product leaves them
        dict(name="gate_prompt", op="gate", T=4096, E=384, k=6, score="softmax", groups=1, top_groups=1, group_score="max",
             bias=False, renorm=False, scale=1.0, dtype="bf16", mask=0.0),
        # the longest batch that one call takes, with groups, a bias and experts masked out
        dict(name="gate_long", op="gate", T=65536, E=384, k=6, score="sigmoid", groups=8, top_groups=4, group_score="top2",
             bias=True, renorm=True, scale=2.5, dtype="f32", mask=0.02),
        # the activations of a 1024-token prompt before the experts
        dict(name="quantize_prompt", op="quantize", M=1024, K=4096, dtype="bf16"),
        # a long batch of fp32 activations at the widest layer
        dict(name="quantize_long", op="quantize", M=16384, K=8192, dtype="f32"),
        # one token through a projection: the weights are read once
        dict(name="matmul_token", op="matmul", M=1, N=4096, K=4096, out="bf16"),
        # a ragged batch, nothing a multiple of a tile, blocks of 128 that end early
        dict(name="matmul_ragged", op="matmul", M=1000, N=1100, K=2064, out="f32"),
        # the largest: a long prompt at the widest layer
        dict(name="matmul_long", op="matmul", M=8192, N=8192, K=8192, out="bf16"),
        # 8 tokens decoded together: some 45 experts of one or two rows each
        dict(name="gateup_8_tokens", op="gateup", T=8, E=384, k=6, d=4096, f=2048, skew=0.0),
        # a 1024-token prompt: every expert is read, 16 rows each
        dict(name="gateup_prompt", op="gateup", T=1024, E=384, k=6, d=4096, f=2048, skew=0.0),
        # one token's down products and their sum
        dict(name="down_token", op="down", T=1, E=384, k=6, d=4096, f=2048, skew=0.0, add=True),
        # a long prompt whose routes crowd on few experts
        dict(name="down_long", op="down", T=4096, E=384, k=6, d=4096, f=2048, skew=1.1, add=False),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "quantize", "matmul", "gateup", "down"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 5, 8])
        E = groups * max(2, _log(rng, 16, 512) // groups)
        k = rng.randint(1, min(8, E // groups))
        return dict(op=op, T=_log(rng, 1, 65536 if E <= 384 else 32768), E=E, k=k, score=rng.choice(["sigmoid", "softmax"]),
                    groups=groups, top_groups=rng.randint(1, groups), group_score=rng.choice(["max", "top2"]),
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "bf16"]), mask=rng.choice([0.0, 0.0, 0.02]))
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 16384), K=16 * _log(rng, 16, 512), dtype=rng.choice(["f32", "bf16"]))
    if op == "matmul":
        N, K = _log(rng, 256, 8192), 16 * _log(rng, 16, 512)
        return dict(op=op, M=_log(rng, 1, 8192), N=N, K=K, out=rng.choice(["f32", "bf16"]))
    E, k = _log(rng, 16, 384), rng.randint(2, 6)
    case = dict(op=op, T=_log(rng, 1, 1024 if op == "gateup" else 4096), E=E, k=k, d=16 * _log(rng, 32, 256),
                f=16 * _log(rng, 16, 128), skew=rng.choice([0.0, 1.1]))
    if op == "down":
        case["add"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs ----
def _codes(g, *shape):
    """E4M3 codes of normal values whose block maximum is near the type's, as a quantiser leaves them."""
    q = torch.empty(shape, dtype=F8, device=DEV)
    for part in q.view(-1, shape[-1]).split(max(1, (1 << 27) // shape[-1])):
        part.copy_((torch.randn(part.shape, dtype=torch.float32, device=DEV, generator=g) * 110.0).clamp_(-448.0, 448.0))
    return q


def _scales(g, rms, *shape):
    """Scales that give values of `rms` on average, each block its own."""
    return (rms / 110.0) * torch.exp(0.3 * torch.randn(shape, device=DEV, generator=g))


def _blocks(n):
    return -(-n // 128)


def _routes(g, T, E, k, skew):
    """Distinct experts per token; with a skew their popularity falls as a power of their rank."""
    z = torch.rand(T, E, device=DEV, generator=g).clamp_(min=1e-30).log_().neg_().log_().neg_()
    if skew:
        order = torch.randperm(E, device=DEV, generator=g)
        z = z - skew * torch.log(1.0 + order.float())
    idx = z.topk(k, dim=1).indices.to(torch.int32)
    wt = torch.rand(T, k, device=DEV, generator=g) + 0.1
    return idx, wt / wt.sum(1, keepdim=True)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "gate":
        T, E = case["T"], case["E"]
        z = torch.randn(T, E, device=DEV, generator=g) * 1.5
        if case["mask"]:  # experts taken out: by -inf, and by the type's lowest value
            out = torch.rand(T, E, device=DEV, generator=g)
            z[out < case["mask"]] = -math.inf
            z[out > 1.0 - case["mask"] / 2] = torch.finfo(DTYPES[case["dtype"]]).min
            z[torch.rand(T, device=DEV, generator=g) < case["mask"] / 8] = -math.inf  # rows with none left
        s["z"] = z.to(DTYPES[case["dtype"]])
        s["bias"] = 0.05 * torch.randn(E, device=DEV, generator=g) if case["bias"] else None
        s["idx"] = torch.empty(T, case["k"], dtype=torch.int32, device=DEV)
        s["wt"] = torch.empty(T, case["k"], dtype=torch.float32, device=DEV)
    elif op == "quantize":
        M, K = case["M"], case["K"]
        x = torch.randn(M, K, device=DEV, generator=g)
        x *= torch.exp(torch.randn(M, 1, device=DEV, generator=g))  # rows differ in size
        x[:, torch.randint(0, K, (max(1, K // 256),), device=DEV, generator=g)] *= 20.0  # channels that stand out
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["q"] = torch.empty(M, K, dtype=F8, device=DEV)
        s["s"] = torch.empty(M, _blocks(K), dtype=torch.float32, device=DEV)
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["xq"], s["xs"] = _codes(g, M, K), _scales(g, 1.0, M, _blocks(K))
        s["wq"], s["ws"] = _codes(g, N, K), _scales(g, 0.02, _blocks(N), _blocks(K))
        s["y"] = torch.empty(M, N, dtype=DTYPES[case["out"]], device=DEV)
    else:
        T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
        s["idx"], s["wt"] = _routes(g, T, E, k, case["skew"])
        # the routes by expert, as lib.bucket gives them
        flat = s["idx"].view(-1).long()
        order = torch.argsort(flat, stable=True)
        s["perm"] = order.to(torch.int32)
        s["pos"] = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=DEV)).to(torch.int32)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        s["offsets"][1:] = torch.bincount(flat, minlength=E).cumsum(0)
        if op == "gateup":
            s["xq"], s["xs"] = _codes(g, T, d), _scales(g, 1.0, T, _blocks(d))
            for n in ("g", "u"):
                s["wq_" + n], s["ws_" + n] = _codes(g, E, f, d), _scales(g, 0.02, E, _blocks(f), _blocks(d))
            s["hq"] = torch.empty(T * k, f, dtype=F8, device=DEV)
            s["hs"] = torch.empty(T * k, _blocks(f), dtype=torch.float32, device=DEV)
        else:
            s["hq"], s["hs"] = _codes(g, T * k, f), _scales(g, 1.0, T * k, _blocks(f))
            s["wq"], s["ws"] = _codes(g, E, d, f), _scales(g, 0.02, E, _blocks(d), _blocks(f))
            s["add"] = torch.randn(T, d, device=DEV, generator=g) if case["add"] else None
            s["y"] = torch.empty(T, d, dtype=torch.float32, device=DEV)
    return s


# --------------------------------------------------------------- the calls ----
def run(s):
    op = s["case"]["op"]
    return (_own if own else _plain)[op](s)


def _workspace(s, bytes_needed):
    """A workspace that the program keeps beside its other buffers."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(256, bytes_needed()), dtype=torch.uint8, device=DEV)
    return s["workspace"]


def _own_gate(s):
    from quantized_moe_amd import lib
    c = s["case"]
    if "gate" not in s:  # the gate's description, made once
        s["gate"] = lib.gate(c["E"], c["k"], score=c["score"], n_groups=c["groups"], top_groups=c["top_groups"],
                             group_score=c["group_score"], renormalize=c["renorm"], scale=c["scale"], bias=s["bias"])
    lib.gate_topk(s["gate"], s["z"], s["idx"], s["wt"])
    return {"idx": s["idx"], "wt": s["wt"]}


def _own_quantize(s):
    from quantized_moe_amd import lib
    lib.blockscale_quantize(s["x"], s["q"], s["s"])
    return {"q": s["q"], "s": s["s"]}


def _own_matmul(s):
    from quantized_moe_amd import lib
    c = s["case"]
    ws = _workspace(s, lambda: lib.blockscale_matmul_workspace_bytes(c["M"], c["N"], c["K"]))
    lib.blockscale_matmul(s["xq"], s["xs"], s["wq"], s["ws"], s["y"], ws)
    return s["y"]


def _own_gateup(s):
    from quantized_moe_amd import lib
    lib.blockscale_gateup(s["xq"], s["xs"], s["case"]["k"], s["offsets"], s["perm"], s["wq_g"], s["ws_g"], s["wq_u"], s["ws_u"],
                          s["hq"], s["hs"])
    return {"hq": s["hq"], "hs": s["hs"]}


def _own_down(s):
    from quantized_moe_amd import lib
    c = s["case"]
    ws = _workspace(s, lambda: lib.blockscale_down_workspace_bytes(c["T"], c["k"], c["d"]))
    lib.blockscale_down(s["hq"], s["hs"], s["wt"], s["offsets"], s["pos"], s["wq"], s["ws"], s["y"], ws, add=s["add"])
    return s["y"]


_own = {"gate": _own_gate, "quantize": _own_quantize, "matmul": _own_matmul, "gateup": _own_gateup, "down": _own_down}


# ---------------------------------------------------------- the plain forms ----
# exp of t in [-80, 80] by the fixed fp32 steps that the gate's scores are
# defined by: every product and sum is rounded on its own, so that selections
# near a tie are the same wherever the steps are followed.
_EXP = [float.fromhex(h) for h in ("0x1.6c16c2p-10", "0x1.111112p-7", "0x1.555556p-5", "0x1.555556p-3", "0x1p-1", "0x1p0", "0x1p0")]
_LOG2E, _LN2_HI, _LN2_LO, _MAGIC = (float.fromhex(h) for h in ("0x1.715476p0", "0x1.62e400p-1", "0x1.7f7d1cp-20", "0x1.8p23"))


def _exp32(t):
    n = (t * _LOG2E + _MAGIC) - _MAGIC
    r = (t - n * _LN2_HI) - n * _LN2_LO
    p = torch.full_like(r, _EXP[0]) * r + _EXP[1]
    p = p * r + _EXP[2]
    p = p * r + _EXP[3]
    p = p * r + _EXP[4]
    p = p * r + _EXP[5]
    p = p * r + _EXP[6]
    return p * ((n.to(torch.int32) + 127) << 23).view(torch.float32)


def _fold_sum(e):
    """Row sums in the gate's order: 64 partial sums, element i in partial i mod 64, then halves added."""
    T, E = e.shape
    e = torch.nn.functional.pad(e, (0, -E % 64)).view(T, -1, 64)
    p = torch.zeros_like(e[:, 0])
    for i in range(e.shape[1]):
        p = p + e[:, i]
    while p.shape[1] > 1:
        p = p[:, : p.shape[1] // 2] + p[:, p.shape[1] // 2:]
    return p


def _plain_gate(s):
    c, z = s["case"], s["z"].float()
    T, E, k, G = z.shape[0], c["E"], c["k"], c["groups"]
    masked = torch.isnan(z) | (z <= -(2.0 ** 127))
    low = torch.full_like(z, -math.inf)
    z = z.clamp(max=torch.finfo(torch.float32).max)
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + _exp32(-z.clamp(-80.0, 80.0)))
    else:
        live = torch.where(masked, low, z)
        e = _exp32((live - live.amax(1, keepdim=True)).clamp(-80.0, 0.0).nan_to_num(-80.0))
        e = torch.where(masked, torch.zeros_like(e), e)
        score = e / _fold_sum(e)
    if s["bias"] is not None:
        v = score + s["bias"]
    elif c["top_groups"] < G and c["group_score"] == "top2":
        v = score
    else:
        v = z
    v = torch.where(masked | ~(v > -math.inf), low, v)
    if c["top_groups"] < G:
        best = v.view(T, G, E // G).sort(dim=2, descending=True).values
        value = best[:, :, 0]
        if c["group_score"] == "top2" and E // G > 1:
            value = torch.where(best[:, :, 1] > -math.inf, value + best[:, :, 1], value)
        order = value.sort(dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, order, True)
        v = torch.where(keep.repeat_interleave(E // G, dim=1), v, low)
    top = v.sort(dim=1, descending=True, stable=True)
    v, idx = top.values[:, :k], top.indices[:, :k]
    found = v > -math.inf
    a = torch.where(found, score.gather(1, idx), torch.zeros_like(v))
    if c["renorm"]:
        total = torch.zeros_like(a[:, 0])
        for j in range(k):
            total = total + a[:, j]
        a = torch.where(found, a / total[:, None], torch.zeros_like(a))
    return {"idx": torch.where(found, idx, torch.full_like(idx, -1)).to(torch.int32), "wt": a * c["scale"]}


def _quantize(x):
    """(codes, scales) of fp32 rows: per 128 values the largest becomes 448."""
    M, K = x.shape
    b = torch.nn.functional.pad(x, (0, -K % 128)).view(M, -1, 128)
    amax = b.abs().amax(2).clamp(min=2.0 ** -100)
    s = amax / torch.full_like(amax, 448.0)  # (a quotient: torch takes a number's reciprocal)
    q = (b / s[:, :, None]).clamp(-448.0, 448.0).view(M, -1)[:, :K].to(F8)
    return q, s


def _plain_quantize(s):
    q, scale = _quantize(s["x"].float())
    return {"q": q, "s": scale}


def _rows(q, s):
    """The values of rows quantised per 128 of a row, in fp32."""
    return q.float() * s.repeat_interleave(128, dim=1)[:, : q.shape[1]]


def _weight(q, s):
    """The values of a matrix quantised per 128 x 128 block, in fp32."""
    N, K = q.shape
    return q.float() * s.repeat_interleave(128, dim=1)[:, :K].repeat_interleave(128, dim=0)[:N]


def _plain_matmul(s):
    return (_rows(s["xq"], s["xs"]) @ _weight(s["wq"], s["ws"]).t()).to(s["y"].dtype)


def _by_expert(offsets):
    """(expert, first row, last row + 1) of the experts that have rows: a product each is what a plain program runs."""
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def _plain_gateup(s):
    x = _rows(s["xq"], s["xs"])[(s["perm"] // s["case"]["k"]).long()]
    h = torch.empty(x.shape[0], s["case"]["f"], device=x.device)
    for e, a, b in _by_expert(s["offsets"]):
        gate = x[a:b] @ _weight(s["wq_g"][e], s["ws_g"][e]).t()
        up = x[a:b] @ _weight(s["wq_u"][e], s["ws_u"][e]).t()
        h[a:b] = gate / (1.0 + torch.exp(-gate)) * up
    hq, hs = _quantize(h)
    return {"hq": hq, "hs": hs}


def _plain_down(s):
    c, h = s["case"], _rows(s["hq"], s["hs"])
    ye = torch.empty(h.shape[0], c["d"], device=h.device)
    for e, a, b in _by_expert(s["offsets"]):
        ye[a:b] = h[a:b] @ _weight(s["wq"][e], s["ws"][e]).t()
    y = (ye[s["pos"].long()].view(c["T"], c["k"], -1) * s["wt"][:, :, None]).sum(1)
    return y if s["add"] is None else s["add"] + y


_plain = {"gate": _plain_gate, "quantize": _plain_quantize, "matmul": _plain_matmul, "gateup": _plain_gateup, "down": _plain_down}


# ------------------------------------------------------- 64-bit definitions ----
def _exact_gate(s):
    """Numpy: the rank values by the fp32 steps of their definition, the weights in 64 bits."""
    f4 = np.float32
    c, k, G = s["case"], s["case"]["k"], s["case"]["groups"]
    z = s["z"].float().cpu().numpy()
    bias = None if s["bias"] is None else s["bias"].cpu().numpy()
    T, E = z.shape
    out = np.isnan(z) | (z <= f4(-(2.0 ** 127)))
    z = np.minimum(np.where(out, f4(0), z), np.finfo(f4).max)

    def exp_steps(t):
        n = (t * f4(_LOG2E) + f4(_MAGIC)) - f4(_MAGIC)
        r = (t - n * f4(_LN2_HI)) - n * f4(_LN2_LO)
        p = np.full(t.shape, f4(_EXP[0]), f4)
        for a in _EXP[1:]:
            p = p * r + f4(a)
        return np.ldexp(p, n.astype(np.int32))

    if c["score"] == "sigmoid":
        rank = f4(1) / (f4(1) + exp_steps(-np.clip(z, f4(-80), f4(80))))
        s64 = 1.0 / (1.0 + np.exp(-np.clip(z, -80.0, 80.0).astype(np.float64)))
    else:
        m = np.where(out, f4(-np.inf), z).max(1, keepdims=True)
        t = np.clip(z - np.where(np.isfinite(m), m, f4(0)), f4(-80), f4(0))
        e = np.where(out, f4(0), exp_steps(t))
        p = np.zeros((T, 64), f4)
        for i in range(0, E, 64):
            w = min(64, E - i)
            p[:, :w] += e[:, i: i + w]
        for h in (32, 16, 8, 4, 2, 1):
            p = p[:, :h] + p[:, h: 2 * h]
        with np.errstate(invalid="ignore"):
            rank = e / p
            s64 = np.where(out, 0.0, np.exp(t.astype(np.float64)))
            s64 = s64 / s64.sum(1, keepdims=True)
    if bias is not None:
        rank = rank + bias
    elif not (c["top_groups"] < G and c["group_score"] == "top2"):
        rank = z
    rank = np.where(out, f4(-np.inf), rank)
    if c["top_groups"] < G:
        groups = -np.sort(-rank.reshape(T, G, -1), axis=2)
        value = groups[:, :, 0].copy()
        if c["group_score"] == "top2" and groups.shape[2] > 1:
            two = groups[:, :, 1] > -np.inf
            value[two] += groups[:, :, 1][two]
        chosen = np.argsort(-value, axis=1, kind="stable")[:, : c["top_groups"]]
        keep = np.zeros((T, G), bool)
        np.put_along_axis(keep, chosen, True, axis=1)
        rank = np.where(np.repeat(keep, E // G, axis=1), rank, f4(-np.inf))
    idx = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    found = np.take_along_axis(rank, idx, axis=1) > -np.inf
    a = np.where(found, np.take_along_axis(s64, idx, axis=1), 0.0)
    if c["renorm"]:
        total = a.sum(1, keepdims=True)
        a = np.divide(a, total, out=np.zeros_like(a), where=total > 0)
    return {"idx": np.where(found, idx, -1).astype(np.int32), "wt": a * c["scale"]}


def _exact_codes(h):
    """Scales and rounded codes (as 64-bit numbers) of 64-bit rows, a group of 128 columns at a time."""
    codes, scales = torch.empty_like(h), []
    for a in range(0, h.shape[1], 128):
        part = h[:, a: a + 128]
        scale = torch.maximum(part.abs().max(dim=1).values, torch.tensor(2.0 ** -100, dtype=torch.float64, device=h.device)) / 448
        v = part / scale[:, None]
        # steps of 1/8 of the power of two below, no finer than 2^-9; halves to even
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, a: a + 128] = torch.round(v / step) * step
        scales.append(scale)
    return codes, torch.stack(scales, 1)


def _exact_product(xq, xs, wq, ws):
    """sum over blocks b of xs[m][b] ws[n / 128][b] (xq_b . wq_b), in 64 bits; the block dots are exact."""
    M, N, K = xq.shape[0], wq.shape[0], xq.shape[1]
    y = torch.zeros(M, N, dtype=torch.float64, device=xq.device)
    col = torch.arange(N, device=xq.device) // 128
    for b in range(_blocks(K)):
        cols = slice(128 * b, min(K, 128 * (b + 1)))
        y += (xq[:, cols].double() * xs[:, b, None].double()) @ (wq[:, cols].double() * ws[col, b, None].double()).t()
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(s)
    if op == "quantize":
        q, scale = _exact_codes(s["x"].double())
        return {"q": q, "s": scale}
    if op == "matmul":
        return _exact_product(s["xq"], s["xs"], s["wq"], s["ws"])
    T, k = case["T"], case["k"]
    expert = torch.repeat_interleave(torch.arange(case["E"], device=DEV), (s["offsets"][1:] - s["offsets"][:-1]).long())
    if op == "gateup":
        h = torch.empty(T * k, case["f"], dtype=torch.float64, device=DEV)
        token = (s["perm"] // k).long()
        for e in expert.unique().tolist():
            r = (expert == e).nonzero()[:, 0]
            xq, xs = s["xq"].view(torch.uint8)[token[r]].view(F8), s["xs"][token[r]]
            gate = _exact_product(xq, xs, s["wq_g"][e], s["ws_g"][e])
            h[r] = gate * torch.sigmoid(gate) * _exact_product(xq, xs, s["wq_u"][e], s["ws_u"][e])
        hq, hs = _exact_codes(h)
        return {"hq": hq, "hs": hs}
    y = torch.zeros(T, case["d"], dtype=torch.float64, device=DEV) if s["add"] is None else s["add"].double()
    route = s["perm"].long()
    for e in expert.unique().tolist():
        r = (expert == e).nonzero()[:, 0]
        ye = _exact_product(s["hq"].view(torch.uint8)[r].view(F8), s["hs"][r], s["wq"][e], s["ws"][e])
        y.index_add_(0, route[r] // k, ye * s["wt"].view(-1)[route[r], None].double())
    return y


def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (2 if case["dtype"] == "bf16" else 4) + 8 * T * k + (4 * E if case["bias"] else 0),
                "flops": 20 * T * E}
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * ((2 if case["dtype"] == "bf16" else 4) + 1) + 4 * M * _blocks(K), "flops": 3 * M * K}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K + 4 * (M + _blocks(N)) * _blocks(K) + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
    used = _distinct(T, E, k, case["skew"])
    if op == "gateup":
        return {"bytes": T * (d + 4 * _blocks(d)) + used * 2 * (f * d + 4 * _blocks(f) * _blocks(d)) + T * k * (f + 4 * _blocks(f)),
                "flops": 4 * T * k * f * d}
    return {"bytes": T * k * (f + 4 * _blocks(f)) + used * (f * d + 4 * _blocks(f) * _blocks(d)) + 4 * T * d * (2 if case["add"] else 1),
            "flops": 2 * T * k * f * d}


def _distinct(T, E, k, skew):
    """How many experts T tokens reach on average, each taking k by their popularity."""
    p = np.arange(1.0, E + 1.0) ** -skew
    p = np.minimum(1.0, k * p / p.sum())
    return float(np.sum(1.0 - (1.0 - p) ** T))
