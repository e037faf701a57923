"""What is measured of the 8-bit integer products and of the router's balance loss.

Five operators, called through quantized_moe_amd.lib:

  quantize  lib.int8_quantize   activations to int8 with one scale per row (token)
  matmul    lib.int8_matmul     int8 x int8 with a scale per row and per output channel
  gateup    lib.int8_gateup     the routed experts' gate/up product with SwiGLU
  down      lib.int8_down       the routed experts' down product and the weighted sum per token
  balance   lib.balance_loss    tokens per expert and the balance loss of each sequence; with "grad" also
            lib.balance_loss_backward, its gradient with respect to the router logits

Sizes are those of this repository's layer (384 experts, 6 per token,
d = 4096, f = 2048) and of its limits (65536 tokens, widths up to 8192).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a few tokens' activations while they are decoded: nothing but latency
        dict(name="quantize_8_tokens", op="quantize", M=8, K=4096, dtype="bf16"),
        # a long batch of fp32 activations at the widest layer
        dict(name="quantize_long", op="quantize", M=16384, K=8192, dtype="f32"),
        # one token through a projection: the weights are read once
        dict(name="matmul_token", op="matmul", M=1, N=4096, K=4096, out="bf16"),
        # a ragged batch, nothing a multiple of a tile
        dict(name="matmul_ragged", op="matmul", M=700, N=1300, K=2320, out="f32"),
        # the largest: a long prompt at the widest layer
        dict(name="matmul_long", op="matmul", M=8192, N=8192, K=8192, out="bf16"),
        # 8 tokens decoded together: some 45 experts of one or two rows each
        dict(name="gateup_8_tokens", op="gateup", T=8, E=384, k=6, d=4096, f=2048, skew=0.0, out="f32"),
        # a 1024-token prompt: every expert is read, 16 rows each
        dict(name="gateup_prompt", op="gateup", T=1024, E=384, k=6, d=4096, f=2048, skew=0.0, out="bf16"),
        # one token's down products and their sum
        dict(name="down_token", op="down", T=1, E=384, k=6, d=4096, f=2048, skew=0.0, add=True),
        # a long prompt whose routes crowd on few experts
        dict(name="down_long", op="down", T=4096, E=384, k=6, d=4096, f=2048, skew=1.1, add=False),
        # how a small batch of one conversation loads the experts: counts and loss while serving
        dict(name="balance_batch", op="balance", T=64, E=384, k=6, S=1, score="sigmoid", dtype="f32", mask=0.0, grad=False),
        # a training step's micro-batch of ragged sequences behind one another, bf16 logits, padding at the end
        dict(name="balance_ragged_step", op="balance", T=4096, E=384, k=6, S=9, score="softmax", dtype="bf16", mask=0.02, grad=True),
        # the longest batch that one call takes, as one sequence
        dict(name="balance_long_step", op="balance", T=65536, E=384, k=6, S=1, score="sigmoid", dtype="f32", mask=0.0, grad=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "gateup", "down", "balance"])
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 16384), K=16 * _log(rng, 16, 512), dtype=rng.choice(["f32", "bf16"]))
    if op == "matmul":
        N, K = _log(rng, 256, 8192), 16 * _log(rng, 16, 512)
        return dict(op=op, M=_log(rng, 1, 8192), N=N, K=K, out=rng.choice(["f32", "bf16"]))
    if op == "balance":
        T, E = _log(rng, 1, 65536), _log(rng, 8, 384)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=_log(rng, 1, min(T, 64)), score=rng.choice(["sigmoid", "softmax"]),
                    dtype=rng.choice(["f32", "bf16"]), mask=rng.choice([0.0, 0.02]), grad=rng.random() < 0.7)
    E, k = _log(rng, 16, 384), rng.randint(2, 6)
    case = dict(op=op, T=_log(rng, 1, 1024 if op == "gateup" else 4096), E=E, k=k, d=16 * _log(rng, 32, 256),
                f=16 * _log(rng, 16, 128), skew=rng.choice([0.0, 1.1]))
    if op == "gateup":
        case["out"] = rng.choice(["f32", "bf16"])
    else:
        case["add"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs ----
def _codes(g, *shape):
    """int8 codes of normal values whose row maximum is near 127, as a quantiser leaves them."""
    q = torch.empty(shape, dtype=torch.int8, device=DEV)
    for part in q.view(-1, shape[-1]).split(max(1, (1 << 27) // shape[-1])):
        part.copy_((torch.randn(part.shape, dtype=torch.float32, device=DEV, generator=g) * 35.0).round_().clamp_(-127.0, 127.0))
    return q


def _scales(g, rms, *shape):
    """Scales that give values of `rms` on average, each row its own."""
    return (rms / 35.0) * torch.exp(0.3 * torch.randn(shape, device=DEV, generator=g))


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
    if op == "quantize":
        M, K = case["M"], case["K"]
        x = torch.randn(M, K, device=DEV, generator=g)
        x *= torch.exp(torch.randn(M, 1, device=DEV, generator=g))  # rows differ in size
        x[:, torch.randint(0, K, (max(1, K // 256),), device=DEV, generator=g)] *= 20.0  # channels that stand out
        x[torch.rand(M, device=DEV, generator=g) < 0.02] = 0.0  # padding
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["q"] = torch.empty(M, K, dtype=torch.int8, device=DEV)
        s["s"] = torch.empty(M, dtype=torch.float32, device=DEV)
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["xq"], s["xs"] = _codes(g, M, K), _scales(g, 1.0, M)
        s["wq"], s["ws"] = _codes(g, N, K), _scales(g, 0.02, N)
        s["y"] = torch.empty(M, N, dtype=DTYPES[case["out"]], device=DEV)
    elif op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        dtype = DTYPES[case["dtype"]]
        z = torch.randn(T, E, device=DEV, generator=g) * 1.5
        z += 0.5 * torch.randn(E, device=DEV, generator=g)  # experts differ in how much they are asked for
        if case["mask"]:  # experts taken out: by -inf, and by the type's lowest value
            out = torch.rand(T, E, device=DEV, generator=g)
            z[out < case["mask"]] = -math.inf
            z[out > 1.0 - case["mask"] / 2] = torch.finfo(dtype).min
            z[torch.rand(T, device=DEV, generator=g) < case["mask"]] = -math.inf  # tokens without an expert
        s["z"] = z.to(dtype)
        best = s["z"].float().clamp(min=-(2.0 ** 127)).topk(k, dim=1)  # (the gate's rule: what lies lower is out)
        s["idx"] = torch.where(best.values > -(2.0 ** 127), best.indices, torch.full_like(best.indices, -1)).to(torch.int32)
        cuts = torch.randint(0, T + 1, (S - 1,), device=DEV, generator=g)  # ragged, some of them empty
        last = T - T // 16 if S > 1 else T  # rows behind the last sequence: padding
        ends = torch.tensor([0, last], device=DEV)
        s["starts"] = None if S == 1 else torch.cat([cuts.clamp(max=last), ends]).sort().values.to(torch.int32)
        s["grad"] = 0.001 * (1.0 + torch.rand(S, device=DEV, generator=g))  # of the total loss by each sequence's
        s["counts"] = torch.empty(S, E, dtype=torch.int32, device=DEV)
        s["tokens"] = torch.empty(S, dtype=torch.int32, device=DEV)
        s["loss"] = torch.empty(S, dtype=torch.float32, device=DEV)
        s["dz"] = torch.empty(T, E, dtype=dtype, device=DEV)
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
            s["xq"], s["xs"] = _codes(g, T, d), _scales(g, 1.0, T)
            for n in ("g", "u"):
                s["wq_" + n], s["ws_" + n] = _codes(g, E, f, d), _scales(g, 0.02, E, f)
            s["h"] = torch.empty(T * k, f, dtype=DTYPES[case["out"]], device=DEV)
        else:
            s["hq"], s["hs"] = _codes(g, T * k, f), _scales(g, 1.0, T * k)
            s["wq"], s["ws"] = _codes(g, E, d, f), _scales(g, 0.02, E, d)
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


def _own_quantize(s):
    from quantized_moe_amd import lib
    lib.int8_quantize(s["x"], s["q"], s["s"])
    return {"q": s["q"], "s": s["s"]}


def _own_matmul(s):
    from quantized_moe_amd import lib
    c = s["case"]
    ws = _workspace(s, lambda: lib.int8_matmul_workspace_bytes(c["M"], c["N"], c["K"]))
    lib.int8_matmul(s["xq"], s["xs"], s["wq"], s["ws"], s["y"], ws)
    return s["y"]


def _own_gateup(s):
    from quantized_moe_amd import lib
    lib.int8_gateup(s["xq"], s["xs"], s["case"]["k"], s["offsets"], s["perm"], s["wq_g"], s["ws_g"], s["wq_u"], s["ws_u"], s["h"])
    return s["h"]


def _own_down(s):
    from quantized_moe_amd import lib
    c = s["case"]
    ws = _workspace(s, lambda: lib.int8_down_workspace_bytes(c["T"], c["k"], c["d"]))
    lib.int8_down(s["hq"], s["hs"], s["wt"], s["offsets"], s["pos"], s["wq"], s["ws"], s["y"], ws, add=s["add"])
    return s["y"]


def _own_balance(s):
    from quantized_moe_amd import lib
    c = s["case"]
    ws = _workspace(s, lambda: lib.balance_loss_workspace_bytes(c["T"], c["S"], c["E"]))
    lib.balance_loss(s["z"], s["idx"], s["counts"], s["tokens"], s["loss"], ws, score=c["score"], starts=s["starts"])
    out = {"counts": s["counts"], "tokens": s["tokens"], "loss": s["loss"]}
    if c["grad"]:
        lib.balance_loss_backward(s["z"], s["idx"], s["counts"], s["tokens"], s["grad"], s["dz"], score=c["score"], starts=s["starts"])
        out["dz"] = s["dz"]
    return out


_own = {"quantize": _own_quantize, "matmul": _own_matmul, "gateup": _own_gateup, "down": _own_down, "balance": _own_balance}


# ---------------------------------------------------------- the plain forms ----
def _plain_quantize(s):
    x = s["x"].float()
    amax = x.abs().amax(1).clamp(min=2.0 ** -100)
    scale = amax / torch.full_like(amax, 127.0)  # (a quotient: torch takes a number's reciprocal)
    return {"q": torch.round(x / scale[:, None]).to(torch.int8), "s": scale}


def _product(xq, xs, wq, ws):
    """(xq . wq) xs ws: whole numbers' sums in fp32, then the two scales."""
    return xq.float() @ wq.float().t() * xs[:, None] * ws


def _plain_matmul(s):
    return _product(s["xq"], s["xs"], s["wq"], s["ws"]).to(s["y"].dtype)


def _by_expert(offsets):
    """(expert, first row, last row + 1) of the experts that have rows: a product each is what a plain program runs."""
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def _plain_gateup(s):
    token = (s["perm"] // s["case"]["k"]).long()
    x, xs = s["xq"][token], s["xs"][token]
    h = torch.empty_like(s["h"])
    for e, a, b in _by_expert(s["offsets"]):
        gate = _product(x[a:b], xs[a:b], s["wq_g"][e], s["ws_g"][e])
        up = _product(x[a:b], xs[a:b], s["wq_u"][e], s["ws_u"][e])
        h[a:b] = gate / (1.0 + torch.exp(-gate)) * up
    return h


def _plain_down(s):
    c = s["case"]
    ye = torch.empty(c["T"] * c["k"], c["d"], device=DEV)
    for e, a, b in _by_expert(s["offsets"]):
        ye[a:b] = _product(s["hq"][a:b], s["hs"][a:b], s["wq"][e], s["ws"][e])
    y = (ye[s["pos"].long()].view(c["T"], c["k"], -1) * s["wt"][:, :, None]).sum(1)
    return y if s["add"] is None else s["add"] + y


def _plain_balance(s):
    c, z, idx = s["case"], s["z"].float(), s["idx"].long()
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    row = torch.arange(T, device=DEV)
    seq = torch.zeros_like(row) if S == 1 else torch.searchsorted(s["starts"].long(), row, right=True) - 1
    # tokens of no sequence, and those without a route, count for a sequence S that is dropped
    live = (idx >= 0).any(1) & (seq >= 0) & (seq < S)
    seq = torch.where(live, seq, torch.full_like(seq, S))
    counts = torch.zeros(S + 1, E + 1, device=DEV, dtype=torch.int32)  # column E: the routes that are none
    column = torch.where(idx >= 0, idx, torch.full_like(idx, E))
    counts.view(-1).scatter_add_(0, (seq[:, None] * (E + 1) + column).view(-1), torch.ones(T * k, device=DEV, dtype=torch.int32))
    counts = counts[:, :E]
    tokens = torch.zeros(S + 1, device=DEV, dtype=torch.int32).scatter_add_(0, seq, torch.ones_like(seq, dtype=torch.int32))
    masked = torch.isnan(z) | (z <= -(2.0 ** 127))
    z = torch.where(masked, torch.zeros_like(z), z.clamp(max=torch.finfo(torch.float32).max))
    if c["score"] == "softmax":
        m = torch.where(masked, torch.full_like(z, -math.inf), z).amax(1, keepdim=True)
        a = torch.where(masked, torch.zeros_like(z), torch.exp(z - m))
    else:
        a = torch.where(masked, torch.zeros_like(z), 1.0 / (1.0 + torch.exp(-z)))
    p = a / a.sum(1, keepdim=True).clamp(min=2.0 ** -126)
    n = tokens.clamp(min=1).float()
    f = counts.float() * (E / k) / n[:, None]  # 1 for an expert that gets its even share
    f[S] = 0.0
    P = torch.nn.functional.one_hot(seq, S + 1).float().t() @ p / n[:, None]
    out = {"counts": counts[:S].clone(), "tokens": tokens[:S].clone(), "loss": (f * P).sum(1)[:S]}
    if c["grad"]:
        grad = torch.cat([s["grad"], torch.zeros(1, device=DEV)])
        w = (f * (grad / n)[:, None])[seq]
        dz = p * (w - (p * w).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            dz = dz / (1.0 + torch.exp(z))  # 1 - sigmoid(z)
        out["dz"] = dz.to(s["z"].dtype)
    return out


_plain = {"quantize": _plain_quantize, "matmul": _plain_matmul, "gateup": _plain_gateup, "down": _plain_down, "balance": _plain_balance}


# ------------------------------------------------------- 64-bit definitions ----
def _exact_product(xq, xs, wq, ws):
    """sum_i (xs xq_i) (ws wq_i) with the scales in 64 bits; the whole numbers' sums are exact in them."""
    return (xq.double() @ wq.double().t()) * (xs.double()[:, None] * ws.double()[None, :])


def _exact_balance(s):
    """A sequence at a time, by the definition: loss = E sum_e (counts_e / (k n)) (sum_t p_te / n)."""
    c = s["case"]
    E, k, S = c["E"], c["k"], c["S"]
    starts = [0, c["T"]] if S == 1 else s["starts"].tolist()
    dz = torch.zeros(c["T"], E, dtype=torch.float64, device=DEV)
    losses = []
    for q in range(S):
        a, b = starts[q], starts[q + 1]
        rows = torch.nonzero((s["idx"][a:b] >= 0).any(1))[:, 0] + a
        n = rows.numel()
        if n == 0:
            losses.append(torch.zeros((), dtype=torch.float64, device=DEV))
            continue
        routes = s["idx"][rows].reshape(-1).long()
        share = torch.bincount(routes[routes >= 0], minlength=E).double() / (k * n)
        z = s["z"][rows].double()
        gone = torch.isnan(z) | (z <= -(2.0 ** 127))
        if c["score"] == "softmax":
            p = torch.softmax(z.masked_fill(gone, -math.inf), dim=1)
            slope = torch.ones_like(p)
        else:
            v = torch.sigmoid(z).masked_fill(gone, 0.0)
            p = v / v.sum(1, keepdim=True)
            slope = torch.sigmoid(-z).masked_fill(gone, 0.0)
        losses.append(E * (share * p.mean(0)).sum())
        w = s["grad"][q].double() * E * share / n
        dz[rows] = p * slope * (w - (p @ w)[:, None])
    out = {"counts": None, "tokens": None, "loss": torch.stack(losses)}
    if c["grad"]:
        out["dz"] = dz
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        # (codes are whole numbers that follow from the fp32 scale; only the scale has a value in 64 bits)
        return {"q": None, "s": s["x"].double().abs().amax(1).clamp(min=2.0 ** -100) / 127}
    if op == "matmul":
        return _exact_product(s["xq"], s["xs"], s["wq"], s["ws"])
    if op == "balance":
        return _exact_balance(s)
    T, k = case["T"], case["k"]
    expert = torch.repeat_interleave(torch.arange(case["E"], device=DEV), (s["offsets"][1:] - s["offsets"][:-1]).long())
    route = s["perm"].long()
    if op == "gateup":
        h = torch.empty(T * k, case["f"], dtype=torch.float64, device=DEV)
        for e in expert.unique().tolist():
            r = (expert == e).nonzero()[:, 0]
            t = route[r] // k
            gate = _exact_product(s["xq"][t], s["xs"][t], s["wq_g"][e], s["ws_g"][e])
            h[r] = gate * torch.sigmoid(gate) * _exact_product(s["xq"][t], s["xs"][t], s["wq_u"][e], s["ws_u"][e])
        return h
    y = torch.zeros(T, case["d"], dtype=torch.float64, device=DEV) if s["add"] is None else s["add"].double()
    for e in expert.unique().tolist():
        r = (expert == e).nonzero()[:, 0]
        ye = _exact_product(s["hq"][r], s["hs"][r], s["wq"][e], s["ws"][e])
        y.index_add_(0, route[r] // k, ye * s["wt"].view(-1)[route[r], None].double())
    return y


def work(case):
    op = case["op"]
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * ((2 if case["dtype"] == "bf16" else 4) + 1) + 4 * M, "flops": 3 * M * K}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K + 4 * (M + N) + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        z = T * E * (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": (2 if case["grad"] else 1) * z + 4 * T * k + 4 * S * (E + 3), "flops": (25 if case["grad"] else 10) * T * E}
    T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
    used = _distinct(T, E, k, case["skew"])
    if op == "gateup":
        return {"bytes": T * (d + 4) + used * 2 * f * (d + 4) + T * k * f * (2 if case["out"] == "bf16" else 4), "flops": 4 * T * k * f * d}
    return {"bytes": T * k * (f + 4) + used * d * (f + 4) + 4 * T * d * (2 if case["add"] else 1), "flops": 2 * T * k * f * d}


def _distinct(T, E, k, skew):
    """How many experts T tokens reach on average, each taking k by their popularity."""
    total = sum((e + 1.0) ** -skew for e in range(E))
    return sum(1.0 - (1.0 - min(1.0, k * (e + 1.0) ** -skew / total)) ** T for e in range(E))
