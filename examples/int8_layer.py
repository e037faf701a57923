"""A routed-expert layer on int8 weights, as a serving loop calls it, and how its routes load the experts.

Makes a layer of random weights (384 experts, 6 per token, d = 4096, f = 2048,
a shared expert, a sigmoid gate with a balance bias), runs one token, 8 tokens and a
1024-token prompt, and prints the time of each, the balance loss of the prompt (1 is
an even load) and how far a few tokens are from the same layer in fp32 on the weights
that the codes stand for.  Then takes the balance loss's gradient for the router.

    python examples/int8_layer.py [--experts 384] [--width 4096] [--hidden 2048] [--tokens 1,8,1024]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_moe_amd import balance, int8, lib  # noqa: E402


def weights(E, N, K, g):
    """Random weights of standard deviation 0.02, quantised an expert at a time."""
    q, s = torch.empty(E, N, K, dtype=torch.int8, device="cuda"), torch.empty(E, N, device="cuda")
    for e in range(E):
        q[e], s[e] = int8.quantize_weight(0.02 * torch.randn(N, K, device="cuda", generator=g))
    return q, s


def reference(layer, x, idx, wt):
    """The layer's sum for given routes, in fp32 on the codes' values."""
    def ffn(w, v):
        gate, up, down = (q.float() * s[:, None] for q, s in w)
        return (torch.nn.functional.silu(v @ gate.t()) * (v @ up.t())) @ down.t()

    out = []
    for t in range(x.shape[0]):
        v = x[t: t + 1].float()
        y = ffn(layer.shared, v)
        for e, w in zip(idx[t].tolist(), wt[t].tolist()):
            if e >= 0:
                y = y + w * ffn([(q[e], s[e]) for q, s in (layer.w_gate, layer.w_up, layer.w_down)], v)
        out.append(y)
    return torch.cat(out)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--experts", type=int, default=384)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--tokens", default="1,8,1024")
    a = ap.parse_args(argv)
    tokens = [int(t) for t in a.tokens.split(",")]
    E, d, f, k = a.experts, a.width, a.hidden, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    bias = 0.05 * torch.randn(E, device="cuda", generator=g)
    gate = lib.gate(E, k, score="sigmoid", scale=2.5, bias=bias)
    shared = [tuple(t[0] for t in weights(1, *s, g)) for s in ((f, d), (f, d), (d, f))]
    w_router = 0.02 * torch.randn(E, d, device="cuda", generator=g)
    layer = int8.Int8Layer(w_router, gate, weights(E, f, d, g), weights(E, f, d, g), weights(E, d, f, g), shared,
                           max_tokens=max(tokens))
    for T in tokens:
        x = torch.randn(T, d, device="cuda", generator=g).to(torch.bfloat16)
        y = torch.empty(T, d, device="cuda")
        layer.forward(x, y)  # (loads the kernels)
        n = 20
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(n):
            layer.forward(x, y)
        end.record()
        end.synchronize()
        counts, _, loss = layer.balance(T)
        few = min(T, 4)
        ref = reference(layer, x[:few], layer.idx[:few], layer.wt[:few])
        err = float((y[:few] - ref).norm() / ref.norm())
        print(f"{T:5d} tokens: {1e3 * start.elapsed_time(end) / n:9.1f} us, {int((counts > 0).sum())} experts, the fullest "
              f"{int(counts.max())} routes, balance loss {float(loss):.3f}, off by {err:.3f} (8-bit activations)")
    # the router's gradient of the loss of the last batch: logits by torch, routes by the gate
    w = w_router.clone().requires_grad_()
    z = x.float() @ w.t()
    loss, _, _ = balance.balance_loss(z, layer.idx[: x.shape[0]], score="sigmoid", alpha=0.001)
    loss.sum().backward()
    print(f"gradient of the balance loss for the router: norm {float(w.grad.norm()):.3e}")
    return w.grad


if __name__ == "__main__":
    main()
