"""A routed-expert layer on block-scaled E4M3 weights, as a serving loop calls it.

Makes a layer of random weights (384 experts, 6 per token, d = 4096, f = 2048,
a shared expert, a grouped sigmoid gate with a balance bias), runs one token, 8
tokens and a 1024-token prompt, and prints the time of each and how far a few
tokens are from the same layer in fp32 on the weights that the codes stand for.

    python examples/blockscale_layer.py [--experts 384] [--tokens 1,8,1024]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_moe_amd import blockscale, lib  # noqa: E402


def values(q, s):
    """The fp32 values of one block-scaled matrix."""
    N, K = q.shape
    return q.float() * s.repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[:N]


def weights(E, N, K, g):
    """Random weights of standard deviation 0.02, quantised an expert at a time."""
    q = torch.empty(E, N, K, dtype=blockscale.E4M3, device="cuda")
    s = torch.empty(E, lib.scale_blocks(N), lib.scale_blocks(K), device="cuda")
    for e in range(E):
        q[e], s[e] = blockscale.quantize_weight(0.02 * torch.randn(N, K, device="cuda", generator=g))
    return q, s


def reference(layer, x, idx, wt):
    """The layer's sum for given routes, in fp32 on the codes' values."""
    def ffn(w, v):
        gate, up, down = (values(*p) for p in w)
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


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--experts", type=int, default=384)
    ap.add_argument("--tokens", default="1,8,1024")
    a = ap.parse_args()
    tokens = [int(t) for t in a.tokens.split(",")]
    E, d, f, k = a.experts, 4096, 2048, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    torch.backends.cuda.matmul.allow_tf32 = False
    bias = 0.05 * torch.randn(E, device="cuda", generator=g)
    gate = lib.gate(E, k, score="sigmoid", n_groups=8, top_groups=4, group_score="top2", scale=2.5, bias=bias)
    shared = [tuple(t[0] for t in weights(1, *s, g)) for s in ((f, d), (f, d), (d, f))]
    layer = blockscale.BlockScaleLayer(0.02 * torch.randn(E, d, device="cuda", generator=g), gate, weights(E, f, d, g),
                                       weights(E, f, d, g), weights(E, d, f, g), shared, max_tokens=max(tokens))
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
        few = min(T, 4)
        ref = reference(layer, x[:few], layer.idx[:few], layer.wt[:few])
        err = float((y[:few] - ref).norm() / ref.norm())
        print(f"{T:5d} tokens: {1e3 * start.elapsed_time(end) / n:9.1f} us, "
              f"{len(set(layer.idx[:T].flatten().tolist()))} experts, off by {err:.3f} (8-bit activations)")


if __name__ == "__main__":
    main()
