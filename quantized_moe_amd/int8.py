"""A routed-expert layer on int8 weights with a scale per output channel.

Memory management and call order only: the gate, the bucketing, the quantisation
of the activations (one scale per token) and the experts' products all run in the
HIP library (lib.router_logits, gate_topk, bucket, int8_quantize, _gateup, _matmul
and _down), and so does the balance of the routes (lib.balance_loss).
"""
from __future__ import annotations

import torch

from . import lib


def quantize_weight(w: torch.Tensor):
    """(codes, scales) of weights [..., N, K]: int8 with one scale per output channel,
    the largest value of a channel becoming 127 (a preparation step for weights that
    do not come quantised)."""
    f = w.float()
    s = f.abs().amax(-1).clamp(min=2.0 ** -100) / 127.0
    return (f / s[..., None]).round().clamp(-127, 127).to(torch.int8).contiguous(), s.contiguous()


class Int8Layer:
    """y = sum_j wt_j * expert_j(x) (+ shared(x)) for up to max_tokens tokens.

    w_router fp32 [E][d], d a power of two in [256, 8192] (router_logits' limits);
    gate: a lib.gate() description; each of w_gate, w_up [E][f][d] and w_down
    [E][d][f] a (codes, scales) pair as quantize_weight returns it; shared: None or
    such pairs of one expert, (gate, up, down) of [f_s][d], [f_s][d], [d][f_s].
    Buffers are allocated here, once; forward and balance allocate nothing and their
    calls can be captured into a graph.  One call at a time: calls on several streams
    need a layer object each.
    """

    def __init__(self, w_router, gate: lib.MoeGate, w_gate, w_up, w_down, shared=None, max_tokens: int = 1024,
                 max_sequences: int = 1):
        E, d = w_router.shape
        self.w_router, self.gate, self.max_tokens, self.max_sequences = w_router, gate, max_tokens, max_sequences
        self.w_gate, self.w_up, self.w_down, self.shared = w_gate, w_up, w_down, shared
        self.E, self.d, self.f, self.k = E, d, w_gate[0].shape[1], gate.top_k
        if gate.n_experts != E:
            raise ValueError(f"Int8Layer: the gate has {gate.n_experts} experts, the router {E}")
        dev, T, R, S = w_router.device, max_tokens, max_tokens * self.k, max_sequences

        def new(*shape, dtype=torch.float32):
            return torch.zeros(shape, dtype=dtype, device=dev)

        self.z = new(T, E)
        self.idx, self.wt = new(T, self.k, dtype=torch.int32), new(T, self.k)
        self.counts, self.offsets = new(E, dtype=torch.int32), new(E + 1, dtype=torch.int32)
        self.perm, self.pos = new(R, dtype=torch.int32), new(R, dtype=torch.int32)
        self.xq, self.xs = new(T, d, dtype=torch.int8), new(T)
        # SwiGLU's outputs wait for their row's maximum in fp32: in bf16 they would be
        # rounded by up to a quarter of a code before they become codes
        self.h, self.hq, self.hs = new(R, self.f), new(R, self.f, dtype=torch.int8), new(R)
        self.work = new(lib.int8_down_workspace_bytes(T, self.k, d), dtype=torch.uint8)
        self.load, self.tokens, self.loss = new(S, E, dtype=torch.int32), new(S, dtype=torch.int32), new(S)
        self.balance_work = new(lib.balance_loss_workspace_bytes(T, S, E), dtype=torch.uint8)
        self.add = None
        if shared is not None:
            f_s = shared[0][0].shape[0]
            self.sh, self.sq, self.ss, self.add = new(T, f_s), new(T, f_s, dtype=torch.int8), new(T), new(T, d)
            self.shared_perm = torch.arange(T, dtype=torch.int32, device=dev)
            # the shared expert is one bucket with every row: [0, t] for t
            # tokens, each pair 16-byte aligned
            self.shared_offsets = torch.zeros(T + 1, 4, dtype=torch.int32, device=dev)
            self.shared_offsets[:, 1] = torch.arange(T + 1, dtype=torch.int32, device=dev)
            # the largest workspace of any token count up to max_tokens
            self.shared_work = new(max(lib.int8_matmul_workspace_bytes(t, d, f_s) for t in range(1, T + 1)), dtype=torch.uint8)

    def forward(self, x, y, stream=None):
        """x [T][d] (float32 or bfloat16) to y fp32 [T][d]; the router's logits and the
        routes are left in self.z, self.idx and self.wt, their first T rows."""
        T, R = x.shape[0], x.shape[0] * self.k
        if T > self.max_tokens:
            raise ValueError(f"Int8Layer: {T} tokens, made for {self.max_tokens}")
        if T == 0:
            return y
        z, idx, wt, perm, pos = self.z[:T], self.idx[:T], self.wt[:T], self.perm[:R], self.pos[:R]
        xq, xs, h, hq, hs = self.xq[:T], self.xs[:T], self.h[:R], self.hq[:R], self.hs[:R]
        lib.router_logits(self.w_router, x, z, stream=stream)
        lib.gate_topk(self.gate, z, idx, wt, stream=stream)
        lib.bucket(idx, self.E, self.counts, self.offsets, perm, pos, stream=stream)
        lib.int8_quantize(x, xq, xs, stream=stream)
        lib.int8_gateup(xq, xs, self.k, self.offsets, perm, *self.w_gate, *self.w_up, h, stream=stream)
        lib.int8_quantize(h, hq, hs, stream=stream)
        add = None
        if self.shared is not None:
            (gq, gs), (uq, us), (dq, ds) = self.shared
            sh, sq, ss, add = self.sh[:T], self.sq[:T], self.ss[:T], self.add[:T]
            lib.int8_gateup(xq, xs, 1, self.shared_offsets[T, :2], self.shared_perm[:T], gq[None], gs[None], uq[None],
                            us[None], sh, stream=stream)
            lib.int8_quantize(sh, sq, ss, stream=stream)
            lib.int8_matmul(sq, ss, dq, ds, add, self.shared_work, stream=stream)
        lib.int8_down(hq, hs, wt, self.offsets, pos, *self.w_down, y, self.work, add=add, stream=stream)
        return y

    def balance(self, T: int, alpha: float = 1.0, starts=None, stream=None):
        """How the last forward call's T tokens load the experts: (counts int32 [S][E],
        tokens int32 [S], loss fp32 [S]) of the S sequences that starts (int32 [S + 1],
        or None: one) cuts them into, in the layer's buffers."""
        S = 1 if starts is None else starts.shape[0] - 1
        if T > self.max_tokens or S > self.max_sequences:
            raise ValueError(f"Int8Layer: {T} tokens in {S} sequences, made for {self.max_tokens} in {self.max_sequences}")
        counts, tokens, loss = self.load[:S], self.tokens[:S], self.loss[:S]
        score = "softmax" if self.gate.score == lib.MOE_SCORE_SOFTMAX else "sigmoid"
        lib.balance_loss(self.z[:T], self.idx[:T], counts, tokens, loss, self.balance_work, score=score, alpha=alpha,
                         starts=starts, stream=stream)
        return counts, tokens, loss
