"""A routed-expert layer on block-scaled E4M3 weights.

Memory management and call order only: the gate, the bucketing, the
quantisation of the activations and the experts' products all run in the HIP
library (lib.router_logits, gate_topk, bucket, blockscale_quantize, _gateup,
_matmul and _down).
"""
from __future__ import annotations

import torch

from . import lib

E4M3 = torch.float8_e4m3fn


def quantize_weight(w: torch.Tensor):
    """(codes, scales) of weights [..., N, K]: E4M3 with one scale per 128 x 128
    block, the largest value of a block becoming 448 (a preparation step for
    weights that do not come quantised)."""
    N, K = w.shape[-2:]
    f = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -N % 128))
    blocks = f.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))  # [..., NB, 128, KB, 128]
    s = blocks.abs().amax((-3, -1)).clamp(min=2.0 ** -100) / 448.0
    q = (blocks / s[..., :, None, :, None]).flatten(-4, -3).flatten(-2, -1)[..., :N, :K]
    return q.clamp(-448.0, 448.0).to(E4M3).contiguous(), s.contiguous()


class BlockScaleLayer:
    """y = sum_j wt_j * expert_j(x) (+ shared(x)) for up to max_tokens tokens.

    w_router fp32 [E][d], d a power of two in [256, 8192] (router_logits' limits);
    gate: a lib.gate() description; each of w_gate, w_up [E][f][d] and w_down
    [E][d][f] a (codes, scales) pair as quantize_weight returns it; shared: None or
    such pairs of one expert, (gate, up, down) of
    [f_s][d], [f_s][d], [d][f_s].  Buffers are allocated here, once; forward
    allocates nothing and its calls can be captured into a graph.  One call at
    a time: calls on several streams need a layer object each.
    """

    def __init__(self, w_router, gate: lib.MoeGate, w_gate, w_up, w_down, shared=None, max_tokens: int = 1024):
        E, d = w_router.shape
        self.w_router, self.gate, self.max_tokens = w_router, gate, max_tokens
        self.w_gate, self.w_up, self.w_down, self.shared = w_gate, w_up, w_down, shared
        self.E, self.d, self.f, self.k = E, d, w_gate[0].shape[1], gate.top_k
        if gate.n_experts != E:
            raise ValueError(f"BlockScaleLayer: the gate has {gate.n_experts} experts, the router {E}")
        dev, T, R = w_router.device, max_tokens, max_tokens * self.k

        def new(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=dev)

        blocks = lib.scale_blocks
        self.z = new(T, E)
        self.idx, self.wt = new(T, self.k, dtype=torch.int32), new(T, self.k)
        self.counts, self.offsets = new(E, dtype=torch.int32), new(E + 1, dtype=torch.int32)
        self.perm, self.pos = new(R, dtype=torch.int32), new(R, dtype=torch.int32)
        self.xq, self.xs = new(T, d, dtype=E4M3), new(T, blocks(d))
        self.hq, self.hs = new(R, self.f, dtype=E4M3), new(R, blocks(self.f))
        self.work = new(lib.blockscale_down_workspace_bytes(T, self.k, d), dtype=torch.uint8)
        self.add = None
        if shared is not None:
            f_s = shared[0][0].shape[0]
            self.sq, self.ss, self.add = new(T, f_s, dtype=E4M3), new(T, blocks(f_s)), new(T, d)
            self.shared_perm = torch.arange(T, dtype=torch.int32, device=dev)
            # the shared expert is one bucket with every row: [0, t] for t
            # tokens, each pair 16-byte aligned
            self.shared_offsets = torch.zeros(T + 1, 4, dtype=torch.int32, device=dev)
            self.shared_offsets[:, 1] = torch.arange(T + 1, dtype=torch.int32, device=dev)
            # the largest workspace of any token count up to max_tokens
            self.shared_work = new(max(lib.blockscale_matmul_workspace_bytes(t, d, f_s) for t in range(1, T + 1)),
                                   dtype=torch.uint8)

    def forward(self, x, y, stream=None):
        """x [T][d] (float32 or bfloat16) to y fp32 [T][d]; the routes are left
        in self.idx and self.wt, their first T rows."""
        T, R = x.shape[0], x.shape[0] * self.k
        if T > self.max_tokens:
            raise ValueError(f"BlockScaleLayer: {T} tokens, made for {self.max_tokens}")
        if T == 0:
            return y
        z, idx, wt, perm, pos = self.z[:T], self.idx[:T], self.wt[:T], self.perm[:R], self.pos[:R]
        xq, xs, hq, hs = self.xq[:T], self.xs[:T], self.hq[:R], self.hs[:R]
        lib.router_logits(self.w_router, x, z, stream=stream)
        lib.gate_topk(self.gate, z, idx, wt, stream=stream)
        lib.bucket(idx, self.E, self.counts, self.offsets, perm, pos, stream=stream)
        lib.blockscale_quantize(x, xq, xs, stream=stream)
        lib.blockscale_gateup(xq, xs, self.k, self.offsets, perm, *self.w_gate, *self.w_up, hq, hs, stream=stream)
        add = None
        if self.shared is not None:
            (gq, gs), (uq, us), (dq, ds) = self.shared
            sq, ss, add = self.sq[:T], self.ss[:T], self.add[:T]
            lib.blockscale_gateup(xq, xs, 1, self.shared_offsets[T, :2], self.shared_perm[:T], gq[None], gs[None],
                                  uq[None], us[None], sq, ss, stream=stream)
            lib.blockscale_matmul(sq, ss, dq, ds, add, self.shared_work, stream=stream)
        lib.blockscale_down(hq, hs, wt, self.offsets, pos, *self.w_down, y, self.work, add=add, stream=stream)
        return y
