"""The router's balance loss as a differentiable torch function."""
from __future__ import annotations

import torch

from . import lib


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, idx, starts, score, alpha):
        (T, E), S = z.shape, 1 if starts is None else starts.shape[0] - 1
        if (E > 1 and z.stride(1) != 1) or (T > 1 and z.stride(0) < E):  # (expanded rows, too)
            z = z.contiguous()
        idx, starts = idx.contiguous(), starts if starts is None else starts.contiguous()
        counts = torch.empty(S, E, dtype=torch.int32, device=z.device)
        tokens = torch.empty(S, dtype=torch.int32, device=z.device)
        loss = torch.empty(S, dtype=torch.float32, device=z.device)
        work = torch.empty(lib.balance_loss_workspace_bytes(T, S, E), dtype=torch.uint8, device=z.device)
        lib.balance_loss(z, idx, counts, tokens, loss, work, score=score, alpha=alpha, starts=starts)
        # A copy of the routes: a gate writes the next batch's over them, and torch, which
        # cannot see that, would take those for this batch's.
        routes = idx.clone() if ctx.needs_input_grad[0] else idx
        ctx.save_for_backward(z, routes, counts, tokens, starts)
        ctx.score, ctx.alpha = score, alpha
        ctx.mark_non_differentiable(counts, tokens)
        return loss, counts, tokens

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, *_):
        z, idx, counts, tokens, starts = ctx.saved_tensors
        dz = torch.empty(z.shape, dtype=z.dtype, device=z.device)
        lib.balance_loss_backward(z, idx, counts, tokens, grad_loss.contiguous(), dz, score=ctx.score, alpha=ctx.alpha,
                                  starts=starts)
        return dz, None, None, None, None


def balance_loss(z: torch.Tensor, idx: torch.Tensor, score: str = "softmax", alpha: float = 1.0, starts=None):
    """(loss fp32 [S], counts int32 [S][E], tokens int32 [S]) of router logits z [T][E]
    (float32 or bfloat16) and the routes idx int32 [T][k] that a gate chose from them, for
    the S sequences that starts (int32 [S + 1], or None: one) cuts the tokens into, with
    any strides.  The
    loss is differentiable with respect to z, once; the counts are constants of it.  idx may
    be a buffer that later calls write over: the backward pass has a copy of it.  z, starts
    and the counts are kept as they are: as with any torch function, the backward pass
    refuses them once they have been written over (by lib.router_logits, a product or
    lib.balance_loss too)."""
    return _BalanceLoss.apply(z, idx, starts, score, alpha)
