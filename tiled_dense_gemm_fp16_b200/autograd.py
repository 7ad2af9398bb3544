"""The gated feed-forward block under torch's autograd."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _binding


def _rows(t):
    """t, or a dense copy where its rows are not evenly spaced with adjacent columns (an expanded gradient)."""
    if t.dim() >= 1 and (t.shape[-1] <= 1 or t.stride(-1) == 1):
        try:
            two = t.view(-1, t.shape[-1]) if t.numel() else t
            if two.dim() != 2 or two.shape[0] <= 1 or two.stride(0) >= two.shape[1]:
                return t
        except RuntimeError:
            pass
    return t.contiguous()


class GatedBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act):
        x, w_gate, w_up = _rows(x), _rows(w_gate), _rows(w_up)
        out, gate, up = _binding.gated(x, w_gate, w_up, act=act, save=True)
        ctx.save_for_backward(x, w_gate, w_up, gate, up)
        ctx.act = act
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w_gate, w_up, gate, up = ctx.saved_tensors
        return (*_binding.gated_backward(_rows(grad), x, w_gate, w_up, gate, up, act=ctx.act,
                                         needs=ctx.needs_input_grad[:3]), None)


def gated_block(x, w_gate, w_up, act="silu"):
    if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad):
        return GatedBlock.apply(x, w_gate, w_up, act)
    return _binding.gated(_rows(x), _rows(w_gate), _rows(w_up), act=act)
