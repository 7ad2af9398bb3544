"""Products whose rows pick their weight, on torch tensors: the grouped products of experts (with their gradients
and an autograd form), and a shared projection with the low-rank adapters of many requests.

As for the feed-forward operators, checks of arguments, results and the call into the C ABI are in the compiled
module ``_calls``; a call runs on the device of its tensors and on its current stream.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .feedforward import _calls, _On, _rows


def grouped(x, w, ends, out=None, stream=None, workspace="auto"):
    """Rows of x (..., K), lying group by group, each times the weight of its group: w (G, N, K) holds the groups'
    weights as linear layers store them, ends (G,) int32 on the device the row behind each group's last
    (``counts.cumsum(0, dtype=torch.int32)`` of the groups' sizes, which may be 0).  float16 or bfloat16.

    Returns (..., N).  The ends are read by the kernels only: nothing waits for the device, and a captured call may be
    replayed with other groups.  Rows behind the last end belong to no group: they are zeros in a new result, and left as
    they are in a given ``out``.  Rows of x, of w and from weight to weight may have any stride; ``workspace``
    ("auto", None or a uint8 CUDA tensor) is needed only where one, or a base, is off 16 bytes (weights are
    copied then, if their rows are evenly spaced).  Runs on ``stream``, or the current one.  Nothing is
    recorded for autograd: ``grouped_linear`` is the differentiable form."""
    if stream is None:
        return _calls.grouped(x, w, ends, out, workspace)
    with _On(stream, x, w, ends, out, workspace):
        return _calls.grouped(x, w, ends, out, workspace)


def grouped_backward(grad, x, w, ends, needs=(True, True), stream=None, workspace="auto"):
    """Gradients of ``grouped`` for grad = dY (..., N): (dx, dw) with dx like x and dw (G, N, K), None where ``needs`` is
    false.  Rows without a group have dx = 0 and nothing in dw; dw of a group without rows is 0.  Sums are 32-bit."""
    if stream is None:
        return _calls.grouped_backward(grad, x, w, ends, *needs, workspace)
    with _On(stream, grad, x, w, ends, workspace):
        return _calls.grouped_backward(grad, x, w, ends, *needs, workspace)


def lora(x, w, a, b, index, scale=None, bias=None, out=None, stream=None, workspace="auto"):
    """x @ w^T + scale[r] (x @ a[r]^T) @ b[r]^T + bias with an adapter r = index[row] for each row, float16 or bfloat16:
    x (..., K), w (N, K), a (adapters, rank, K), b (adapters, N, rank), index int32 with a value for each row of x.

    Rows whose index is outside [0, adapters), -1 say, have no adapter.  Rows may come in any order; those of one
    request next to each other are faster.  ``scale``: (adapters,) float32, or None for 1.  ``bias``: (N,) of x's type.
    rank is a multiple of 8, at most 512, and rows of a and b start on 16-byte boundaries (pad a rank with zeros
    once); x, w and ``out`` may have any row stride.  x @ a[r]^T, scaled, is rounded to the 16-bit type (in float16 times
    a power of two where its range needs one; such rows are slower); sums are 32-bit.  No value of another request or adapter reaches a row.  For serving: nothing is recorded for autograd.  ``workspace``
    ("auto" or a uint8 CUDA tensor) holds those inner products; calls whose work may overlap need one each."""
    if stream is None:
        return _calls.lora(x, w, a, b, index, scale, bias, out, workspace)
    with _On(stream, x, w, a, b, index, scale, bias, out, workspace):
        return _calls.lora(x, w, a, b, index, scale, bias, out, workspace)


# ---------------------------------------------------------------------------
# Autograd
# ---------------------------------------------------------------------------

def _stacked(w):
    """w, or a dense copy where its rows do not lie apart with adjacent columns or its values are negated."""
    if w.is_neg():
        return w.resolve_neg().contiguous()
    if w.dim() == 3 and w.numel() and not w.is_contiguous():
        G, N, K = w.shape
        if not ((K == 1 or w.stride(2) == 1) and (N == 1 or w.stride(1) >= K) and (G == 1 or w.stride(0) >= K)):
            return w.contiguous()
        on16 = w.data_ptr() % 16 == 0 and (N == 1 or w.stride(1) % 8 == 0) and (G == 1 or w.stride(0) % 8 == 0)
        if not on16 and G > 1 and w.stride(0) != N * w.stride(1):  # unevenly spaced rows that TMA cannot describe
            return w.contiguous()
    return w


class GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, ends):
        x, w = _rows(x), _stacked(w)
        ctx.save_for_backward(x, w, ends)
        return grouped(x, w, ends)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w, ends = ctx.saved_tensors
        return (*grouped_backward(_rows(grad), x, w, ends, needs=ctx.needs_input_grad[:2]), None)


def grouped_linear(x, w, ends):
    """``grouped`` under autograd: gradients reach x and w (those that ask for one).

    Runs on the current stream.  Reverse mode, once: second derivatives, forward mode (dual tensors) and the transforms of
    ``torch.func`` are refused.  To capture a training step into a CUDA graph, let go of every earlier autograd
    graph of the same leaves first, as torch asks for any operator."""
    if _calls.has_tangent(x, w):
        raise NotImplementedError("grouped_linear has no forward-mode derivative")
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        return GroupedLinear.apply(x, w, ends)
    return grouped(_rows(x), _stacked(w), ends)
