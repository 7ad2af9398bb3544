"""The feed-forward operators on torch tensors: the gated block (and its autograd form), row
quantization and the 8-bit products.

The checks of arguments, the allocation of results and the call into the C ABI are in the compiled
module ``_calls`` (csrc/torch_calls.cpp), which runs them on the device of the tensors and on its
current stream.
"""
from __future__ import annotations

import os

import torch
from torch.autograd.function import once_differentiable

from . import _binding, build

if not os.path.exists(_binding.CALLS_PATH):
    raise ImportError(f"{_binding.CALLS_PATH} is not built; run `python -m tiled_dense_gemm_fp16_b200.build` "
                      "(there is no fallback implementation)")
_binding.lib()  # the C library first: _calls links to it

from . import _calls  # noqa: E402

if _calls.target != build.calls_target():
    raise ImportError(f"{_binding.CALLS_PATH} was built for {_calls.target}, this is {build.calls_target()}; run "
                      "`python -m tiled_dense_gemm_fp16_b200.build`")
_calls.set_error(_binding.TGError)


class _On:
    """Context of a call on a given stream.

    What the call allocates belongs to that stream.  Tensors made on another stream are recorded on it, so
    that their memory is not reused before the call's work is done (making the streams wait for each
    other stays the caller's part)."""

    def __init__(self, stream, *tensors):
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                if t.device != stream.device:
                    raise ValueError(f"stream is on {stream.device}, a tensor on {t.device}")
                if stream != torch.cuda.current_stream(t.device):
                    t.record_stream(stream)
        self.context = torch.cuda.stream(stream)

    def __enter__(self):
        self.context.__enter__()

    def __exit__(self, *exc):
        self.context.__exit__(*exc)


def gated(x, w_gate, w_up, act="silu", out=None, save=False, stream=None, workspace="auto"):
    """act(x @ w_gate^T) * (x @ w_up^T) for float16 or bfloat16 CUDA tensors: x (..., K), w_gate and
    w_up (N, K) as linear layers store them (the halves of one (2N, K) weight do too).

    ``act``: "silu", "gelu" (tanh form) or "relu".  Returns H (..., N); with ``save`` the tuple
    (H, gate, up) with the two projections, which ``gated_backward`` takes (their rows may have gaps).
    ``out`` receives H (it may lie beside x in one wider buffer).  Rows may have any stride; ``workspace``
    ("auto", None or a uint8 CUDA tensor) is needed only where a row stride or base is off 16 bytes.  Runs on
    ``stream``, or the current one; what the call allocates belongs to that stream.  Nothing is recorded for
    autograd, in reverse or forward mode: ``gated_block`` is the differentiable form.
    """
    if stream is None:
        return _calls.gated(x, w_gate, w_up, act, out, save, workspace)
    with _On(stream, x, w_gate, w_up, out, workspace):
        return _calls.gated(x, w_gate, w_up, act, out, save, workspace)


def gated_backward(grad, x, w_gate, w_up, gate, up, act="silu", needs=(True, True, True), stream=None,
                   workspace="auto"):
    """Gradients of ``gated`` for grad = dH (..., N), with the projections that ``gated(..., save=True)``
    returned: (dx, dw_gate, dw_up), None where ``needs`` is false.

    gate and up, and dG and dU between the two steps, are of the operands' 16-bit type; sums are 32-bit.
    ``workspace``: "auto" lets torch allocate the bytes for dG and dU; a uint8 CUDA tensor is used as
    given (calls whose work may overlap need one each).
    """
    if stream is None:
        return _calls.gated_backward(grad, x, w_gate, w_up, gate, up, act, *needs, workspace)
    with _On(stream, grad, x, w_gate, w_up, gate, up, workspace):
        return _calls.gated_backward(grad, x, w_gate, w_up, gate, up, act, *needs, workspace)


def quantize_i8(x, out=None, scales=None, stream=None):
    """Rows of x (..., K), float16 or bfloat16, as 8-bit integers with one scale each: (codes, scales) with
    codes (..., K) int8 and scales (...) float32, scale = max |x| / 127, codes = x / scale rounded to
    nearest even.  Rows of codes that the call allocates start on 16-byte boundaries whatever K is, as
    ``gemm_i8`` and ``gated_i8`` want them.  Serves activations (a row is a token) and weights (a row is
    a channel).  Rows of zeros: scale 0.  Rows with an infinity or a NaN: scale NaN, codes 0."""
    if stream is None:
        return _calls.quantize_i8(x, out, scales)
    with _On(stream, x, out, scales):
        return _calls.quantize_i8(x, out, scales)


def gemm_i8(a, a_scale, w, w_scale, bias=None, relu=False, dtype=None, out=None, stream=None):
    """(a @ w^T) * a_scale * w_scale + bias, with an optional ReLU, for int8 CUDA tensors a (..., K) and
    w (N, K) with a float32 scale for each of their rows; bias (N,) of the result's type.

    Returns (..., N) of ``dtype`` (float16 unless given, or ``out``'s).  The integer sums are exact.
    Rows of a and w must start on 16-byte boundaries (as those of ``quantize_i8`` do)."""
    if stream is None:
        return _calls.gemm_i8(a, a_scale, w, w_scale, bias, relu, dtype, out)
    with _On(stream, a, a_scale, w, w_scale, bias, out):
        return _calls.gemm_i8(a, a_scale, w, w_scale, bias, relu, dtype, out)


def gated_i8(a, a_scale, w_gate, gate_scale, w_up, up_scale, act="silu", dtype=None, out=None, stream=None):
    """``gated`` on 8-bit operands: a (..., K) int8 with a scale a row, w_gate and w_up (N, K) int8 with a
    scale a row.  Returns (..., N) of ``dtype`` (float16 unless given, or ``out``'s).  Operands as for
    ``gemm_i8``."""
    if stream is None:
        return _calls.gated_i8(a, a_scale, w_gate, gate_scale, w_up, up_scale, act, dtype, out)
    with _On(stream, a, a_scale, w_gate, gate_scale, w_up, up_scale, out):
        return _calls.gated_i8(a, a_scale, w_gate, gate_scale, w_up, up_scale, act, dtype, out)


# ---------------------------------------------------------------------------
# Autograd
# ---------------------------------------------------------------------------

def _rows(t):
    """t, or a dense copy where its rows are not evenly spaced with adjacent columns (an expanded gradient) or its
    values are the negatives of its memory."""
    if t.is_neg():
        return t.resolve_neg().contiguous()
    if t.is_contiguous():
        return t
    if t.dim() >= 2 and t.numel() and (t.shape[-1] == 1 or t.stride(-1) == 1):
        try:
            two = t.view(-1, t.shape[-1])
            if two.shape[0] == 1 or two.stride(0) >= two.shape[1]:
                return t
        except RuntimeError:
            pass
    return t.contiguous()


class GatedBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act):
        x, w_gate, w_up = _rows(x), _rows(w_gate), _rows(w_up)
        out, gate, up = gated(x, w_gate, w_up, act=act, save=True)
        ctx.save_for_backward(x, w_gate, w_up, gate, up)
        ctx.act = act
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w_gate, w_up, gate, up = ctx.saved_tensors
        return (*gated_backward(_rows(grad), x, w_gate, w_up, gate, up, act=ctx.act, needs=ctx.needs_input_grad[:3]),
                None)


def gated_block(x, w_gate, w_up, act="silu"):
    """``gated`` under autograd: gradients reach x, w_gate and w_up (those that ask for one).

    Runs on the current stream.  Without a gradient to take, neither projection is stored.  Reverse mode, once:
    second derivatives, forward mode (dual tensors) and the transforms of ``torch.func`` are refused.  Under
    ``torch.compile`` the call runs as it is, between compiled parts.  To capture a training step into a CUDA
    graph, let go of every earlier autograd graph of the same leaves first, as torch asks for any operator."""
    if _calls.has_tangent(x, w_gate, w_up):
        raise NotImplementedError("gated_block has no forward-mode derivative")
    if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad):
        return GatedBlock.apply(x, w_gate, w_up, act)
    return gated(_rows(x), _rows(w_gate), _rows(w_up), act=act)
