"""The feed-forward operators on torch tensors: the gated block (and its autograd form), row
quantization and the 8-bit products.

Argument checks and marshalling to the C ABI only.  A decoding step makes these calls for a few
microseconds of GPU work each, so the checks touch each property of a tensor once, a call on the
current stream enters no context, and sizes go to new_empty as numbers (1.4 us; as a tuple 1.8).
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _binding
from ._binding import ACT_GELU, ACT_RELU, ACT_SILU, TYPE_BF16, TYPE_F16, GatedOptions, Status, TGError

_ACTS = {"relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU}
_TYPES = {torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16}
_F32, _I8, _U8 = torch.float32, torch.int8, torch.uint8
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

_lib = _binding.lib()
_options_cache: dict = {}


def _options(*fields):
    """A tg_gated_options reference for these leading fields (the values are all there is to it)."""
    ref = _options_cache.get(fields)
    if ref is None:
        if len(_options_cache) >= 1024:
            _options_cache.clear()
        ref = _options_cache[fields] = ctypes.byref(GatedOptions(*fields))
    return ref


def _codes(dtype, act="relu"):
    """The TG_TYPE_* and TG_ACT_* of these."""
    try:
        return _TYPES[dtype], _ACTS[act]
    except KeyError:
        if dtype not in _TYPES:
            raise TypeError(f"expected torch.float16 or torch.bfloat16, got {dtype}") from None
        raise ValueError(f"unknown activation {act!r}; one of {sorted(_ACTS)}") from None


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _flat(t, name):
    """(..., K) as (rows, K), without a copy."""
    if t.dim() == 2:
        return t
    if t.dim() < 1:
        raise ValueError(f"{name} needs at least one dimension")
    rows = 1
    for d in t.shape[:-1]:
        rows *= d
    try:
        return t.view(rows, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: the leading dimensions of shape {tuple(t.shape)} with strides {t.stride()} "
                         "are not evenly spaced rows") from None


def _row_stride(t, rows, cols, name):
    """Elements between the rows of a 2-D tensor whose columns are adjacent (0: dense, or a single row)."""
    if t.is_contiguous():
        return 0
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have adjacent columns (stride 1), got strides {(s0, s1)}")
    if rows <= 1 or cols == 0:
        return 0
    if s0 < cols:
        raise ValueError(f"{name} has overlapping rows: strides {(s0, s1)} for shape {(rows, cols)}")
    return s0


def _matrix(t, name, rows, cols, dtype, index):
    """Check a 2-D operand; returns its row stride (0: dense)."""
    if t.is_contiguous() and t.dtype is dtype and t.shape == (rows, cols) and t.get_device() == index:
        return 0
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    return _row_stride(t, rows, cols, name)


def _vector(t, name, n, dtype, index):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be {n} contiguous values on cuda:{index}")
    return t.data_ptr()


def _result(out, lead, M, N, dtype, index):
    """(2-D view of the given result, its row stride)."""
    if out.shape != (*lead, N):
        raise ValueError(f"out must have shape {(*lead, N)}, got {tuple(out.shape)}")
    out2 = _flat(out, "out")
    return out2, _matrix(out2, "out", M, N, dtype, index)


class _Elsewhere:
    """Context of a call on another stream than the current one, or on another device than the current one.

    What the call allocates belongs to its stream.  Tensors made on another stream are recorded on it, so
    that their memory is not reused before the call's work is done (making the streams wait for each
    other stays the caller's part)."""

    def __init__(self, index, stream, tensors):
        self.context = torch.cuda.device(index)
        if stream is not None:
            if stream.device.index != index:
                raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
            if stream != torch.cuda.current_stream(index):
                for t in tensors:
                    if isinstance(t, torch.Tensor) and t.is_cuda:
                        t.record_stream(stream)
            self.context = torch.cuda.stream(stream)

    def __enter__(self):
        self.context.__enter__()

    def __exit__(self, *exc):
        self.context.__exit__(*exc)


def _scratch(workspace, need, like):
    """The workspace tensor of a call that needs `need` bytes (None: none), held by the caller until it launched."""
    if need < 0:
        raise TGError(Status.INVALID_ARG, "workspace size")
    if workspace is None:
        return None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        return like.new_empty(need, dtype=_U8) if need else None
    if workspace.dtype is not _U8 or not workspace.is_contiguous() or workspace.get_device() != like.get_device():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {like.device}")
    return workspace


def _check(st, what):
    if st:
        raise TGError(st, what)


def gated(x, w_gate, w_up, act="silu", out=None, save=False, stream=None, workspace="auto"):
    """act(x @ w_gate^T) * (x @ w_up^T) for float16 or bfloat16 CUDA tensors: x (..., K), w_gate and
    w_up (N, K) as linear layers store them (the halves of one (2N, K) weight do too).

    ``act``: "silu", "gelu" (tanh form) or "relu".  Returns H (..., N); with ``save`` the tuple
    (H, gate, up) with the two projections, which ``gated_backward`` takes (their rows may have gaps).
    ``out`` receives H.  Rows may have any stride; ``workspace`` ("auto", None or a uint8 CUDA tensor) is
    needed only where a row stride or base is off 16 bytes.  Runs on ``stream``, or the current one; what
    the call allocates belongs to that stream.  Nothing is recorded for autograd: ``gated_block`` is the
    differentiable form.
    """
    index = _device(x, "x")
    if stream is not None or index != _current_device():
        with _Elsewhere(index, stream, (x, w_gate, w_up, out, workspace)):
            return gated(x, w_gate, w_up, act, out, save, None, workspace)
    x2 = _flat(x, "x")
    M, K = x2.shape
    dtype = x.dtype
    code, act_code = _codes(dtype, act)
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be (N, K), got {tuple(w_gate.shape)}")
    N = w_gate.shape[0]
    ldx = _row_stride(x2, M, K, "x")
    ldg = _matrix(w_gate, "w_gate", N, K, dtype, index)
    ldu = _matrix(w_up, "w_up", N, K, dtype, index)
    if out is None:
        ldh, out2 = 0, x.new_empty(M, N)
        out = out2 if x2 is x else out2.view(*x.shape[:-1], N)
    else:
        out2, ldh = _result(out, x.shape[:-1], M, N, dtype, index)
    options = _options(code, act_code, ldx, ldg, ldu, ldh)
    px, pg, pu = x2.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    ws, ws_ptr, ws_bytes = None, 0, 0
    if (px | pg | pu | 2 * (ldx or K) | 2 * (ldg or K) | 2 * (ldu or K)) & 15 or not isinstance(workspace, str):
        ws = _scratch(workspace, _lib.tg_gated_workspace_size(px, pg, pu, M, N, K, options), x)
        if ws is not None:
            ws_ptr, ws_bytes = ws.data_ptr(), ws.numel()
    elif workspace != "auto":
        raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
    if not save:
        _check(_lib.tg_gated(px, pg, pu, out2.data_ptr(), 0, 0, M, N, K, options, _raw_stream(index), ws_ptr, ws_bytes),
               "tg_gated")
        return out
    # Rows of the stored projections start on 16-byte boundaries whatever N is: they leave by TMA and come
    # back in whole vectors (forward of 2000 x 4095 x 2047 with both stored: 84 us dense, 73 us so).
    ld = (N + 7) & -8
    gate, up = x.new_empty(M, ld), x.new_empty(M, ld)
    if ld != N:
        options = _options(code, act_code, ldx, ldg, ldu, ldh, ld, ld)
    _check(_lib.tg_gated(px, pg, pu, out2.data_ptr(), gate.data_ptr(), up.data_ptr(), M, N, K, options,
                         _raw_stream(index), ws_ptr, ws_bytes), "tg_gated")
    if x2 is not x:
        gate, up = gate.view(*x.shape[:-1], ld), up.view(*x.shape[:-1], ld)
    return (out, gate, up) if ld == N else (out, gate[..., :N], up[..., :N])


def gated_backward(grad, x, w_gate, w_up, gate, up, act="silu", needs=(True, True, True), stream=None,
                   workspace="auto"):
    """Gradients of ``gated`` for grad = dH (..., N), with the projections that ``gated(..., save=True)``
    returned: (dx, dw_gate, dw_up), None where ``needs`` is false.

    ``workspace``: "auto" lets torch allocate the bytes for dG and dU; a uint8 CUDA tensor is used as
    given (calls whose work may overlap need one each).
    """
    index = _device(x, "x")
    if stream is not None or index != _current_device():
        with _Elsewhere(index, stream, (grad, x, w_gate, w_up, gate, up, workspace)):
            return gated_backward(grad, x, w_gate, w_up, gate, up, act, needs, None, workspace)
    x2, grad2, gate2, up2 = _flat(x, "x"), _flat(grad, "grad"), _flat(gate, "gate"), _flat(up, "up")
    M, K = x2.shape
    dtype = x.dtype
    code, act_code = _codes(dtype, act)
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be (N, K), got {tuple(w_gate.shape)}")
    N = w_gate.shape[0]
    options = _options(code, act_code, _row_stride(x2, M, K, "x"), _matrix(w_gate, "w_gate", N, K, dtype, index),
                       _matrix(w_up, "w_up", N, K, dtype, index), _matrix(grad2, "grad", M, N, dtype, index),
                       _matrix(gate2, "gate", M, N, dtype, index), _matrix(up2, "up", M, N, dtype, index))
    need_x, need_g, need_u = needs
    dx = x.new_empty(M, K) if need_x else None
    dg = x.new_empty(N, K) if need_g else None
    du = x.new_empty(N, K) if need_u else None
    pdx, pdg, pdu = (dx.data_ptr() if need_x else 0), (dg.data_ptr() if need_g else 0), (du.data_ptr() if need_u else 0)
    px, pg, pu = x2.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    ws = _scratch(workspace, _lib.tg_gated_backward_workspace_size(px, pg, pu, pdx, pdg, pdu, M, N, K, options), x)
    ws_ptr, ws_bytes = (ws.data_ptr(), ws.numel()) if ws is not None else (0, 0)
    _check(_lib.tg_gated_backward(grad2.data_ptr(), px, pg, pu, gate2.data_ptr(), up2.data_ptr(), pdx, pdg, pdu, M, N, K,
                                  options, _raw_stream(index), ws_ptr, ws_bytes), "tg_gated_backward")
    return dx if x2 is x or dx is None else dx.view(x.shape), dg, du


def quantize_i8(x, out=None, scales=None, stream=None):
    """Rows of x (..., K), float16 or bfloat16, as 8-bit integers with one scale each: (codes, scales) with
    codes (..., K) int8 and scales (...) float32, scale = max |x| / 127, codes = x / scale rounded to
    nearest even.  Rows of codes that the call allocates start on 16-byte boundaries whatever K is, as
    ``gemm_i8`` and ``gated_i8`` want them.  Serves activations (a row is a token) and weights (a row is
    a channel).  Rows of zeros: scale 0.  Rows with an infinity or a NaN: scale NaN, codes 0."""
    index = _device(x, "x")
    if stream is not None or index != _current_device():
        with _Elsewhere(index, stream, (x, out, scales)):
            return quantize_i8(x, out, scales)
    x2 = _flat(x, "x")
    M, K = x2.shape
    code, ldx = _codes(x.dtype)[0], _row_stride(x2, M, K, "x")
    if out is None:
        ldq = (K + 15) & -16
        out2 = out = x.new_empty(M, ldq, dtype=_I8)
        if x2 is not x:
            out = out.view(*x.shape[:-1], ldq)
        if ldq != K:
            out = out[..., :K]
    else:
        out2, ldq = _result(out, x.shape[:-1], M, K, _I8, index)
    if scales is None:
        scales = x.new_empty(M, dtype=_F32)
        if x2 is not x:
            scales = scales.view(x.shape[:-1])
    else:
        _vector(scales, "scales", M, _F32, index)
    _check(_lib.tg_quantize_rows_i8(x2.data_ptr(), out2.data_ptr(), scales.data_ptr(), M, K, ldx, ldq, code,
                                    _raw_stream(index)), "tg_quantize_rows_i8")
    return out, scales


def gemm_i8(a, a_scale, w, w_scale, bias=None, relu=False, dtype=None, out=None, stream=None):
    """(a @ w^T) * a_scale * w_scale + bias, with an optional ReLU, for int8 CUDA tensors a (..., K) and
    w (N, K) with a float32 scale for each of their rows; bias (N,) of the result's type.

    Returns (..., N) of ``dtype`` (float16 unless given, or ``out``'s).  The integer sums are exact.
    Rows of a and w must start on 16-byte boundaries (as those of ``quantize_i8`` do)."""
    index = _device(a, "a")
    if stream is not None or index != _current_device():
        with _Elsewhere(index, stream, (a, a_scale, w, w_scale, bias, out)):
            return gemm_i8(a, a_scale, w, w_scale, bias, relu, dtype, out)
    a2 = _flat(a, "a")
    M, K = a2.shape
    if w.dim() != 2:
        raise ValueError(f"w must be (N, K), got {tuple(w.shape)}")
    N = w.shape[0]
    lda, ldw = _matrix(a2, "a", M, K, _I8, index), _matrix(w, "w", N, K, _I8, index)
    sa, sw = _vector(a_scale, "a_scale", M, _F32, index), _vector(w_scale, "w_scale", N, _F32, index)
    if dtype is None:
        dtype = torch.float16 if out is None else out.dtype
    code = _codes(dtype)[0]
    pb = _vector(bias, "bias", N, dtype, index) if bias is not None else 0
    if out is None:
        ldc, out2 = 0, a.new_empty(M, N, dtype=dtype)
        out = out2 if a2 is a else out2.view(*a.shape[:-1], N)
    else:
        out2, ldc = _result(out, a.shape[:-1], M, N, dtype, index)
    _check(_lib.tg_gemm_i8(a2.data_ptr(), sa, w.data_ptr(), sw, pb, out2.data_ptr(), M, N, K, lda, ldw, ldc,
                           1 if relu else 0, code, _raw_stream(index)), "tg_gemm_i8")
    return out


def gated_i8(a, a_scale, w_gate, gate_scale, w_up, up_scale, act="silu", dtype=None, out=None, stream=None):
    """``gated`` on 8-bit operands: a (..., K) int8 with a scale a row, w_gate and w_up (N, K) int8 with a
    scale a row.  Returns (..., N) of ``dtype`` (float16 unless given, or ``out``'s).  Operands as for
    ``gemm_i8``."""
    index = _device(a, "a")
    if stream is not None or index != _current_device():
        with _Elsewhere(index, stream, (a, a_scale, w_gate, gate_scale, w_up, up_scale, out)):
            return gated_i8(a, a_scale, w_gate, gate_scale, w_up, up_scale, act, dtype, out)
    a2 = _flat(a, "a")
    M, K = a2.shape
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be (N, K), got {tuple(w_gate.shape)}")
    N = w_gate.shape[0]
    if dtype is None:
        dtype = torch.float16 if out is None else out.dtype
    code, act_code = _codes(dtype, act)
    lda = _matrix(a2, "a", M, K, _I8, index)
    ldg, ldu = _matrix(w_gate, "w_gate", N, K, _I8, index), _matrix(w_up, "w_up", N, K, _I8, index)
    sa = _vector(a_scale, "a_scale", M, _F32, index)
    sg, su = _vector(gate_scale, "gate_scale", N, _F32, index), _vector(up_scale, "up_scale", N, _F32, index)
    if out is None:
        ldh, out2 = 0, a.new_empty(M, N, dtype=dtype)
        out = out2 if a2 is a else out2.view(*a.shape[:-1], N)
    else:
        out2, ldh = _result(out, a.shape[:-1], M, N, dtype, index)
    _check(_lib.tg_gated_i8(a2.data_ptr(), sa, w_gate.data_ptr(), sg, w_up.data_ptr(), su, out2.data_ptr(), M, N, K,
                            _options(code, act_code, lda, ldg, ldu, ldh), _raw_stream(index)), "tg_gated_i8")
    return out


# ---------------------------------------------------------------------------
# Autograd
# ---------------------------------------------------------------------------

def _rows(t):
    """t, or a dense copy where its rows are not evenly spaced with adjacent columns (an expanded gradient)."""
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

    Runs on the current stream.  Without a gradient to take, neither projection is stored."""
    if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad):
        return GatedBlock.apply(x, w_gate, w_up, act)
    return gated(_rows(x), _rows(w_gate), _rows(w_up), act=act)
