"""The torch side of the feed-forward calls: what it refuses before any device is needed."""
import pytest

torch = pytest.importorskip("torch")

import tiled_dense_gemm_fp16_b200 as tg  # noqa: E402


def _operands():
    return torch.ones(4, 8, dtype=torch.float16), torch.ones(16, 8, dtype=torch.float16), torch.ones(16, 8, dtype=torch.float16)


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("requires_grad", [False, True])
def test_forward_mode_is_refused(which, requires_grad):
    """A tangent of any operand would be lost without a word."""
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        args = [t.requires_grad_(requires_grad) for t in _operands()]
        args[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            tg.gated_block(*args)
    with pytest.raises(ValueError, match="CUDA"):  # without a tangent the call is as ever
        tg.gated_block(*_operands())


def test_negated_views_are_refused():
    """Views whose values are the negatives of their memory, which the kernels would read with the wrong sign."""
    from tiled_dense_gemm_fp16_b200 import feedforward
    calls = feedforward._calls
    x, w = torch.ones(4, 1, dtype=torch.complex32).conj().imag, torch.ones(16, 1, dtype=torch.float16)
    assert x.is_neg() and not w.is_neg()
    q, s = torch._neg_view(torch.ones(4, 16, dtype=torch.int8)), torch.ones(4)
    for call in (lambda: tg.gated(x, w, w), lambda: tg.gated(w, x, w), lambda: tg.gated_block(x, w, w),
                 lambda: tg.gated_backward(x, w, w, w, w, w), lambda: tg.quantize_i8(x),
                 lambda: calls.gemm_i8(q, s, q, s, None, False, None, None),
                 lambda: calls.gated_i8(q, s, q, s, q, s, "silu", None, None)):
        with pytest.raises(ValueError, match="negated view|CUDA"):
            call()
    with pytest.raises(ValueError, match="negated view"):
        tg.gated(x, w, w)
    with pytest.raises(ValueError, match="negated view"):
        calls.gemm_i8(q, s, q, s, None, False, None, None)
