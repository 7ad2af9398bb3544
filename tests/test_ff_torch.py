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
