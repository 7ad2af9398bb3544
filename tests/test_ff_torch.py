"""The torch side of the feed-forward calls: what it refuses before any device is needed."""
import os
import subprocess
import sys

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


# ---------------------------------------------------------------------------
# The compiled module and what it was built for
# ---------------------------------------------------------------------------

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_module_for_another_torch_is_stale(monkeypatch):
    from tiled_dense_gemm_fp16_b200 import build, feedforward
    if not build.calls_stale():
        assert feedforward._calls.key == build._calls_key() and feedforward._calls.target == build.calls_target()
    here, command = build.calls_target(), build._calls_command
    assert torch.__version__ in here
    for other in (here.replace(torch.__version__, "0.0"), here.replace("Python c", "Python d"), here + "x"):
        with monkeypatch.context() as m:
            m.setattr(build, "calls_target", lambda: other)
            assert build.calls_stale()
    with monkeypatch.context() as m:
        m.setattr(build, "_calls_command", lambda out: [*command(out), "-O3"])
        assert build.calls_stale()


def test_a_built_module_needs_no_compiler(monkeypatch):
    from tiled_dense_gemm_fp16_b200 import build
    stale = build.calls_stale()

    def missing():
        raise RuntimeError("nvcc not found")
    monkeypatch.setattr(build, "_nvcc", missing)
    assert stale or not build.calls_stale()
    monkeypatch.setattr(build, "calls_target", lambda: "torch 0.0")
    assert build.calls_stale()


def test_a_module_for_another_torch_is_not_loaded():
    code = """
import tiled_dense_gemm_fp16_b200 as tg
from tiled_dense_gemm_fp16_b200 import build
build.calls_target = lambda: "torch 0.0"
try:
    tg.gated
except ImportError as e:
    assert "torch 0.0" in str(e) and "build" in str(e)
    print("refused")
"""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "refused", p.stderr[-2000:]
