"""The feed-forward operators at the edges of their ranges and in uses that cross: overflowed projections, far gates,
results between the rows of other matrices, row blocks of every height, captured training steps.  Tolerances: ff_ref.py."""
import numpy as np
import pytest

import ff_ref as ref

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _randn(seed, shape, dt, scale=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(ref.torch_type(dt))


def _ok():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    torch.cuda.synchronize()
    st, word = tg.device_status()
    assert st == tg.Status.OK, hex(word)


# ---------------------------------------------------------------------------
# Gradients at projections that overflowed when they were stored
# ---------------------------------------------------------------------------

def _row_gradients(dh, g, u, act, dt):
    """dG and dU of one row: with X = 1 they are the columns of dWg and dWu."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    t = ref.torch_type(dt)
    dh, g, u = (torch.tensor([v], device="cuda").to(t) for v in (dh, g, u))
    n = g.shape[1]
    x, w = torch.ones((1, 1), dtype=t, device="cuda"), torch.ones((n, 1), dtype=t, device="cuda")
    dx, dwg, dwu = tg.gated_backward(dh, x, w, w, g, u, act=act)
    _ok()
    return dx.item(), dwg[:, 0].tolist(), dwu[:, 0].tolist()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_no_gradient_at_overflowed_projections(act, dt):
    """A token without a gradient (padded, masked) has none through stored infinities either; a NaN stays one."""
    for zero in (0.0, -0.0):
        g, u = [INF, 1.0, -INF, INF, 2.0, -INF], [2.0, INF, 3.0, -INF, -INF, INF]
        dx, dg, du = _row_gradients([zero] * 6, g, u, act, dt)
        assert dx == 0 and not any(dg) and not any(du), (dx, dg, du)
        _, dg, du = _row_gradients([zero] * 2, [2.0, NAN], [NAN, 1.0], act, dt)
        assert np.isnan(dg[0]) and du[0] == 0
        assert act == "relu" or (np.isnan(dg[1]) and np.isnan(du[1]))  # relu: a gate that is not > 0 is closed


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_closed_gates_hide_no_gradient(act, dt):
    """A closed gate gives dG = 0 whatever U is; dH that is not finite shows in dG and in dU."""
    closed = [-INF] * 6
    dh, u = [NAN, INF, -INF, 0.5, 0.5, 0.5], [1.0, 1.0, 0.0, INF, NAN, 7.0]
    _, dg, du = _row_gradients(dh, closed, u, act, dt)
    assert np.isnan(dg[:3]).all() and np.isnan(du[:3]).all(), (dg, du)
    assert not any(dg[3:]) and not any(du[3:]), (dg, du)
