"""Ends that break their rule, where they decrease or leave the rows: each counts as the greatest before it, or as the number of
rows, so that every row has one group at most.  All values are checked, and the surroundings of all results."""
import numpy as np
import pytest

import grp_ref as ref
from test_gpu_grp import _ok, _randn

pytestmark = pytest.mark.gpu


def _sizes(ends, M):
    raised = np.maximum.accumulate(np.clip(np.asarray(ends, np.int64), 0, M))
    return np.diff(np.r_[0, raised]).tolist()


def _guarded(shape, dtype):
    """A result with 64 values of 5 on both sides, and a check of those."""
    import torch
    n = int(np.prod(shape))
    flat = torch.full((n + 128,), 5.0, dtype=dtype, device="cuda")
    return flat[64:64 + n].view(shape), lambda: bool((flat[:64] == 5).all()) and bool((flat[64 + n:] == 5).all())


def _check(M, ends, N, K, dt):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    G, sizes = len(ends), _sizes(ends, M)
    x, w = _randn(1, (M, K), dt), _randn(2, (G, N, K), dt, K ** -0.5)
    dy = _randn(3, (M, N), dt)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    y, tol = ref.grouped(ref.f64(x), ref.f64(w), sizes, dt)
    out, intact = _guarded((M, N), x.dtype)
    tg.grouped(x, w, e, out=out)
    got = tg.grouped(x, w, e)
    dx, dx_intact = _guarded((M, K), x.dtype)
    dw, dw_intact = _guarded((G, N, K), x.dtype)
    opts = tg.grouped_options(type=tg.TYPE_BF16 if dt == "bf16" else tg.TYPE_F16)
    need = tg.grouped_backward_workspace_size(*(t.data_ptr() for t in (dy, x, w, dx, dw)), G, M, N, K, opts)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    st = tg.grouped_backward_raw(dy.data_ptr(), x.data_ptr(), w.data_ptr(), e.data_ptr(), dx.data_ptr(), dw.data_ptr(), G, M, N, K, opts,
                                 torch.cuda.current_stream().cuda_stream, ws.data_ptr(), need)
    assert st == tg.Status.OK
    _ok()
    assert intact() and dx_intact() and dw_intact()
    used = sum(sizes)
    ref.check(ref.f64(got), y, tol, f"y {ends}")
    assert torch.equal(out[:used], got[:used]) and bool((out[used:] == 5).all()) and bool((dx[used:] == 5).all())
    (want_x, want_w), (tx, tw) = ref.grouped_backward(ref.f64(dy), ref.f64(x), ref.f64(w), sizes, dt)
    ref.check(ref.f64(dx)[:used], want_x[:used], tx[:used], f"dx {ends}")
    ref.check(ref.f64(dw), want_w, tw, f"dw {ends}")


ENDS = [[5, 3, 40], [-7, 10, 64], [70, 64, 64], [2 ** 31 - 1, -(2 ** 31), 9], [0, 0, 0], [9, 64, 9], [64, 0, 64, 0, 64, 0], [-1, -5], [30, 20, 10, 40, 35, 50]]


@pytest.mark.parametrize("ends", ENDS)
@pytest.mark.parametrize("N", [40, 2304])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_few_rows(ends, N, dt):
    _check(64, ends, N, 16, dt)


@pytest.mark.parametrize("ends", [[1500, 900, 2900, 100, 2700], [5000, 0, 2600], [-3, 1, 1, 0, 3001, -9]])
@pytest.mark.parametrize("N,K", [(2304, 72), (72, 2304), (61, 45)])
def test_many_rows(ends, N, K):
    _check(3000, ends, N, K, "f16")


@pytest.mark.parametrize("G", [33, 64, 1024])
def test_many_groups(G):
    """Random ends over groups of several warps' lanes."""
    rng = np.random.default_rng(G)
    _check(700, rng.integers(-50, 750, G).tolist(), 40, 24, "f16")
    _check(700, np.where(np.arange(G) % 2 == 0, 700, 0).tolist(), 40, 24, "f16")
    _check(700, (700 - np.arange(G)).tolist(), 40, 24, "f16")


def test_sums_over_nothing():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    e = torch.tensor([20, 3, 9], dtype=torch.int32, device="cuda")
    x, w = torch.zeros(24, 0, dtype=torch.float16, device="cuda"), torch.zeros(3, 40, 0, dtype=torch.float16, device="cuda")
    out = torch.ones(24, 40, dtype=torch.float16, device="cuda")
    tg.grouped(x, w, e, out=out)
    _ok()
    assert bool((out[:20] == 0).all()) and bool((out[20:] == 1).all())
