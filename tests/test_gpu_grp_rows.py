"""Gradients of the grouped product where the C call puts them: rows and matrices any distance apart, on any 2-byte boundary,
beside values that stay as they are; rows without a group; calls without rows."""
import numpy as np
import pytest

import grp_ref as ref
from test_gpu_grp import _check_backward, _check_forward, _ends, _ok, _randn

pytestmark = pytest.mark.gpu
REST = 9.0  # what lies between results


def _result(shape, strides, off, dtype):
    """A result `off` elements from a 16-byte boundary, and a check that nothing around or between its values has changed."""
    import torch
    span = sum((n - 1) * s for n, s in zip(shape, strides)) + 1 if min(shape) else 0
    flat = torch.full((off + span + 128,), REST, dtype=dtype, device="cuda")
    view = flat[64 + off:].as_strided(shape, strides)

    def intact():
        other = torch.ones_like(flat, dtype=torch.bool)
        other[64 + off:].as_strided(shape, strides).fill_(False)
        return bool((flat[other] == REST).all())
    return view, intact


def _backward(M, sizes, N, K, dt, lddw=0, stride_dw=0, lddx=0, off=0, rest=0, want=("dx", "dw")):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    G = len(sizes)
    x, w, dy = _randn(1, (M, K), dt), _randn(2, (G, N, K), dt, K ** -0.5), _randn(3, (M, N), dt)
    ends = _ends(sizes)
    dx, dx_intact = _result((M, K), (lddx or K, 1), off, x.dtype)
    dw, dw_intact = _result((G, N, K), (stride_dw or N * (lddw or K), lddw or K, 1), off, x.dtype)
    opts = tg.grouped_options(type=tg.TYPE_BF16 if dt == "bf16" else tg.TYPE_F16, rest=rest, lddw=lddw, stride_dw=stride_dw, lddx=lddx)
    at = {"dx": dx.data_ptr() if "dx" in want else 0, "dw": dw.data_ptr() if "dw" in want else 0}
    inputs = [t.data_ptr() for t in (dy, x, w)]
    need = tg.grouped_backward_workspace_size(*inputs, at["dx"], at["dw"], G, M, N, K, opts)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    st = tg.grouped_backward_raw(*inputs, ends.data_ptr(), at["dx"], at["dw"], G, M, N, K, opts, torch.cuda.current_stream().cuda_stream,
                                 ws.data_ptr(), need)
    assert st == tg.Status.OK
    _ok()
    assert dx_intact() and dw_intact(), "values between the results"
    (want_x, want_w), (tx, tw) = ref.grouped_backward(ref.f64(dy), ref.f64(x), ref.f64(w), sizes, dt)
    used = sum(sizes)
    what = f"{M} {sizes} {N} {K} {dt} {lddw} {stride_dw} {off}"
    if "dx" in want:
        ref.check(ref.f64(dx)[:used], want_x[:used], tx[:used], "dx " + what)
        assert bool((dx[used:] == (0 if rest else REST)).all())
    else:
        assert bool((dx == REST).all())
    if "dw" in want:
        ref.check(ref.f64(dw), want_w, tw, "dw " + what)
    else:
        assert bool((dw == REST).all())


# K that ends inside 16 bytes in rows on 16 bytes: boxes by TMA and value by value in turn; rows off 16 bytes: words.
@pytest.mark.parametrize("K,lddw", [(37, 48), (300, 312), (300, 304), (40, 40), (296, 320), (37, 37), (37, 41), (300, 305)])
@pytest.mark.parametrize("gap", [0, 8, 24, 1001])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_rows_and_matrices_apart(K, lddw, gap, off):
    N = 70
    for dt, rest in (("f16", 0), ("bf16", 1)):
        _backward(150, [33, 0, 64, 40], N, K, dt, lddw=lddw, stride_dw=N * lddw + gap, lddx=K + 3 if off else lddw, off=off, rest=rest)


@pytest.mark.parametrize("N,K,lddw", [(520, 300, 304), (300, 520, 528), (257, 263, 264), (512, 512, 520)])
def test_several_tiles_of_each_matrix(N, K, lddw):
    """Empty groups among them, whose zeros take the same ways out."""
    _backward(700, [0, 260, 1, 0, 400, 30, 0], N, K, "f16", lddw=lddw, stride_dw=N * lddw + 16)
    _backward(700, [0, 260, 1, 0, 400, 30, 0], N, K, "bf16", lddw=lddw + 1, stride_dw=N * (lddw + 1) + 7)


@pytest.mark.parametrize("want", [("dx",), ("dw",)])
def test_one_gradient(want):
    for N, K in ((72, 40), (61, 45)):
        _backward(150, [33, 0, 64, 40], N, K, "f16", want=want, lddx=K + 3, lddw=K + 8)


@pytest.mark.parametrize("sizes", [[0, 0, 0], [0, 0, 5]])
@pytest.mark.parametrize("gap", [0, 1, 24])
def test_no_rows(sizes, gap):
    """Weights of groups without rows are +0, evenly spaced or not; without any rows the call writes zeros alone."""
    N, K, lddw = 30, 37, 41
    _backward(0 if sum(sizes) == 0 else 8, sizes, N, K, "f16", lddw=lddw, stride_dw=N * lddw + gap)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_strips_of_several_tiles(dt):
    """More than eight tiles of rows of dW, the last strip narrower, by several tiles of columns; groups of one tile and of none."""
    _check_backward(400, [130, 0, 201, 64], 2309, 600, dt)
    _check_backward(300, [0, 300], 4400, 776, dt)
    _check_forward(900, [130, 0, 701, 64], 2309, 600, dt)
