"""Grouped products, their gradients and the adapters on the GPU, against their definitions in 64 bits (grp_ref.py)."""
import numpy as np
import pytest

import grp_ref as ref

pytestmark = pytest.mark.gpu


def _randn(seed, shape, dt, scale=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(ref.torch_type(dt))


def _ends(sizes):
    import torch
    return torch.tensor(list(sizes), dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _ok():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    torch.cuda.synchronize()
    st, word = tg.device_status()
    assert st == tg.Status.OK, hex(word)


def _operands(M, sizes, N, K, dt, seed=1):
    return _randn(seed, (M, K), dt), _randn(seed + 1, (len(sizes), N, K), dt, K ** -0.5), _ends(sizes)


def _check_forward(M, sizes, N, K, dt):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, ends = _operands(M, sizes, N, K, dt)
    y, tol = ref.grouped(ref.f64(x), ref.f64(w), sizes, dt)
    got = tg.grouped(x, w, ends)
    _ok()
    ref.check(ref.f64(got), y, tol, f"grouped {M} {sizes} {N} {K} {dt}")
    # A given result: the rows without a group stay as they were.
    out = torch.full((M, N), 7.0, dtype=x.dtype, device="cuda")
    assert tg.grouped(x, w, ends, out=out) is out
    _ok()
    used = sum(sizes)
    assert torch.equal(out[:used], got[:used]) and bool((out[used:] == 7).all())


def _check_backward(M, sizes, N, K, dt):
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, ends = _operands(M, sizes, N, K, dt)
    dy = _randn(5, (M, N), dt)
    outs, tols = ref.grouped_backward(ref.f64(dy), ref.f64(x), ref.f64(w), sizes, dt)
    got = tg.grouped_backward(dy, x, w, ends)
    _ok()
    for name, g, o, tol in zip(("dx", "dw"), got, outs, tols):
        ref.check(ref.f64(g), o, tol, f"{name} {M} {sizes} {N} {K} {dt}")


# Few rows a group, or few tiles: the narrow kernel.
NARROW = [
    (1, [1], 64, 64), (1, [0, 1, 0], 8, 8), (8, [3, 0, 5], 128, 128), (5, [1, 1, 1, 1, 1], 200, 72), (17, [16, 0, 1], 136, 264),
    (40, [33, 2], 256, 512), (130, [129, 0, 1], 264, 1000), (300, [100, 150, 50], 512, 512), (64, [0, 0], 96, 80), (7, [7], 1, 8),
    (77, [3, 70, 4], 40, 1048), (33, [1] * 33, 128, 320),
]
# Whole tiles on CTA pairs.
PAIR = [
    (5000, [2000, 1500, 1499], 2048, 64), (4500, [0, 4100, 257, 0], 2304, 136), (4096, [256, 3840], 4096, 512),
    (2100, [33, 1025, 511, 513], 4104, 200),
]


@pytest.mark.parametrize("M,sizes,N,K", NARROW)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_grouped_narrow(M, sizes, N, K, dt):
    _check_forward(M, sizes, N, K, dt)


@pytest.mark.parametrize("M,sizes,N,K", PAIR)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_grouped_pair(M, sizes, N, K, dt):
    _check_forward(M, sizes, N, K, dt)


@pytest.mark.parametrize("M,sizes,N,K", NARROW + [(5000, [2000, 1500, 1499], 64, 2048), (2100, [33, 1025, 511, 513], 200, 4104)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_grouped_backward(M, sizes, N, K, dt):
    _check_backward(M, sizes, N, K, dt)


@pytest.mark.parametrize("tail", range(1, 65))
def test_weight_gradient_tails(tail):
    """Groups that end at every place of a k-block, next to rows of another group that are not finite."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    sizes, N, K = [tail, 70, 64 + tail, 3], 264, 312
    M = sum(sizes) + 5
    x, w, ends = _operands(M, sizes, N, K, "f16")
    dy = _randn(5, (M, N), "f16")
    (dx, dw), (tx, tw) = ref.grouped_backward(ref.f64(dy), ref.f64(x), ref.f64(w), sizes, "f16")
    for lo, hi in (ref.bounds(sizes)[1], (M - 5, M)):
        x[lo:hi], dy[lo:hi] = float("inf"), float("nan")
    gx, gw = tg.grouped_backward(dy, x, w, ends)
    _ok()
    for g in (0, 2, 3):
        ref.check(ref.f64(gw[g]), dw[g], tw[g], f"dw of group {g}, tail {tail}")
        lo, hi = ref.bounds(sizes)[g]
        ref.check(ref.f64(gx[lo:hi]), dx[lo:hi], tx[lo:hi], f"dx of group {g}, tail {tail}")
    assert bool((gx[M - 5:] == 0).all()) and bool(torch.isnan(gw[1]).any())


# (rows, N, K, rank, adapters)
LORA = [(1, 64, 64, 8, 1), (3, 128, 128, 16, 4), (16, 200, 72, 24, 5), (33, 264, 1000, 32, 40), (64, 512, 512, 64, 64), (100, 136, 264, 72, 3),
        (250, 512, 320, 16, 9), (2600, 4104, 64, 16, 4), (4100, 2304, 136, 136, 7), (2111, 4096, 264, 64, 30)]


def _index(kind, M, R, seed):
    rng = np.random.default_rng(seed)
    if kind == "none":
        return np.full(M, -1)
    if kind == "one":
        return np.full(M, R - 1)
    if kind == "random":  # some without an adapter, by values of either sign
        return rng.choice(np.r_[np.arange(R), -1, R, -7, 1 << 30], M)
    cuts = np.sort(rng.integers(0, M + 1, 6))  # runs
    owner = rng.permutation(np.r_[np.arange(R), -1])
    return owner[np.searchsorted(cuts, np.arange(M), side="right") % len(owner)]


@pytest.mark.parametrize("M,N,K,rank,R", LORA)
@pytest.mark.parametrize("kind", ["random", "runs", "one", "none"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_lora(M, N, K, rank, R, kind, dt):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w = _randn(1, (M, K), dt), _randn(2, (N, K), dt, K ** -0.5)
    a, b = _randn(3, (R, rank, K), dt, K ** -0.5), _randn(4, (R, N, rank), dt, rank ** -0.5)
    index = _index(kind, M, R, M + R)
    with_scale = kind != "one"
    scale = torch.rand(R, generator=torch.Generator().manual_seed(3)).cuda() + 0.5 if with_scale else None
    bias = _randn(6, (N,), dt) if kind != "runs" else None
    got = tg.lora(x, w, a, b, torch.from_numpy(index.astype(np.int32)).cuda(), scale=scale, bias=bias)
    _ok()
    y, tol = ref.lora(ref.f64(x), ref.f64(w), ref.f64(a), ref.f64(b), index, None if scale is None else ref.f64(scale),
                      None if bias is None else ref.f64(bias), dt)
    ref.check(ref.f64(got), y, tol, f"lora {M} {N} {K} {rank} {R} {kind} {dt}")
