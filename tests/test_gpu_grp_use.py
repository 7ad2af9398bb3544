"""Grouped products and adapters as they are used: rows of any stride and boundary, values that are not finite, other streams,
graphs, autograd, several together, offsets past 32 bits, refusals.  Tolerances: grp_ref.py."""
import numpy as np
import pytest

import ff_ref
import grp_ref as ref
from test_gpu_grp import _ends, _index, _ok, _operands, _randn

pytestmark = pytest.mark.gpu


def _spread(t, ld, off):
    """t's values in rows of ld elements, `off` elements from a 16-byte boundary, amid NaN."""
    import torch
    flat = torch.full((off + t.shape[0] * ld + 8,), float("nan"), dtype=t.dtype, device="cuda")
    view = flat[off:off + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
    view.copy_(t)
    return view


def _stack(t, ld, stride, off=0):
    """A stack of matrices with rows of ld elements, `stride` from one to the next, amid NaN."""
    import torch
    G, N, K = t.shape
    flat = torch.full((off + G * stride + N * ld + 8,), float("nan"), dtype=t.dtype, device="cuda")
    view = flat[off:].as_strided((G, N, K), (stride, ld, 1))
    view.copy_(t)
    return view


def _lora_operands(M, N, K, rank, R, dt, kind, seed=1):
    import torch
    x, w = _randn(seed, (M, K), dt), _randn(seed + 1, (N, K), dt, K ** -0.5)
    a, b = _randn(seed + 2, (R, rank, K), dt, K ** -0.5), _randn(seed + 3, (R, N, rank), dt, rank ** -0.5)
    index = _index(kind, M, R, seed)
    return x, w, a, b, index, torch.from_numpy(index.astype(np.int32)).cuda()


# ---------------------------------------------------------------------------
# Strides and boundaries
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,sizes,N,K", [(70, [30, 0, 40], 61, 45), (3000, [1400, 100, 1500], 2309, 61), (20, [5, 15], 1, 1), (9, [9], 33, 7)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_odd_sizes(M, sizes, N, K, dt):
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, ends = _operands(M, sizes, N, K, dt)
    dy = _randn(7, (M, N), dt)
    y, tol = ref.grouped(ref.f64(x), ref.f64(w), sizes, dt)
    got = tg.grouped(x, w, ends)
    grads = tg.grouped_backward(dy, x, w, ends)
    _ok()
    ref.check(ref.f64(got), y, tol, "y")
    for name, g, o, t in zip(("dx", "dw"), grads, *ref.grouped_backward(ref.f64(dy), ref.f64(x), ref.f64(w), sizes, dt)):
        ref.check(ref.f64(g), o, t, name)


@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("M,sizes,N,K", [(70, [30, 0, 40], 72, 40), (2700, [1400, 100, 1200], 2312, 64)])
def test_strides(M, sizes, N, K, off):
    """Rows in wider buffers, halves of fused weights, results on any 2-byte boundary with their surroundings untouched."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x0, w0, ends = _operands(M, sizes, N, K, "f16")
    dy0 = _randn(7, (M, N), "f16")
    y, tol = ref.grouped(ref.f64(x0), ref.f64(w0), sizes, "f16")
    grads, tols = ref.grouped_backward(ref.f64(dy0), ref.f64(x0), ref.f64(w0), sizes, "f16")
    x, dy = _spread(x0, K + 13, off), _spread(dy0, N + 8, off)
    for w in (_stack(w0, K + 8, 2 * N * (K + 8)), _stack(w0, K, N * K, off), _stack(w0, len(sizes) * K, K)):  # halves; dense; interleaved
        if off and w.stride(1) == len(sizes) * K:
            w = w0
        flat = torch.full((M * (N + 5) + 64,), 9.0, dtype=torch.float16, device="cuda")
        out = flat[off + 16:off + 16 + M * (N + 5)].view(M, N + 5)[:, :N]
        tg.grouped(x, w, ends, out=out)
        got = tg.grouped_backward(dy, x, w, ends)
        _ok()
        ref.check(ref.f64(out), y, tol, f"y {off}")
        for name, g, o, t in zip(("dx", "dw"), got, grads, tols):
            ref.check(ref.f64(g), o, t, f"{name} {off}")
        rows = flat[off + 16:off + 16 + M * (N + 5)].view(M, N + 5)
        assert bool((rows[:, N:] == 9).all()) and bool((flat[:off + 16] == 9).all()) and bool((flat[off + 16 + M * (N + 5):] == 9).all())


@pytest.mark.parametrize("stride", [8, 9, 40])
@pytest.mark.parametrize("K", [5, 8])
def test_weights_of_one_row(K, stride):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    sizes = [30, 0, 34, 6]
    x, w0, ends = _operands(70, sizes, 1, K, "f16")
    dy = _randn(7, (70, 1), "f16")
    w = _stack(w0, K, stride)
    y, tol = ref.grouped(ref.f64(x), ref.f64(w0), sizes, "f16")
    got = tg.grouped(x, w, ends)
    grads = tg.grouped_backward(dy, x, w, ends)
    leaf = w.detach().requires_grad_()
    auto = tg.grouped_linear(x, leaf, ends)
    auto.backward(dy)
    _ok()
    ref.check(ref.f64(got), y, tol, "y")
    for name, g, o, t in zip(("dx", "dw"), grads, *ref.grouped_backward(ref.f64(dy), ref.f64(x), ref.f64(w0), sizes, "f16")):
        ref.check(ref.f64(g), o, t, name)
    assert torch.equal(auto, got) and torch.equal(leaf.grad, grads[1])


@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("M,N,K", [(60, 72, 40), (60, 73, 41), (2700, 2311, 72)])
def test_lora_strides(M, N, K, off):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    rank, R = 24, 5
    x0, w0, a0, b0, index, ix = _lora_operands(M, N, K, rank, R, "bf16", "runs")
    y, tol = ref.lora(ref.f64(x0), ref.f64(w0), ref.f64(a0), ref.f64(b0), index, None, None, "bf16")
    lda = (K + 7) // 8 * 8 + 8
    a, b = _stack(a0, lda, rank * lda + 16), _stack(b0, rank + 16, N * (rank + 16) + 8)
    x, w = _spread(x0, K + 13, off), _spread(w0, K + 3, off)
    flat = torch.full((M * (N + 5) + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = flat[off + 16:off + 16 + M * (N + 5)].view(M, N + 5)[:, :N]
    tg.lora(x, w, a, b, ix, out=out)
    _ok()
    ref.check(ref.f64(out), y, tol, f"lora {off}")
    rows = flat[off + 16:off + 16 + M * (N + 5)].view(M, N + 5)
    assert bool((rows[:, N:] == 9).all()) and bool((flat[:off + 16] == 9).all()) and bool((flat[off + 16 + M * (N + 5):] == 9).all())


def test_leading_dimensions_and_empty_calls():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, ends = _operands(24, [10, 0, 14], 40, 16, "bf16")
    assert torch.equal(tg.grouped(x.view(2, 3, 4, 16), w, ends), tg.grouped(x, w, ends).view(2, 3, 4, 40))
    dx, dw = tg.grouped_backward(tg.grouped(x, w, ends).view(4, 6, 40), x.view(4, 6, 16), w, ends, needs=(True, False))
    assert dx.shape == (4, 6, 16) and dw is None
    new = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert tg.grouped(new(0, 16), w, ends).shape == (0, 40)
    assert bool((tg.grouped(x[:, :0], w[:, :, :0], ends) == 0).all())
    out = torch.full((24, 40), 3.0, dtype=torch.bfloat16, device="cuda")
    two = _ends([10, 0, 4])
    tg.grouped(x[:, :0], w[:, :, :0], two, out=out)               # sums over nothing, in the groups' rows alone
    assert bool((out[:14] == 0).all()) and bool((out[14:] == 3).all())
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert bool((tg.grouped(x, w[:0], none) == 0).all())
    assert bool((tg.grouped(x, w[:0], none, out=torch.ones_like(out)) == 1).all())
    dx, dw = tg.grouped_backward(new(0, 40), new(0, 16), w, _ends([0, 0, 0]))
    assert dx.shape == (0, 16) and dw.shape == w.shape and bool((dw == 0).all())
    dx, dw = tg.grouped_backward(new(24, 0), x, w[:, :0], ends)
    assert bool((dx == 0).all()) and dw.shape == (3, 0, 16)
    a, b, index, bias = new(2, 8, 16), new(2, 40, 8), torch.zeros(24, dtype=torch.int32, device="cuda"), _randn(3, (40,), "bf16")
    assert tg.lora(new(0, 16), w[0], a, b, index[:0]).shape == (0, 40)
    assert torch.equal(tg.lora(x[:, :0], w[0][:, :0], a[:, :, :0], b, index, bias=bias), bias.expand(24, 40))
    base = tg.lora(x, w[0], a[:0], b[:0], index - 1, bias=bias)     # no adapters at all
    assert torch.equal(base, tg.lora(x, w[0], a, b, index - 1, bias=bias)) and torch.equal(base, tg.lora(x, w[0], a[:, :0], b[:, :, :0], index, bias=bias))
    assert torch.equal(tg.lora(x.view(4, 6, 16), w[0], a, b, index.view(4, 6)), tg.lora(x, w[0], a, b, index).view(4, 6, 40))
    _ok()


@pytest.mark.parametrize("ends", [[5, 3, 40], [-7, 10, 64], [70, 64, 64], [2 ** 31 - 1, -(2 ** 31), 9], [0, 0, 0]])
@pytest.mark.parametrize("N", [40, 2304])
def test_ends_that_break_the_rule(ends, N):
    """Ends that decrease or leave the rows: wrong rows, but every access inside, and the groups that are whole are right."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, _ = _operands(64, [1, 1, 1], N, 16, "f16")
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    guard = torch.full((3, 64, N), 5.0, dtype=torch.float16, device="cuda")
    tg.grouped(x, w, e, out=guard[1])
    tg.grouped_backward(_randn(3, (64, N), "f16"), x, w, e)
    _ok()
    assert bool((guard[0] == 5).all()) and bool((guard[2] == 5).all())


# ---------------------------------------------------------------------------
# Values that are not finite stay where they belong
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,sizes,N,K", [(90, [20, 33, 0, 30], 96, 72), (3000, [1000, 277, 0, 1500], 2304, 72)])
def test_nothing_crosses_groups(M, sizes, N, K):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, ends = _operands(M, sizes, N, K, "bf16")
    dy = _randn(9, (M, N), "bf16")
    y, tol = ref.grouped(ref.f64(x), ref.f64(w), sizes, "bf16")
    (dx, dw), (tx, tw) = ref.grouped_backward(ref.f64(dy), ref.f64(x), ref.f64(w), sizes, "bf16")
    lo, hi = ref.bounds(sizes)[1]
    x[lo:hi], dy[lo:hi] = float("nan"), float("inf")
    x[sum(sizes):], dy[sum(sizes):] = float("inf"), float("nan")
    w[1], w[2] = float("inf"), float("nan")
    got = tg.grouped(x, w, ends)
    gx, gw = tg.grouped_backward(dy, x, w, ends)
    _ok()
    keep = np.r_[0:lo, hi:M]
    kt = torch.from_numpy(keep).cuda()
    ref.check(ref.f64(got[kt]), y[keep], tol[keep], "y")
    ref.check(ref.f64(gx[kt]), dx[keep], tx[keep], "dx")
    for g in (0, 2, 3):
        ref.check(ref.f64(gw[g]), dw[g], tw[g], f"dw {g}")


@pytest.mark.parametrize("M,N,K", [(50, 96, 72), (2600, 4104, 72)])
@pytest.mark.parametrize("kind", ["random", "runs"])
def test_nothing_crosses_requests(M, N, K, kind):
    """A broken adapter, or broken rows, of one request change no other's results."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    rank, R = 16, 6
    x, w, a, b, index, ix = _lora_operands(M, N, K, rank, R, "f16", kind, seed=5)
    y, tol = ref.lora(ref.f64(x), ref.f64(w), ref.f64(a), ref.f64(b), index, None, None, "f16")
    broken = [r for r in range(R) if (index == r).any()][:2]
    a[broken[0]] = float("nan")
    b[broken[1]] = float("inf")
    rows = np.flatnonzero(index == index[0])  # rows that are broken themselves
    x[torch.from_numpy(rows).cuda()] = float("inf")
    got = tg.lora(x, w, a, b, ix)
    _ok()
    keep = np.flatnonzero(~np.isin(index, broken) & (index != index[0]))
    ref.check(ref.f64(got)[keep], y[keep], tol[keep], f"lora {kind}")
    assert not np.isfinite(ref.f64(got)[np.isin(index, broken)]).all()


# ---------------------------------------------------------------------------
# Large sizes, offsets past 32 bits
# ---------------------------------------------------------------------------

def test_rows_past_32_bits():
    """x, y and dy of more than 2^31 elements, the last groups behind that."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    K, N, M = 64, 72, 4000
    ld = 600_000  # elements between rows: 4.8 GB
    sizes = [100, 3800, 90]
    x0, w, ends = _operands(M, sizes, N, K, "f16")
    dy0 = _randn(5, (M, N), "f16")
    buf = torch.empty(M * ld, dtype=torch.float16, device="cuda")
    wide = buf.view(M, ld)
    x, dy, out = wide[:, :K], wide[:, 64:64 + N], wide[:, 256:256 + N]
    x.copy_(x0)
    dy.copy_(dy0)
    tg.grouped(x, w, ends, out=out)
    dx, dw = tg.grouped_backward(dy, x, w, ends)
    _ok()
    y, tol = ref.grouped(ref.f64(x0), ref.f64(w), sizes, "f16")
    used = sum(sizes)
    ref.check(ref.f64(out)[:used], y[:used], tol[:used], "y")
    for name, g, o, t in zip(("dx", "dw"), (dx, dw), *ref.grouped_backward(ref.f64(dy0), ref.f64(x0), ref.f64(w), sizes, "f16")):
        ref.check(ref.f64(g), o, t, name)


def test_weights_and_adapters_past_32_bits():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    G, N, K, M = 40, 8192, 8192, 128  # 2.7e9 elements of weights
    w = torch.zeros(G, N, K, dtype=torch.bfloat16, device="cuda")
    w[G - 1] = _randn(2, (N, K), "bf16", K ** -0.5)
    x = _randn(1, (M, K), "bf16")
    sizes = [0] * (G - 2) + [30, 98]
    got = tg.grouped(x, w, _ends(sizes))
    dy = _randn(3, (M, N), "bf16")
    dx, _ = tg.grouped_backward(dy, x, w, _ends(sizes), needs=(True, False))
    _ok()
    cols = np.array([0, 1, 127, 128, 4095, N - 1])
    ci = torch.from_numpy(cols).cuda()
    xs, ws = ref.f64(x[30:]), ref.f64(w[G - 1][ci])
    tol = ref.sum_error(np.abs(xs) @ np.abs(ws).T, K) + ref.round_error(xs @ ws.T, "bf16")
    ref.check(ref.f64(got[30:, ci]), xs @ ws.T, 1.01 * tol, "y")
    ds, ws = ref.f64(dy[30:]), ref.f64(w[G - 1][:, ci])
    tol = ref.sum_error(np.abs(ds) @ np.abs(ws), N) + ref.round_error(ds @ ws, "bf16")
    ref.check(ref.f64(dx[30:, ci]), ds @ ws, 1.01 * tol, "dx")
    assert bool((got[:30] == 0).all())
    # The same memory as adapters' B, the last of which lies behind 2^31 elements.
    rank = 64
    b = w.view(-1, N, rank)
    R = b.shape[0]
    a = _randn(6, (R, rank, 64), "bf16", 0.1)
    xk, wk = _randn(7, (M, 64), "bf16"), _randn(8, (N, 64), "bf16", 0.1)
    for kind in ("one", "mixed"):
        index = np.full(M, R - 1) if kind == "one" else np.where(np.arange(M) % 2 == 0, R - 1, R - 2)
        got = tg.lora(xk, wk, a, b, torch.from_numpy(index.astype(np.int32)).cuda())
        _ok()
        y, tol = _lora_last(xk, wk, a, b, index, cols, R, rank)
        ref.check(ref.f64(got[:, ci]), y, tol, f"lora {kind}")


def _lora_last(x, w, a, b, index, cols, R, rank):
    import torch
    ci = torch.from_numpy(cols).cuda()
    few = torch.tensor([R - 2, R - 1], device="cuda")
    return ref.lora(ref.f64(x), ref.f64(w[ci]), ref.f64(a[few]), ref.f64(b[few][:, ci]), index - (R - 2), None, None, "bf16")


@pytest.mark.parametrize("rank", [256, 512])
def test_deep_adapters(rank):
    import tiled_dense_gemm_fp16_b200 as tg
    for M, N, kind in ((40, 200, "random"), (2600, 4104, "runs")):
        x, w, a, b, index, ix = _lora_operands(M, N, 136, rank, 3, "f16", kind)
        got = tg.lora(x, w, a, b, ix)
        _ok()
        y, tol = ref.lora(ref.f64(x), ref.f64(w), ref.f64(a), ref.f64(b), index, None, None, "f16")
        ref.check(ref.f64(got), y, tol, f"lora rank {rank} {kind}")


# (rows, rank): few values of T, one and more a warp, ranks inside 32, rows whose values of T pass from one kernel to two.
@pytest.mark.parametrize("M,rank", [(1, 8), (1, 16), (1, 128), (1, 512), (2, 40), (5, 8), (8, 16), (9, 16), (16, 8), (33, 8), (64, 8)])
@pytest.mark.parametrize("N,K", [(72, 65), (264, 136), (2000, 4100), (5200, 1000), (129, 64), (40, 512)])
@pytest.mark.parametrize("kind", ["random", "one", "none"])
def test_few_rows(M, rank, N, K, kind):
    """A value of T for each row and rank, by whichever kernel; twice in a row, since the second call may start early."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    R = 6
    x, w, a0, b, index, ix = _lora_operands(M, N, K, rank, R, "bf16", kind, seed=M + rank)
    lda = (K + 7) // 8 * 8
    a = _stack(a0, lda, rank * lda)
    scale = torch.rand(R, generator=torch.Generator().manual_seed(1)).cuda() + 0.5
    bias = _randn(9, (N,), "bf16")
    y, tol = ref.lora(ref.f64(x), ref.f64(w), ref.f64(a0), ref.f64(b), index, ref.f64(scale), ref.f64(bias), "bf16")
    got = tg.lora(x, w, a, b, ix, scale=scale, bias=bias)
    again = tg.lora(x, w, a, b, ix, scale=scale, bias=bias)
    _ok()
    ref.check(ref.f64(got), y, tol, f"lora {M} {rank} {N} {K} {kind}")
    assert torch.equal(got, again)


def test_many_groups():
    import tiled_dense_gemm_fp16_b200 as tg
    rng = np.random.default_rng(0)
    for M, N in ((700, 40), (30000, 264)):
        sizes = rng.multinomial(M - 3, np.ones(1024) / 1024).tolist()
        x, w, ends = _operands(M, sizes, N, 24, "f16")
        dy = _randn(4, (M, N), "f16")
        y, tol = ref.grouped(ref.f64(x), ref.f64(w), sizes, "f16")
        got, grads = tg.grouped(x, w, ends), tg.grouped_backward(dy, x, w, ends)
        _ok()
        ref.check(ref.f64(got), y, tol, "y")
        for name, g, o, t in zip(("dx", "dw"), grads, *ref.grouped_backward(ref.f64(dy), ref.f64(x), ref.f64(w), sizes, "f16")):
            ref.check(ref.f64(g), o, t, name)


# ---------------------------------------------------------------------------
# Streams, graphs, repeats
# ---------------------------------------------------------------------------

def _calls(seed):
    """(run, expected) of calls that take every kernel; run(stream) returns their outputs."""
    import tiled_dense_gemm_fp16_b200 as tg
    small, big = _operands(60, [20, 0, 37], 200, 320, "f16", seed), _operands(2600, [1100, 1300, 177], 2304, 200, "bf16", seed + 10)
    dy = _randn(seed + 20, (2600, 2304), "bf16")
    few, many = _lora_operands(40, 264, 520, 16, 9, "f16", "random", seed), _lora_operands(2600, 4104, 136, 72, 9, "bf16", "runs", seed)

    def run(stream=None):
        return [tg.grouped(*small, stream=stream), tg.grouped(*big, stream=stream), *tg.grouped_backward(dy, *big, stream=stream),
                tg.lora(*few[:4], few[5], stream=stream), tg.lora(*many[:4], many[5], stream=stream)]
    return run


def _same(a, b):
    import torch
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


def test_equal_inputs_give_equal_bits():
    run = _calls(1)
    first = run()
    for _ in range(5):
        assert _same(first, run())
    _ok()


def test_two_streams_at_once():
    import torch
    runs = [_calls(1), _calls(2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[], []]
    for _ in range(6):
        for i, r in enumerate(runs):
            got[i].append(r(streams[i]))
    _ok()
    for i in range(2):
        assert all(_same(want[i], g) for g in got[i])


def test_results_of_one_call_feed_the_next():
    """Kernels start before the one before them has ended: what it writes is waited for."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    w = _randn(1, (3, 256, 256), "f16", 256 ** -0.5)
    a, b = _randn(2, (4, 16, 256), "f16", 256 ** -0.5), _randn(3, (4, 256, 16), "f16", 0.25)
    for M in (20, 3000):
        ends = _ends([M // 4, M // 2, M - M // 4 - M // 2])
        index = torch.randint(-1, 4, (M,), dtype=torch.int32, device="cuda")

        def chain(wait):
            x = _randn(4, (M, 256), "f16")
            for _ in range(8):
                x = tg.grouped(x, w, ends)
                wait()
                x = tg.lora(x, w[0], a, b, index)
                wait()
            return x
        assert torch.equal(chain(torch.cuda.synchronize), chain(lambda: None))
    _ok()


def test_gradients_feed_the_next_call():
    """dX is computed beside the last tiles of dW, and whoever reads either waits for both."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    for M, G in ((24, 3), (900, 3), (4000, 5)):
        w0 = _randn(1, (G, 256, 256), "f16", 256 ** -0.5)
        ends = _ends([M // G] * (G - 1) + [M - M // G * (G - 1)])
        x0, dy = _randn(4, (M, 256), "f16"), _randn(5, (M, 256), "f16", M ** -0.5 / 16)

        def chain(wait):
            x, w = x0, w0
            for _ in range(6):
                dx, dw = tg.grouped_backward(dy, x, w, ends)
                wait()
                y = tg.grouped(dx, dw, ends)
                wait()
                z, w = tg.grouped_backward(y, x0, w0, ends)
                wait()
                x = tg.grouped(z, dw, ends)
                wait()
            return x, w, dx, dw
        assert _same(chain(torch.cuda.synchronize), chain(lambda: None))
    _ok()


def test_captured_calls_with_other_groups():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    for M, N, K in ((50, 136, 200), (2600, 2304, 136)):
        x, w, ends = _operands(M, [M // 2, 0, M // 3], N, K, "f16")
        dy = _randn(5, (M, N), "f16")
        a, b = _randn(6, (5, 16, K), "f16", K ** -0.5), _randn(7, (5, N, 16), "f16", 0.25)
        index = torch.zeros(M, dtype=torch.int32, device="cuda")

        def step():
            return [tg.grouped(x, w, ends), *tg.grouped_backward(dy, x, w, ends), tg.lora(x, w[0], a, b, index)]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for seed, sizes in enumerate(([M, 0, 0], [1, M - 7, 3], [0, 0, 0], [M // 3, M // 3, M - 2 * (M // 3)])):
            ends.copy_(_ends(sizes))
            index.copy_(torch.from_numpy(_index("random" if seed % 2 else "runs", M, 5, seed).astype(np.int32)))
            x.copy_(_randn(20 + seed, (M, K), "f16"))
            graph.replay()
            torch.cuda.synchronize()
            assert _same(out, step()), sizes
    _ok()


def test_other_device():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    x, w, ends = (t.to("cuda:1") for t in _operands(60, [20, 40], 72, 40, "f16"))
    assert torch.equal(tg.grouped(x, w, ends).cpu(), tg.grouped(x.cuda(0), w.cuda(0), ends.cuda(0)).cpu())


# ---------------------------------------------------------------------------
# Autograd
# ---------------------------------------------------------------------------

def test_grouped_linear_gradients():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, sizes, N, K = 200, [64, 0, 77, 50], 136, 72
    x, w, ends = _operands(M, sizes, N, K, "f16")
    x, w = x.requires_grad_(), w.requires_grad_()
    dy = _randn(9, (M, N), "f16")
    tg.grouped_linear(x, w, ends).backward(dy)
    want = tg.grouped_backward(dy, x.detach(), w.detach(), ends)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])
    with torch.no_grad():
        y = tg.grouped_linear(x, w, ends)
    assert not y.requires_grad and torch.equal(y, tg.grouped(x.detach(), w.detach(), ends))
    (only,) = torch.autograd.grad(tg.grouped_linear(x, w, ends), [w], dy)
    assert torch.equal(only, want[1])
    with pytest.raises(RuntimeError, match="once_differentiable|twice|does not require"):
        g = torch.autograd.grad(tg.grouped_linear(x, w, ends).float().pow(2).sum(), [x], create_graph=True)[0]
        g.float().sum().backward()
    _ok()


def test_grouped_linear_of_views():
    """Broadcast weights and rows, transposed weights, expanded gradients: copied where the kernels cannot take them."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    sizes, N, K = [30, 34], 40, 24
    x, w, ends = _operands(64, sizes, N, K, "f16")
    one = w[0].clone().requires_grad_()
    tg.grouped_linear(x, one.expand(2, N, K), ends).sum().backward()
    dw = tg.grouped_backward(torch.ones(64, N, dtype=torch.float16, device="cuda"), x, one.detach().expand(2, N, K).contiguous(), ends)[1]
    assert torch.equal(one.grad, dw.sum(0))
    row = x[0].clone().requires_grad_()
    tg.grouped_linear(row.expand(64, K), w, ends).sum().backward()
    dx = tg.grouped_backward(torch.ones(64, N, dtype=torch.float16, device="cuda"), row.detach().expand(64, K).contiguous(), w, ends)[0]
    assert torch.equal(row.grad, dx.sum(0))
    t = w.transpose(1, 2).contiguous().requires_grad_()  # (G, K, N)
    tg.grouped_linear(x, t.transpose(1, 2), ends).sum().backward()
    want = tg.grouped_backward(torch.ones(64, N, dtype=torch.float16, device="cuda"), x, w, ends)[1]
    assert torch.equal(t.grad, want.transpose(1, 2))
    _ok()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gradients_against_differences(dt):
    """Along random directions: the loss is linear in x and in w, so a difference quotient has no error of its own; it is taken
    in 64 bits from the outputs, each off by half a step at most."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, sizes, N, K = 96, [40, 0, 56], 64, 48
    x, w, ends = _operands(M, sizes, N, K, dt)
    dy = _randn(3, (M, N), dt)
    dx, dw = tg.grouped_backward(dy, x, w, ends)
    for i, (t, g) in enumerate(((x, dx), (w, dw))):
        d = _randn(10 + i, tuple(t.shape), dt, 2.0 ** -3)
        ends_of = []
        for s in (1, -1):
            args = [x, w]
            args[i] = t + s * d
            ends_of.append((args[i].double(), tg.grouped(*args, ends).double()))
        step = (ends_of[0][0] - ends_of[1][0])  # what the rounded steps really were
        slope = ((ends_of[0][1] - ends_of[1][1]) * dy.double()).sum()
        half = ff_ref.HALF[dt]
        tol = half * sum((y.abs() * dy.double().abs()).sum() for _, y in ends_of) + half * (step.abs() * g.double().abs()).sum()
        assert abs(float(slope - (step * g.double()).sum())) <= 1.05 * float(tol), i
    _ok()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tokens", [7, 900])
def test_a_block_of_experts_behind_an_adapted_projection(tokens):
    """A projection with adapters, a router, the gated experts and their sum, against the same steps in 64 bits on the 16-bit
    values between them."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    D, F, E, top, dt = 128, 192, 6, 2, "bf16"
    x, w, a, b, index, ix = _lora_operands(tokens, D, D, 16, 4, dt, "random")
    h = tg.lora(x, w, a, b, ix)
    y, tol = ref.lora(ref.f64(x), ref.f64(w), ref.f64(a), ref.f64(b), index, None, None, dt)
    ref.check(ref.f64(h), y, tol, "projection")
    gate_up, down = _randn(11, (E, 2 * F, D), dt, D ** -0.5), _randn(12, (E, D, F), dt, F ** -0.5)
    probs, expert = torch.softmax(h.float() @ _randn(13, (D, E), dt, D ** -0.5).float(), -1).topk(top)
    order = expert.flatten().argsort(stable=True)
    counts = torch.bincount(expert.flatten(), minlength=E)
    ends = counts.cumsum(0, dtype=torch.int32)
    rows = h[order // top]
    both = tg.grouped(rows, gate_up, ends)
    assert torch.equal(tg.grouped(rows, gate_up[:, :F], ends), both[:, :F])  # half of a fused weight
    act = (torch.nn.functional.silu(both[:, :F].float()) * both[:, F:].float()).to(h.dtype)
    out = tg.grouped(act, down, ends)
    _ok()
    sizes = counts.tolist()
    y, tol = ref.grouped(ref.f64(rows), ref.f64(gate_up), sizes, dt)
    ref.check(ref.f64(both), y, tol, "gate and up")
    y, tol = ref.grouped(ref.f64(act), ref.f64(down), sizes, dt)
    ref.check(ref.f64(out), y, tol, "down")
    mixed = torch.zeros(tokens, D, device="cuda").index_add_(0, order // top, out.float() * probs.flatten()[order, None])
    assert bool(torch.isfinite(mixed).all())


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------

def test_refusals():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, ends = _operands(24, [10, 14], 40, 16, "f16")
    a, b, ix = _randn(3, (2, 8, 16), "f16"), _randn(4, (2, 40, 8), "f16"), torch.zeros(24, dtype=torch.int32, device="cuda")
    dy = _randn(5, (24, 40), "f16")
    for error, call in (
            (TypeError, lambda: tg.grouped(x.float(), w.float(), ends)), (TypeError, lambda: tg.grouped(x, w.bfloat16(), ends)),
            (TypeError, lambda: tg.grouped(x, w, ends.long())), (ValueError, lambda: tg.grouped(x, w, ends.cpu())),
            (ValueError, lambda: tg.grouped(x, w, ends[:1])), (ValueError, lambda: tg.grouped(x, w[0], ends)),
            (ValueError, lambda: tg.grouped(x, w[:, :, :8], ends)), (ValueError, lambda: tg.grouped(x[:, ::2], w[:, :, :8], ends)),
            (ValueError, lambda: tg.grouped(x, w.transpose(1, 2).contiguous().transpose(1, 2), ends)),
            (ValueError, lambda: tg.grouped(x, w[:1].expand(2, 40, 16), ends)), (ValueError, lambda: tg.grouped(x[:1].expand(24, 16), w, ends)),
            (ValueError, lambda: tg.grouped(x, w, ends, out=dy[:, :39])), (TypeError, lambda: tg.grouped(x, w, ends, out=dy.float())),
            (tg.TGError, lambda: tg.grouped(x, w, ends, out=w.view(-1)[:960].view(24, 40))),
            (tg.TGError, lambda: tg.grouped(x[:, 1:], w[:, :, 1:], ends, workspace=None)),
            (ValueError, lambda: tg.grouped(x, w, ends, workspace=x)), (ValueError, lambda: tg.grouped(x, w, ends, workspace="none")),
            (ValueError, lambda: tg.grouped_backward(dy[:, :39], x, w, ends)), (TypeError, lambda: tg.grouped_backward(dy.bfloat16(), x, w, ends)),
            (tg.TGError, lambda: tg.grouped_backward(dy[:, 1:], x, w[:, 1:], ends, workspace=None)),
            (ValueError, lambda: tg.lora(x, w[0], a[:, :4], b[:, :, :4], ix)), (ValueError, lambda: tg.lora(x, w[0], a, b, ix[:5])),
            (TypeError, lambda: tg.lora(x, w[0], a, b, ix.long())), (ValueError, lambda: tg.lora(x, w[0], a, b[:, :39], ix)),
            (ValueError, lambda: tg.lora(x[:, :12], w[0][:, :12], a[:, :, :12].contiguous(), b, ix)),
            (TypeError, lambda: tg.lora(x, w[0], a, b, ix, scale=torch.ones(2, device="cuda").half())),
            (ValueError, lambda: tg.lora(x, w[0], a, b, ix, scale=torch.ones(3, device="cuda"))),
            (TypeError, lambda: tg.lora(x, w[0], a, b, ix, bias=torch.ones(40, device="cuda"))),
            (tg.TGError, lambda: tg.lora(x, w[0], a, b, ix, workspace=None)),
            (tg.TGError, lambda: tg.lora(x, w[0], a, b, ix, out=w.view(-1)[:960].view(24, 40))),
            (NotImplementedError, lambda: _dual(tg, x, w, ends))):
        with pytest.raises(error):
            call()
    _ok()
    tg.grouped(x, w, ends)
    _ok()


def _dual(tg, x, w, ends):
    import torch
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        tg.grouped_linear(forward_ad.make_dual(x, torch.ones_like(x)), w, ends)


def test_first_calls_of_host_threads():
    """A thread whose first call is one of these, with memory out of torch's cache."""
    import threading

    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, ends = _operands(60, [20, 40], 72, 40, "f16")
    dy = _randn(5, (60, 72), "f16")
    a, b, ix = _randn(3, (2, 8, 40), "f16"), _randn(4, (2, 72, 8), "f16"), torch.zeros(60, dtype=torch.int32, device="cuda")
    calls = (lambda: [tg.grouped(x, w, ends)], lambda: tg.grouped_backward(dy, x, w, ends), lambda: [tg.lora(x, w[0], a, b, ix)])
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for c, first in zip(calls, want):
        got = []
        t = threading.Thread(target=lambda: got.extend(c()))
        t.start()
        t.join()
        _ok()
        assert len(got) == len(first) and _same(got, first)
