"""Adapters in fp16 whose inner products lie outside fp16: scale A X of 1e6 or 1e-7 beside B, with results that are ordinary
numbers.  Against the definition in 64 bits.

As in grp_ref, with one difference: an inner product is rounded in steps of its own or of its row's largest magnitude, so it
is off by 2^-11 of either, wherever they lie; fp16's smallest step does not enter.  B T is summed in fp32 by warp-level or
tcgen05 MMAs of 16 ranks, each addition off by at most 2^-22 of the magnitudes: within (rank / 8 + 4) 2^-22 |B||T|."""
import numpy as np
import pytest

import grp_ref as ref
from test_gpu_grp import _ok, _randn

pytestmark = pytest.mark.gpu


def _reference(x, w, a, b, index, scale, bias):
    M, K = x.shape
    rank = a.shape[1]
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = ref.sum_error(mag, K)
    for r in sorted(set(index.tolist())):
        if not 0 <= r < a.shape[0]:
            continue
        at = np.flatnonzero(index == r)
        t = scale[r] * (x[at] @ a[r].T)
        err = abs(scale[r]) * ref.sum_error(np.abs(x[at]) @ np.abs(a[r]).T, K) + np.abs(t) * 2.0 ** -23
        top = np.abs(t).max(1, keepdims=True)
        err = 1.01 * err + 2.0 ** -11 * (np.abs(t) + top)
        product = (np.abs(t) + err) @ np.abs(b[r]).T
        y[at] += t @ b[r].T
        mag[at] += product
        tol[at] += err @ np.abs(b[r]).T + (rank / 8 + 4) * 2.0 ** -22 * product
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    tol = 1.01 * (tol + 3 * 2.0 ** -24 * mag)
    return y, tol + ref.round_error(y, "f16")


# |A| sqrt(K), scale, |B| sqrt(rank), |W| sqrt(K): inner products of about |A| sqrt(K) scale
RANGES = {"loud": (2.0 ** 8, 2.0 ** 12, 2.0 ** -12, 1.0), "quiet": (2.0 ** -9, 2.0 ** -12, 2.0 ** 9, 2.0 ** -13)}


def _operands(M, N, K, rank, kinds, seed=1):
    """Adapters of the given kinds in turn, "loud", "quiet" or "plain"; W as the quietest of them wants it."""
    import torch
    parts = [RANGES.get(k, (1.0, 1.0, 1.0, 1.0)) for k in kinds]
    x = _randn(seed, (M, K), "f16")
    w = _randn(seed + 1, (N, K), "f16", K ** -0.5 * min(p[3] for p in parts))
    a = torch.stack([_randn(seed + 2 + 2 * i, (rank, K), "f16", p[0] * K ** -0.5) for i, p in enumerate(parts)])
    b = torch.stack([_randn(seed + 3 + 2 * i, (N, rank), "f16", p[2] * rank ** -0.5) for i, p in enumerate(parts)])
    return x, w, a, b, torch.tensor([1.1 * p[1] for p in parts], device="cuda")


def _index(layout, M, R):
    if layout == "runs":  # blocks of 32 rows of one adapter, and some of two
        return (np.arange(M) // 75 + 1) % (R + 1) - 1
    if layout == "one":
        return np.zeros(M, np.int64)
    return np.random.default_rng(M).integers(-1, R, M)


def _check(M, N, K, rank, kinds, layout, what, change=None, with_bias=True):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, a, b, scale = _operands(M, N, K, rank, kinds)
    if change is not None:
        change(x, a)
    index = _index(layout, M, len(kinds))
    bias = _randn(90, (N,), "f16", 2.0 ** -8) if with_bias else None
    got = tg.lora(x, w, a, b, torch.from_numpy(index.astype(np.int32)).cuda(), scale=scale, bias=bias)
    _ok()
    y, tol = _reference(*(ref.f64(t) for t in (x, w, a, b)), index, ref.f64(scale), None if bias is None else ref.f64(bias))
    assert np.abs(y).max() < 60000
    ref.check(ref.f64(got), y, tol, what)


# One token and two, whose inner products the main kernel makes itself (over 2 and 4 CTAs); a kernel with a warp each;
# blocks of 32, 64 and 128 tokens, with and without a split of their sums, ranks of one, two and four times 128.
SIZES = [(1, 264, 136, 8), (1, 264, 520, 16), (2, 136, 520, 8), (1, 5200, 520, 16), (5, 264, 136, 24), (40, 264, 520, 16), (96, 136, 72, 72),
         (128, 72, 2056, 8), (200, 264, 520, 16), (200, 520, 64, 40), (200, 264, 264, 136), (300, 264, 200, 512), (1500, 264, 136, 64),
         (1500, 136, 264, 8), (9600, 72, 72, 16)]


@pytest.mark.parametrize("M,N,K,rank", SIZES)
@pytest.mark.parametrize("kind", ["loud", "quiet"])
@pytest.mark.parametrize("layout", ["one", "runs", "random"])
def test_inner_products_outside_the_type(M, N, K, rank, kind, layout):
    _check(M, N, K, rank, [kind] if layout == "one" else [kind] * 3, layout, f"{kind} {layout} {M} {N} {K} {rank}")


@pytest.mark.parametrize("M,N,K,rank", SIZES)
@pytest.mark.parametrize("layout", ["runs", "random"])
def test_requests_of_all_ranges_beside_each_other(M, N, K, rank, layout):
    """Each row as near as alone: quiet rows lose nothing beside loud ones."""
    _check(M, N, K, rank, ["plain", "loud", "quiet", "plain", "loud"], layout, f"{layout} {M} {N} {K} {rank}", with_bias=False)


@pytest.mark.parametrize("M,N,K,rank", SIZES)
@pytest.mark.parametrize("kind", ["loud", "quiet", "plain"])
def test_single_rows_and_ranks_outside(M, N, K, rank, kind):
    """One row of 37 louder, one of 41 quieter, one of 43 zero; the ranks' magnitudes 2^-20 .. 1 apart."""
    def change(x, a):
        import torch
        x[::37] *= 8
        x[5::41] *= 2.0 ** -8
        x[11::43] = 0
        a *= torch.exp2(-(torch.arange(rank, device="cuda") % 21).float()).half()[None, :, None]
    _check(M, N, K, rank, [kind], "one", f"{kind} {M} {N} {K} {rank}", change=change)


def test_edges_of_the_range():
    """Inner products that are exactly the borders between plain and divided ones, and fp16's largest and smallest."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    values = [0.0, 2.0 ** -140, 2.0 ** -112, 2.0 ** -100, 2.0 ** -30, 2.0 ** -25, 2.0 ** -24, 2.0 ** -15, 2.0 ** -14 * (1 - 2.0 ** -11), 2.0 ** -14, 1.0, 32736.0, 32751.0, 32752.0, 32760.0, 32768.0, 65504.0,
              65519.0, 65520.0, 65535.0, 65536.0, 2.0 ** 30, 2.0 ** 60, 2.0 ** 100]
    K, N = 72, 40
    for rank in (8, 16):
        for M in (1, 20, 200):
            for v in values:
                x = torch.zeros(M, K, dtype=torch.float16, device="cuda")
                x[:, 0] = 1
                a = torch.zeros(1, rank, K, dtype=torch.float16, device="cuda")
                a[0, rank - 3, 0] = 1
                b = torch.zeros(1, N, rank, dtype=torch.float16, device="cuda")
                b[0, :, rank - 3] = 2.0 ** (-12 if v > 1 else 12)
                w = torch.zeros(N, K, dtype=torch.float16, device="cuda")
                index = torch.zeros(M, dtype=torch.int32, device="cuda")
                got = tg.lora(x, w, a, b, index, scale=torch.tensor([v], device="cuda"))
                _ok()
                want = v * 2.0 ** (-12 if v > 1 else 12)
                if want > 65536:
                    assert bool(torch.isinf(got).all()), (rank, M, v)
                else:
                    # Two roundings of 2^-11, and half of the result's own smallest step: 2^-140 2^12 can only be 0.
                    assert float((got.double() - want).abs().max()) <= 2.0 ** -10 * 1.001 * want + 2.0 ** -25, (rank, M, v)


def test_values_that_are_not_finite_beside_powers():
    """Rows or adapters that are not finite leave the divided rows beside them as they are."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    for M, N, K, rank in ((1, 264, 520, 16), (40, 264, 520, 16), (200, 264, 520, 40), (1500, 136, 264, 136)):
        for layout in ("runs", "random", "one"):
            kinds = ["loud"] if layout == "one" else ["loud", "quiet", "loud"]
            x, w, a, b, scale = _operands(M, N, K, rank, kinds)
            index = _index(layout, M, len(kinds))
            y, tol = _reference(*(ref.f64(t) for t in (x, w, a, b)), index, ref.f64(scale), None)
            x[3::7] = float("inf")
            x[4::11, 5] = float("nan")
            if layout != "one":
                a[2], b[2] = float("nan"), float("inf")
            rows = np.arange(M)
            broken = ((rows - 3) % 7 == 0) & (rows >= 3) | ((rows - 4) % 11 == 0) & (rows >= 4) | (index == 2)
            got = ref.f64(tg.lora(x, w, a, b, torch.from_numpy(index.astype(np.int32)).cuda(), scale=scale))
            _ok()
            ref.check(got[~broken], y[~broken], tol[~broken], f"{layout} {M}")
            assert not np.isfinite(got[broken]).any()


def test_a_workspace_that_held_powers():
    """What one call left in the workspace says nothing to the next; a captured call replayed with other magnitudes."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    for M, N, K, rank in ((40, 264, 520, 16), (200, 264, 520, 40), (1500, 136, 264, 136)):
        x, w, a, b, scale = _operands(M, N, K, rank, ["loud", "loud", "quiet"])
        index = torch.from_numpy(_index("runs", M, 3).astype(np.int32)).cuda()
        one = torch.ones(3, device="cuda") * 2.0 ** -8
        size = tg.lora_workspace_size(x.data_ptr(), w.data_ptr(), M, N, K, rank, 3)
        ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
        want = {id(s): tg.lora(x, w, a, b, index, scale=s) for s in (scale, one)}
        for s in (one, scale, one, one, scale):
            assert torch.equal(tg.lora(x, w, a, b, index, scale=s, workspace=ws), want[id(s)])
        held = scale.clone()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = tg.lora(x, w, a, b, index, scale=held, workspace=ws)
        for s in (scale, one, scale):
            held.copy_(s)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[id(s)])
    _ok()
