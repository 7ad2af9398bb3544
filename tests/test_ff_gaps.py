"""Matrices of the feed-forward calls in the gaps between each other's rows: which ones overlap (host logic only; without
a GPU a call that passes every check ends in UNSUPPORTED_DEVICE)."""
import itertools

import pytest

import tiled_dense_gemm_fp16_b200 as tg
from tiled_dense_gemm_fp16_b200 import Status

P = [0x10_0000_0000 * (i + 1) for i in range(12)]
BAD, TAKEN = Status.INVALID_ARG, Status.UNSUPPORTED_DEVICE


def _gpu():
    import torch
    return torch.cuda.is_available()


pytestmark = pytest.mark.skipif("_gpu()", reason="fake addresses must not reach a device")

M, N, K = 5, 24, 32


def gated(h, g, u, ldh, ldg, ldu, x=P[0], ldx=0, m=M):
    opts = tg.gated_options(ldh=ldh, ldg=ldg, ldu=ldu, ldx=ldx)
    return tg.gated_raw(x, P[1], P[2], h, g, u, m, N, K, opts, 0, P[9], 1 << 20)


def test_results_side_by_side():
    """H, G and U as column ranges of one buffer, in any order; one element too close is refused."""
    wide = 3 * N
    for order in itertools.permutations(range(3)):
        h, g, u = (P[3] + 2 * N * i for i in order)
        assert gated(h, g, u, wide, wide, wide) == TAKEN
        assert gated(h, g, u, wide - 8, wide - 8, wide - 8) == BAD      # the last range runs into the first's next row
        assert gated(h, g, u, wide, wide, wide + 8) == BAD              # another pitch
    assert gated(P[3], P[3] + 2 * N - 2, P[3] + 4 * N, wide, wide, wide) == BAD
    assert gated(P[3] + 2, P[3] + 2 * N, P[3] + 4 * N, wide, wide, wide) == BAD
    # A range that starts in another row is judged by its columns.
    assert gated(P[3], P[3] + 2 * (N + 2 * wide), P[3] + 2 * (2 * N - wide), wide, wide, wide) == TAKEN
    assert gated(P[3], P[3] + 2 * (N + 2 * wide), P[3] + 2 * (2 * N - wide) - 2, wide, wide, wide) == BAD


def test_result_beside_an_input():
    wide = K + N
    assert gated(P[0] + 2 * K, 0, 0, wide, 0, 0, ldx=wide) == TAKEN
    assert gated(P[0], 0, 0, wide, 0, 0, x=P[0] + 2 * N, ldx=wide) == TAKEN
    assert gated(P[0] + 2 * K - 2, 0, 0, wide, 0, 0, ldx=wide) == BAD
    assert gated(P[0] + 2 * K, 0, 0, wide - 1, 0, 0, ldx=wide - 1) == BAD
    assert gated(P[0] + 2 * K, 0, 0, 2 * wide, 0, 0, ldx=wide) == BAD


def test_single_rows():
    """A matrix of one row in the gap of one with several; two single rows by their ranges."""
    assert gated(P[0] + 2 * K, 0, 0, 0, 0, 0, m=1) == TAKEN and gated(P[0] + 2 * K - 2, 0, 0, 0, 0, 0, m=1) == BAD
    ldc = 2 * N + 8  # gaps of N + 8 values
    def product(bias):
        return tg.gemm_i8_raw(P[0], P[1], P[2], P[3], bias, P[5], M, N, K, ldc=ldc)
    for row in (0, M - 2):
        gap = P[5] + 2 * (row * ldc + N)
        assert product(gap) == TAKEN and product(gap + 16) == TAKEN
        assert product(gap - 2) == BAD and product(gap + 18) == BAD
    assert product(P[5] + 2 * ((M - 1) * ldc + N)) == TAKEN  # behind the last row


def test_codes_beside_values():
    """Codes and values of rows with one pitch in bytes."""
    assert tg.quantize_rows_i8_raw(P[0], P[0] + 2 * K, P[2], M, K, ldx=2 * K, ldq=4 * K) == TAKEN
    assert tg.quantize_rows_i8_raw(P[0], P[0] + 2 * K - 1, P[2], M, K, ldx=2 * K, ldq=4 * K) == BAD
    assert tg.quantize_rows_i8_raw(P[0], P[0] + 3 * K + 1, P[2], M, K, ldx=2 * K, ldq=4 * K) == BAD
    assert tg.quantize_rows_i8_raw(P[0], P[0] + 2 * K, P[2], M, K, ldx=2 * K, ldq=2 * K) == BAD


def test_every_pair_of_column_ranges():
    """The answer is that of marking each byte, for every offset of H against X."""
    for ld_x, ld_h in ((56, 56), (60, 60), (56, 64)):
        x_bytes = {2 * (r * ld_x + c) + b for r in range(M) for c in range(K) for b in (0, 1)}
        for off in range(-2 * M * ld_h - 4, 2 * M * ld_x + 6, 2):
            h_bytes = {off + 2 * (r * ld_h + c) for r in range(M) for c in range(N)}
            meets = any(b in x_bytes for b in h_bytes)
            got = gated(P[0] + off, 0, 0, ld_h, 0, 0, ldx=ld_x)
            if meets:
                assert got == BAD, (ld_x, ld_h, off)
            elif ld_x == ld_h and 0 <= off <= 2 * (M - 1) * ld_x:
                assert got == TAKEN, (ld_x, ld_h, off)
