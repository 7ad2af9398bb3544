"""C rows that start on 16-byte boundaries and end inside 16 bytes: the values behind each row, and behind the last one,
stay (run_ex checks both), on every kernel."""
import pytest

from gpu_util import assert_bitexact
from test_gpu_layouts import run_ex
from tiled_dense_gemm_fp16_b200 import Path

pytestmark = pytest.mark.gpu

PATHS = {"auto": Path.AUTO, "tc": Path.TC, "pair": Path.TC_PAIR, "pair512": Path.TC_PAIR512, "skinny": Path.SKINNY}


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("N,ldc", [(1, 8), (33, 40), (261, 264), (517, 528), (1002, 1008), (1028, 1032)])
def test_values_behind_rows(N, ldc, path):
    for M in (40, 200) if path == "skinny" else (40, 200, 530):
        got, ref, guards = run_ex(M, N, 136, lda=136, ldb=136, ldc=ldc, b_nk=True, bias=True, path=PATHS[path], seed=M + N)
        assert guards
        assert_bitexact(got[0], ref[0], f"{(M, N)} {path}")


@pytest.mark.parametrize("a_km", [False, True], ids=["A_MK", "A_KM"])
@pytest.mark.parametrize("b_nk", [False, True], ids=["B_KN", "B_NK"])
def test_values_behind_rows_of_other_layouts(a_km, b_nk):
    """Operands that need copies, and a batch whose entries follow one another closely."""
    M, N, K = 300, 261, 137
    got, ref, guards = run_ex(M, N, K, lda=(M if a_km else K) + 3, ldb=(K if b_nk else N) + 3, ldc=264, b_nk=b_nk, bias=False,
                              a_km=a_km, batch=2, gap=3, seed=5)
    assert guards
    for g, r in zip(got, ref):
        assert_bitexact(g, r, "batch entry")
