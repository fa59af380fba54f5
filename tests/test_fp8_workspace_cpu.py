"""The size query of the e4m3 product: the workspace for any operands (whole_rows 0, which is
what a caller asks for who does not know their layout) holds what every layout needs.  No GPU
needed."""
import pytest

from trellis_coded_weight_amd import _native as nat

ROWS = [1, 4, 8, 16, 32, 33, 40, 48, 49, 64, 65, 100, 300, 1000]
COLS = [1, 16, 128, 512, 1024, 4096, 8208, 28672]
INNER = [16, 128, 1024, 1536, 2048, 4096, 8192, 14336]


@pytest.mark.parametrize("M", ROWS)
def test_workspace_for_any_operands_holds_that_of_whole_rows(M):
    for N in COLS:
        for K in INNER:
            some, whole = (nat.qtcq_matmul_fp8_workspace_bytes(M, N, K, w) for w in (False, True))
            assert some >= whole, (M, N, K, some, whole)


def test_workspace_of_the_other_products_too():
    for query in (nat.qtcq_matmul_int8_workspace_bytes, nat.qtcq_gated_workspace_bytes):
        for M in ROWS:
            for N in COLS:
                for K in INNER:
                    assert query(M, N, K, False) >= query(M, N, K, True), (query.__name__, M, N, K)
