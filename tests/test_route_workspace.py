"""The routing call's workspace leaves room for the status word at its start."""
import pytest

import dense_gemm_persistent_gb300 as dg
from dense_gemm_persistent_gb300 import build

STATUS_BYTES, CHUNK = 256, 64     # DGEMM_WS_STATUS_BYTES; most tokens of a chunk


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.mark.parametrize("T,E,k", [(65, 1, 1), (65, 5, 2), (128, 64, 8), (5000, 257, 4), (16001, 256, 8), (100000, 1024, 32)])
def test_counts_come_behind_the_status_word(T, E, k):
    """Up to 64 chunks more than the fewest, a byte an expert (rounded up to four) in each."""
    most = (T + CHUNK - 1) // CHUNK + 64
    assert dg.dgemm_route_workspace_size(T, E, k) == STATUS_BYTES + most * ((E + 3) // 4 * 4)


@pytest.mark.parametrize("T", [0, 1, 64])
def test_one_chunk_needs_none(T):
    assert dg.dgemm_route_workspace_size(T, 16, 2) == 0
