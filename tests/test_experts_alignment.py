"""Alignment rules of K x N expert weights, refused before anything touches a device: rows of
N elements on 16 bytes, and with a gated activation rows of N / 2 (the up half is copied
from its own start)."""
import pytest

import dense_gemm_persistent_gb300 as dg
from dense_gemm_persistent_gb300 import build

MISALIGNED, KN, NK, NONE, SWIGLU = 3, 0, 1, 0, 4
P = 4096   # an aligned non-null address: never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dg.load()


def grouped(lib, layout, act, N, R=32):
    return lib.dgemm_grouped_bf16(P, R, None, P, layout, P, 4, P, 1, R, N, 128, 1.0, None, act, None, 0, None)


@pytest.mark.parametrize("N", [8, 24, 40, 120, 2056])
def test_gated_kn_needs_sixteen_channels(lib, N):
    assert grouped(lib, KN, SWIGLU, N) == MISALIGNED
    assert grouped(lib, KN, SWIGLU, N, R=0) == MISALIGNED      # by its sizes, whatever the rows
    assert grouped(lib, KN, NONE, N, R=0) == 0
    assert grouped(lib, NK, SWIGLU, N, R=0) == 0


@pytest.mark.parametrize("N", [4, 12, 20, 100])
def test_kn_needs_eight_channels(lib, N):
    assert grouped(lib, KN, NONE, N) == MISALIGNED
    assert grouped(lib, NK, NONE, N, R=0) == 0


@pytest.mark.parametrize("N", [16, 32, 48, 2048])
def test_gated_kn_in_range(lib, N):
    assert grouped(lib, KN, SWIGLU, N, R=0) == 0
